"""gemm_linear_grad without an activation: a copy of dy with offsets, where rows of no group are zero, and dy itself without."""
import pytest

from linear_helpers import KINDS, L, buffer, no_device_error, require_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("act", [None, "none"])
@pytest.mark.parametrize("ends", [[0, 40, 40, 77], [9, 20, 60, 70], [5, 5], [0, 77]])
def test_rows_of_no_group_are_zero(ends, act, kind, bias):
    require_gpu()
    rows, n = 77, 264
    dy = torch.randn(rows, n, device="cuda").to(KINDS[kind])
    dy[: ends[0]], dy[ends[-1]:] = float("inf"), float("nan")
    was = dy.clone()
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out = L.gemm_linear_grad(dy, act=act, offsets=offsets, bias_grad=bias, workspace=buffer(len(ends) - 1, rows, n, 0))
    dz, db = out if bias else (out, None)
    no_device_error()
    assert dz.data_ptr() != dy.data_ptr() and torch.equal(dy.view(torch.int16), was.view(torch.int16))
    assert not dz[: ends[0]].any() and not dz[ends[-1]:].any()
    assert torch.equal(dz[ends[0]:ends[-1]], dy[ends[0]:ends[-1]])
    if bias:
        for g in range(len(ends) - 1):
            part = dy[ends[g]:ends[g + 1]].double()
            # a sum of at most 77 values in fp32, in any order
            assert ((db[g].double() - part.sum(0)).abs() <= 77 * 2.0 ** -24 * part.abs().sum(0)).all()
    # in place, and into another tensor
    other = torch.full_like(dy, 7.0)
    assert L.gemm_linear_grad(dy, act=act, offsets=offsets, dz=other) is other and torch.equal(other, dz)
    assert L.gemm_linear_grad(dy, act=act, offsets=offsets, dz=dy) is dy and torch.equal(dy, dz)
    no_device_error()


def test_without_offsets_it_is_dy():
    require_gpu()
    dy = torch.randn(33, 72, device="cuda").half()
    assert L.gemm_linear_grad(dy) is dy
    copy = torch.empty_like(dy)
    assert L.gemm_linear_grad(dy, dz=copy) is copy and torch.equal(copy, dy)
    no_device_error()
