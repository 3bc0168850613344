"""Matrices of more than 2^32 elements: the last rows, and sums over all of them, of the products with an epilogue and their
gradients."""
import numpy as np
import pytest

from linear_helpers import G, L, buffer, eighths, grad_ref, near, no_device_error, nt_ref, offsets_of, require_gpu, rounded, torch

pytestmark = pytest.mark.gpu

ROWS, WIDE, NARROW = (1 << 20) + 77, 4104, 24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")


def ends():
    """Rows at the start, around 2^32 elements, and at the end."""
    at = (1 << 32) // WIDE
    return torch.cat([torch.arange(0, 40), torch.arange(at - 20, at + 20), torch.arange(ROWS - 40, ROWS)])


def fill(rng, rows, cols):
    """A piece of random rows again and again."""
    piece = eighths(rng, (1009, cols), torch.float16).cuda()
    return piece.repeat(-(-rows // 1009), 1)[:rows].contiguous()


@pytest.mark.parametrize("grouped", [False, True])
def test_forward(grouped):
    rng = np.random.default_rng(1)
    x, r, at = fill(rng, ROWS, NARROW), fill(rng, ROWS, WIDE), ends()
    offsets = offsets_of([ROWS - 60, 60]) if grouped else None
    stack = (2,) if grouped else ()
    w, b = eighths(rng, stack + (WIDE, NARROW), torch.float16), eighths(rng, stack + (WIDE,), torch.float16)
    y, z = L.gemm_linear_nt(x, w.cuda(), bias=b.cuda(), residual=r, act="silu", offsets=None if offsets is None else offsets.cuda(), keep=True,
                            workspace=buffer(2 if grouped else 1, ROWS, WIDE, NARROW))
    no_device_error()
    few = None if offsets is None else offsets_of([int((at < ROWS - 60).sum()), int((at >= ROWS - 60).sum())])
    want, off, zz = nt_ref(x[at].cpu(), w, b, r[at].cpu(), "silu", few)
    assert torch.equal(z[at].cpu(), zz.half())
    near(y[at].cpu(), want, rounded(torch.float16, want, off), "y")


def test_backward():
    rng = np.random.default_rng(2)
    dy, z, at = fill(rng, ROWS, NARROW), fill(rng, ROWS, WIDE), ends()
    w = eighths(rng, (NARROW, WIDE), torch.float16)
    dx, db = L.gemm_linear_nn(dy, w.cuda(), z=z, act="relu", bias_grad=True, workspace=buffer(1, ROWS, NARROW, WIDE))
    no_device_error()
    d = dy[at].double().cpu() @ w.double()
    want, off, _, _ = grad_ref(d, z[at].cpu(), "relu", None)
    near(dx[at].cpu(), want, rounded(torch.float16, want, off), "dx")
    # relu passes what it passes whole: the sum over all rows, of multiples of 1/64, in 64 bits
    # (at most 660 additions one after another: 128 rows of a tile, 4097 tiles over eight warps, and theirs)
    sums, sizes = torch.zeros(WIDE, dtype=torch.float64), torch.zeros(WIDE, dtype=torch.float64)
    for lo in range(0, ROWS, 1 << 16):
        hi = min(lo + (1 << 16), ROWS)
        terms = (dy[lo:hi].double() @ w.double().cuda()) * (z[lo:hi] > 0)
        sums += terms.sum(0).cpu()
        sizes += terms.abs().sum(0).cpu()
    near(db.cpu(), sums, 660 * 2.0 ** -24 * sizes, "dbias")
    del dx, db
    dz, db = L.gemm_linear_grad(z, z=z, act="relu", bias_grad=True, workspace=buffer(1, ROWS, WIDE, 0))
    no_device_error()
    assert torch.equal(dz[at], torch.where(z[at] > 0, z[at], torch.zeros_like(z[at])))
    sums = torch.zeros(WIDE, dtype=torch.float64)
    for lo in range(0, ROWS, 1 << 16):
        sums += torch.relu(z[lo:lo + (1 << 16)].double()).sum(0).cpu()
    # (pieces of some 15000 rows by eight threads each: at most 1900 additions one after another)
    near(db.cpu(), sums, 1900 * 2.0 ** -24 * sums, "dbias of grad")
    assert G.gemm_f16_take_device_error()[0] == G.GEMM_OK
