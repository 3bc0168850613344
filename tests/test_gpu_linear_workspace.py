"""The workspace that gemm_linear_workspace_size reports serves every call of its sizes, and of fewer rows.

Whether a size is enough is decided before anything is launched, and before the workspace's alignment is looked at: with an address
that is not aligned a call that has enough ends in GEMM_ERR_ALIGNMENT, and nothing runs."""
import ctypes

import numpy as np
import pytest

from linear_helpers import G, L, eighths, no_device_error, require_gpu, torch

pytestmark = pytest.mark.gpu

P = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    L.lib()


def statuses(groups, rows, n, k, size):
    """What nt, nn, nn with dbias and grad with dbias answer to so many bytes at an address that is not aligned."""
    lib, off, ws = L.lib(), P if groups > 1 else None, P + 128
    return {lib.gemm_linear_nt(0, 5, groups, rows, n, k, off, P, P, P, P, P, P, ws, size, None),
            lib.gemm_linear_nn(0, 5, groups, rows, n, k, off, P, P, P, P, None, ws, size, None),
            lib.gemm_linear_nn(0, 5, groups, rows, n, k, off, P, P, P, P, P, ws, size, None),
            lib.gemm_linear_grad(0, 5, groups, rows, n, off, P, P, P, P, ws, size, None)}


def reported(groups, rows, n, k):
    b = ctypes.c_size_t()
    assert L.lib().gemm_linear_workspace_size(groups, rows, n, k, ctypes.byref(b)) == G.GEMM_OK
    return b.value


WIDTHS = [8, 64, 136, 520, 1024, 2056, 2168, 4096, 4808, 6144, 8192, 10752, 13824, 16384, 19584, 22016, 24576, 28672, 29568, 36864, 40960, 43008,
          65536, 100000, 151936, 262144]
DEPTHS = [8, 64, 200, 768, 1024, 2048, 2304, 3840, 4096, 4056, 5120, 5376, 6144, 7168, 8192, 16384, 28672]


@pytest.mark.parametrize("groups", [1, 2, 3, 5, 8, 10, 16, 17, 32, 38, 64])
def test_few_rows(groups):
    for rows in [*range(1, 10), 12, 16, 18, 24, 31, 32, 33, 36, 48, 57, 63, 64, 65, 66, 80]:
        for n in WIDTHS:
            for k in DEPTHS:
                assert statuses(groups, rows, n, k, reported(groups, rows, n, k)) == {G.GEMM_ERR_ALIGNMENT}, (groups, rows, n, k)
                # (the data gradient's way through a wide layer)
                assert statuses(groups, rows, k, n, reported(groups, rows, k, n)) == {G.GEMM_ERR_ALIGNMENT}, (groups, rows, k, n)


def test_random_sizes_and_fewer_rows():
    rng = np.random.default_rng(1)
    for _ in range(20000):
        groups = int(np.exp(rng.uniform(0, np.log(1024))))
        rows = int(np.exp(rng.uniform(0, np.log(40000))))
        n, k = (8 * int(np.exp(rng.uniform(0, np.log(32768)))) for _ in range(2))
        size = reported(groups, rows, n, k)
        for r in {rows, min(rows, 64), int(rng.integers(1, rows + 1)), int(rng.integers(1, min(rows, 64) + 1))}:
            assert statuses(groups, r, n, k, size) == {G.GEMM_ERR_ALIGNMENT}, (groups, rows, r, n, k)


def test_too_little_is_refused():
    """The way of asking does tell: a byte is never enough where a bias gradient of many rows is asked for."""
    assert G.GEMM_ERR_WORKSPACE in statuses(1, 1000, 520, 520, 256)


@pytest.mark.parametrize("groups,rows,n,k", [(1, 64, 28672, 8192), (1, 1, 28672, 8192), (1, 8, 22016, 4096), (38, 18, 2168, 4096)])
def test_wide_layers_of_few_rows(groups, rows, n, k):
    """With exactly the reported bytes, forward and backward; the sums of integers over 8 are exact."""
    rng = np.random.default_rng(rows)
    stack = (groups,) if groups > 1 else ()
    # a row of groups in turn: groups of some rows and, where there are fewer rows than groups, empty ones
    offsets = None if groups == 1 else torch.linspace(0, rows, groups + 1).int()
    ends = [0, rows] if groups == 1 else offsets.tolist()
    piece = eighths(rng, (1 << 20,), torch.float16).cuda()
    count = max(groups, 1) * n * k
    w = piece.repeat(-(-count // (piece.numel() - 5)))[:count].view(*stack, n, k)
    x, r, dy, z = (eighths(rng, (rows, c), torch.float16).cuda() for c in (k, n, n, k))
    bias = eighths(rng, stack + (n,), torch.float16).cuda()
    size = L.gemm_linear_workspace_size(groups, rows, n, k)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    off = None if offsets is None else offsets.cuda()
    y, kept = L.gemm_linear_nt(x, w, bias=bias, residual=r, act="relu", offsets=off, keep=True, workspace=ws)
    dx, db = L.gemm_linear_nn(dy, w, z=z, act="relu", offsets=off, bias_grad=True, workspace=ws)
    only = L.gemm_linear_nn(dy, w, z=z, act="relu", offsets=off, workspace=ws)
    no_device_error()
    for g in range(groups):
        lo, hi = ends[g], ends[g + 1]
        if lo == hi:
            assert groups == 1 or not db[g].any()
            continue
        wg, bg = (w, bias) if groups == 1 else (w[g], bias[g])
        for at in range(0, n, 4096):
            cols = slice(at, min(at + 4096, n))
            want = x[lo:hi].double() @ wg[cols].double().T + bg[cols].double()
            assert torch.equal(kept[lo:hi, cols], want.half())
            # relu and the residual are exact in fp32
            assert torch.equal(y[lo:hi, cols], (want.clamp(min=0) + r[lo:hi, cols].double()).half())
        for at in range(0, k, 4096):
            cols = slice(at, min(at + 4096, k))
            want = (dy[lo:hi].double() @ wg[:, cols].double()) * (z[lo:hi, cols] > 0)
            assert torch.equal(dx[lo:hi, cols], want.half()) and torch.equal(only[lo:hi, cols], want.half())
            got = (db if groups == 1 else db[g])[cols].double()
            # a sum of hi - lo values of one tile, in fp32 in any order
            assert ((got - want.sum(0)).abs() <= (hi - lo) * 2.0 ** -24 * want.abs().sum(0)).all()
