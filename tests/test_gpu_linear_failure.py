"""Waits that run out in the products with an epilogue: reported, not hung, and calls and replays after them are right."""
import numpy as np
import pytest

from linear_helpers import G, L, buffer, draw, eighths, grad_ref, near, no_device_error, nt_ref, require_gpu, rounded, torch

pytestmark = pytest.mark.gpu

# single CTAs whole and split, pairs whole, split, and split in their last wave; rows, n, k of nt (nn: n and k changed places)
SIZES = {"single CTAs": (5, 264, 136), "single CTAs, split": (7, 264, 8200), "pairs": (300, 264, 520), "pairs, split": (700, 2000, 8192),
         "pairs, last wave split": (2500, 2304, 8192)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("name", sorted(SIZES))
@pytest.mark.parametrize("skip", [0, 3])
def test_replays_after_an_aborted_one(mode, name, skip):
    """The hook leaves a fill undone while the error word is clear: of the replays, the first is aborted and those before the
    error is taken run through."""
    rows, other, long = SIZES[name]
    n, k = (long, other) if mode else (other, long)
    if -(-long // 64) <= skip:
        pytest.skip("no such fill")
    rng = np.random.default_rng(skip)
    _, w, _, _, _ = draw(rng, [rows], n, k, torch.float16, False, False, False)
    width = k if mode else n
    first = torch.empty((rows, n if mode else k), dtype=torch.float16, device="cuda")
    wd, extra = w.cuda(), eighths(rng, (rows, width), torch.float16)
    ed, out, db = extra.cuda(), torch.zeros((rows, width), dtype=torch.float16, device="cuda"), torch.zeros(k, device="cuda")
    ws = buffer(1, rows, n, k)

    def check(x):
        if mode:
            want, off, wb, wb_off = grad_ref(x.double() @ w.double(), extra, "silu", None)
            near(db.cpu(), wb, wb_off + wb.abs() * 2.0 ** -24, "dbias")
        else:
            want, off, _ = nt_ref(x, w, None, extra, "silu", None)
        near(out.cpu(), want, rounded(torch.float16, want, off), "out")

    def call():
        if mode:
            L.gemm_linear_nn(first, wd, z=ed, act="silu", bias_grad=True, dx=out, dbias=db, workspace=ws)
        else:
            L.gemm_linear_nt(first, wd, residual=ed, act="silu", y=out, workspace=ws)

    x = eighths(rng, tuple(first.shape), torch.float16)
    first.copy_(x)
    call()
    no_device_error()
    check(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert L.gemm_linear_stall_test(mode, first, wd, ed, out, db if mode else None, ws, skip, 1 << 24, act="silu") == G.GEMM_OK
    for _ in range(2):
        graph.replay()  # aborted
        torch.cuda.synchronize()
        for _ in range(2):
            x = eighths(rng, tuple(first.shape), torch.float16)
            first.copy_(x)
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            check(x)
        st, code = G.gemm_f16_take_device_error()
        assert st == G.GEMM_ERR_TIMEOUT and (code & 0xFF) in range(1, 12)
    call()
    no_device_error()
    check(x)


def test_calls_on_streams_of_their_own():
    """Split products that overlap on the GPU wait only for workers before them."""
    rng = np.random.default_rng(4)
    rows, n, k = 2500, 2304, 8192
    x, w, b, r, _ = draw(rng, [rows], n, k, torch.float16, False)
    xd, wd, bd, rd = (t.cuda() for t in (x, w, b, r))
    want = L.gemm_linear_nt(xd, wd, bias=bd, residual=rd, act="gelu", workspace=buffer(1, rows, n, k))
    few = L.gemm_linear_nt(xd[:7], wd, bias=bd, residual=rd[:7], act="gelu", workspace=buffer(1, 7, n, k))
    streams = [torch.cuda.Stream() for _ in range(4)]
    spaces = [buffer(1, rows, n, k) for _ in streams]
    outs = [torch.empty_like(want if i < 2 else few) for i in range(4)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (s, o, ws) in enumerate(zip(streams, outs, spaces)):
            rows_i = rows if i < 2 else 7
            L.gemm_linear_nt(xd[:rows_i], wd, bias=bd, residual=rd[:rows_i], act="gelu", y=o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    no_device_error()
    assert all(torch.equal(o, want if i < 2 else few) for i, o in enumerate(outs))


def test_column_sums_on_streams_of_their_own():
    """Split products with column sums in chains, in place and not, that overlap on the GPU."""
    torch.manual_seed(5)
    rows, n, k = 2500, 4096, 2304
    dyd = torch.randn(rows, n, device="cuda").bfloat16()
    wd = (torch.randn(n, k, device="cuda") / 64).bfloat16()
    z = torch.randn(rows, k, device="cuda").bfloat16()
    want = [L.gemm_linear_nn(dyd[:r], wd, z=z[:r], act="gelu", bias_grad=True, workspace=buffer(1, rows, n, k)) for r in (rows, 40)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    spaces = [buffer(1, rows, n, k) for _ in streams]
    # (every second call writes dx over its z)
    zs = [[z[:rows if i < 2 else 40].clone() for _ in range(10)] for i in range(4)]
    dbs = [[torch.empty(k, device="cuda") for _ in range(10)] for _ in range(4)]
    outs = [[zs[i][j] if j % 2 else torch.empty_like(zs[i][j]) for j in range(10)] for i in range(4)]
    torch.cuda.synchronize()
    for j in range(10):
        for i, s in enumerate(streams):
            r = rows if i < 2 else 40
            L.gemm_linear_nn(dyd[:r], wd, z=zs[i][j], act="gelu", bias_grad=True, dx=outs[i][j], dbias=dbs[i][j], workspace=spaces[i], stream=s)
    torch.cuda.synchronize()
    no_device_error()
    for i in range(4):
        dx, db = want[0 if i < 2 else 1]
        assert all(torch.equal(o, dx) for o in outs[i]) and all(torch.equal(d, db) for d in dbs[i])
