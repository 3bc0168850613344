"""Products with an epilogue and their gradients against 64-bit host implementations.

Operands are integers over 8, so that the products' sums are exact in fp32 in any order: z, and y without an activation, must be
the exact sum rounded once; what goes through an activation is within the bounds of linear_helpers."""
import numpy as np
import pytest

from linear_helpers import (ACTS, KINDS, G, L, buffer, cuda, draw, eighths, grad_ref, near, no_device_error, nt_ref, offsets_of,
                            require_gpu, rounded, torch, value)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def run_nt(x, w, b, r, act, offsets, keep=True, workspace=True, stream=None):
    groups = 1 if offsets is None else len(offsets) - 1
    ws = buffer(groups, x.shape[0], w.shape[-2], w.shape[-1]) if workspace else None
    out = L.gemm_linear_nt(cuda(x), cuda(w), bias=cuda(b), residual=cuda(r), act=act, offsets=cuda(offsets), keep=keep, workspace=ws,
                           stream=stream)
    no_device_error(stream)
    return out


def check_nt(sizes, n, k, kind, act, grouped, seed, bias=True, residual=True, workspace=True, extra=0, head=0):
    rng = np.random.default_rng(seed)
    x, w, b, r, offsets = draw(rng, sizes, n, k, kind, grouped, bias, residual, extra=extra + head)
    if grouped and head:
        offsets = offsets_of(sizes, head)
    y, z = run_nt(x, w, b, r, act, offsets, workspace=workspace)
    want, off, zz = nt_ref(x, w, b, r, act, offsets)
    assert torch.equal(z.cpu(), zz.to(kind))
    if act == "none":
        assert torch.equal(y.cpu(), want.to(kind))
    near(y.cpu(), want, rounded(kind, want, off), "y")


def check_nn(sizes, n, k, kind, act, grouped, seed, bias=True, workspace=True, extra=0, head=0, inplace=False):
    rng = np.random.default_rng(seed)
    rows, groups = int(sum(sizes)) + extra + head, len(sizes)
    _, w, _, _, _ = draw(rng, sizes, n, k, kind, grouped, False, False)
    dy, z = eighths(rng, (rows, n), kind), torch.from_numpy(rng.normal(0, 2, (rows, k))).to(kind)
    offsets = offsets_of(sizes, head) if grouped else None
    stack = groups if grouped else 1
    d = torch.zeros((rows, k), dtype=torch.float64)
    if grouped:
        for g in range(groups):
            lo, hi = int(offsets[g]), int(offsets[g + 1])
            d[lo:hi] = dy[lo:hi].double() @ w[g].double()
    else:
        d = dy.double() @ w.double()
    ws = buffer(stack, rows, n, k) if workspace else None
    zc = cuda(z)
    out = L.gemm_linear_nn(cuda(dy), cuda(w), z=None if act == "none" else zc, act=act, offsets=cuda(offsets), bias_grad=bias,
                           dx=zc if inplace else None, workspace=ws)
    no_device_error()
    dx, db = out if bias else (out, None)
    want, off, wb, wb_off = grad_ref(d, z, act, offsets)
    if act == "none":
        assert torch.equal(dx.cpu(), want.to(kind))
    near(dx.cpu(), want, rounded(kind, want, off), "dx")
    if bias:
        near(db.cpu(), wb, wb_off + wb.abs() * 2.0 ** -24, "dbias")


def check_grad(sizes, n, kind, act, grouped, seed, bias=True, extra=0, head=0, scale=2.0):
    rng = np.random.default_rng(seed)
    rows, groups = int(sum(sizes)) + extra + head, len(sizes)
    dy = torch.from_numpy(rng.normal(0, 1, (rows, n))).to(kind)
    z = torch.from_numpy(rng.normal(0, scale, (rows, n))).to(kind)
    offsets = offsets_of(sizes, head) if grouped else None
    ws = buffer(groups if grouped else 1, rows, n, 0)
    out = L.gemm_linear_grad(cuda(dy), z=cuda(z), act=act, offsets=cuda(offsets), bias_grad=bias, dz=torch.empty_like(dy, device="cuda"),
                             workspace=ws)
    no_device_error()
    dz, db = out if bias else (out, None)
    want, off, wb, wb_off = grad_ref(dy.double(), z, act, offsets)
    near(dz.cpu(), want, rounded(kind, want, off), "dz")
    if bias:
        near(db.cpu(), wb, wb_off + wb.abs() * 2.0 ** -24, "dbias")


# rows that single CTAs take (whole and split), that CTA pairs take, around every step of the instruction and tile
ROWS = [1, 2, 15, 33, 63, 64, 65, 130, 255, 256, 257, 700]
SHAPES = [(8, 8), (64, 72), (136, 200), (264, 520), (1000, 72), (520, 2056)]
SIZES = {"few": [1, 0, 15, 16, 17, 31, 3, 0], "around 64": [63, 64, 65, 1], "wide": [255, 256, 257, 0, 90], "uneven": [700, 1, 33, 0, 128],
         "one group": [300]}


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind", sorted(KINDS))
def test_nt_activations(kind, act):
    check_nt([70], 136, 200, KINDS[kind], act, False, seed=1)
    check_nt([1], 520, 2056, KINDS[kind], act, False, seed=2)
    check_nt([700], 264, 520, KINDS[kind], act, False, seed=3)
    check_nt([300, 0, 290], 264, 520, KINDS[kind], act, True, seed=4)


@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("rows", ROWS)
def test_nt_sizes(rows, n, k):
    check_nt([rows], n, k, torch.float16, "silu", False, seed=rows + n)
    check_nt([rows], n, k, torch.bfloat16, "none", False, seed=rows + k)


@pytest.mark.parametrize("bias,residual", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("rows", [3, 300])
def test_nt_without(rows, bias, residual):
    for act in ("none", "gelu"):
        check_nt([rows], 264, 328, torch.bfloat16, act, False, seed=rows, bias=bias, residual=residual)
        check_nt([rows, 2], 264, 328, torch.float16, act, True, seed=rows, bias=bias, residual=residual)
    check_nt([rows], 264, 328, torch.float16, "relu", False, seed=rows, workspace=False)


@pytest.mark.parametrize("sizes", sorted(SIZES))
@pytest.mark.parametrize("n,k", [(64, 72), (264, 520)])
def test_nt_groups(sizes, n, k):
    check_nt(SIZES[sizes], n, k, torch.float16, "gelu_tanh", True, seed=n)
    check_nt(SIZES[sizes], n, k, torch.bfloat16, "relu2", True, seed=k, extra=70, head=9)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind", sorted(KINDS))
def test_nn_activations(kind, act):
    check_nn([70], 136, 200, KINDS[kind], act, False, seed=1)
    check_nn([1], 2056, 520, KINDS[kind], act, False, seed=2)
    check_nn([700], 264, 520, KINDS[kind], act, False, seed=3)
    check_nn([300, 0, 290], 264, 520, KINDS[kind], act, True, seed=4)


@pytest.mark.parametrize("n,k", [(8, 8), (72, 64), (200, 136), (520, 264), (72, 1000), (2056, 520)])
@pytest.mark.parametrize("rows", ROWS)
def test_nn_sizes(rows, n, k):
    check_nn([rows], n, k, torch.float16, "gelu", False, seed=rows + n)
    check_nn([rows], n, k, torch.bfloat16, "none", False, seed=rows + k)


@pytest.mark.parametrize("sizes", sorted(SIZES))
@pytest.mark.parametrize("n,k", [(72, 64), (520, 264)])
def test_nn_groups(sizes, n, k):
    check_nn(SIZES[sizes], n, k, torch.float16, "gelu", True, seed=n)
    check_nn(SIZES[sizes], n, k, torch.bfloat16, "silu", True, seed=k, extra=70, head=9)
    check_nn(SIZES[sizes], n, k, torch.bfloat16, "relu", True, seed=k, bias=False, workspace=False)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rows,n", [(1, 8), (7, 264), (33, 1000), (200, 64), (777, 2056)])
def test_grad(rows, n, kind, act):
    check_grad([rows], n, KINDS[kind], act, False, seed=rows)
    check_grad([rows], n, KINDS[kind], act, False, seed=rows, scale=9.0)


@pytest.mark.parametrize("sizes", sorted(SIZES))
@pytest.mark.parametrize("n", [8, 264, 1000])
def test_grad_groups(sizes, n):
    check_grad(SIZES[sizes], n, torch.float16, "gelu", True, seed=n)
    check_grad(SIZES[sizes], n, torch.bfloat16, "silu", True, seed=n, extra=70, head=9)


def test_grad_long():
    check_grad([20000], 520, torch.bfloat16, "gelu", False, seed=5)
    check_grad([9000, 0, 11000], 264, torch.float16, "gelu_tanh", True, seed=6)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_grad_of_every_value(kind):
    """f' of every finite 16-bit value, at d = 1."""
    every = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(KINDS[kind])
    every = every[torch.isfinite(every)]
    z = every[: every.numel() // 8 * 8].reshape(-1, 8).contiguous()
    big = z.double().abs() > 1e18  # (z^3 and z^2 leave the range of fp32; f' is 0 or 1 there)
    for act in ACTS[1:]:
        dz = L.gemm_linear_grad(torch.ones_like(z).cuda(), z=z.cuda(), act=act)
        no_device_error()
        want, off, _, _ = grad_ref(torch.ones_like(z).double(), torch.where(big, 0, z), act, None)
        want = torch.where(torch.isinf(want.to(KINDS[kind])), want.to(KINDS[kind]).double(), want)  # past the type's range
        near(torch.where(big, 0, dz.cpu()), torch.where(big, 0.0, want), rounded(KINDS[kind], want, off), act)
        if act not in ("relu2",):
            assert torch.equal(dz.cpu()[big].double(), (z[big] > 0).double()), act


def test_grad_without_activation_is_dy():
    dy = torch.randn(33, 72, device="cuda").half()
    ws = buffer(1, 33, 72, 0)
    dz, db = L.gemm_linear_grad(dy, bias_grad=True, workspace=ws)
    assert dz is dy
    near(db.cpu(), dy.double().cpu().sum(0), 33 * 2.0 ** -23 * dy.double().cpu().abs().sum(0), "dbias")


@pytest.mark.parametrize("rows", [5, 300])
def test_in_place(rows):
    check_nn([rows], 264, 328, torch.float16, "gelu", False, seed=rows, inplace=True)
    rng = np.random.default_rng(rows)
    x, w, b, r, _ = draw(rng, [rows], 264, 328, torch.bfloat16, False)
    y = r.cuda()
    out = L.gemm_linear_nt(x.cuda(), w.cuda(), bias=b.cuda(), residual=y, y=y, workspace=buffer(1, rows, 264, 328))
    assert out is y
    assert torch.equal(y.cpu(), nt_ref(x, w, b, r, "none", None)[0].to(torch.bfloat16))
    for to in ("dy", "z"):
        dy, z = torch.randn(rows, 264, device="cuda").half(), torch.randn(rows, 264, device="cuda").half()
        want = L.gemm_linear_grad(dy, z=z, act="silu")
        got = L.gemm_linear_grad(dy, z=z, act="silu", dz=dy if to == "dy" else z)
        assert torch.equal(got, want)
    no_device_error()


def test_gradients_against_differences():
    """The gradients of sum(y * dy) with respect to bias and x, by central differences of the 64-bit forward pass."""
    rng = np.random.default_rng(3)
    for act in ACTS[1:]:
        x, w, b, _, _ = draw(rng, [40], 64, 72, torch.float16, False, residual=False)
        dy = eighths(rng, (40, 64), torch.float16)
        ws = buffer(1, 40, 64, 72)
        _, z = L.gemm_linear_nt(x.cuda(), w.cuda(), bias=b.cuda(), act=act, keep=True, workspace=ws)
        dz, db = L.gemm_linear_grad(dy.cuda(), z=z, act=act, bias_grad=True, workspace=ws)
        dx = L.gemm_linear_nn(dz, w.cuda(), workspace=ws)
        no_device_error()
        zz = nt_ref(x, w, b, None, "none", None)[0]
        keep = zz.abs() > 1e-3  # relu is not differentiable at 0
        h = 1e-5

        def loss(z):
            return torch.where(keep, value(act, z) * dy.double(), 0.0)

        want = (loss(zz + h) - loss(zz - h)) / (2 * h)
        got = torch.where(keep, dz.cpu().double(), 0.0)
        # dz is off by its rounding, by z's (half a step of z times f'' of at most 2), and by the differences' h^2
        bound = torch.finfo(torch.float16).eps / 2 * (want.abs() + 2 * zz.abs() * dy.double().abs()) + 2e-4
        near(got, want, bound, act)
        near(dx.cpu(), dz.cpu().double() @ w.double(), rounded(torch.float16, dz.cpu().double() @ w.double(),
             2.0 ** -20 * (dz.cpu().double().abs() @ w.double().abs())), "dx")
        near(db.cpu(), want.sum(0) + torch.where(keep, 0.0, dz.cpu().double()).sum(0), bound.sum(0), "dbias")


def test_rows_of_other_groups_never_reach_a_result():
    """Infinities and NaN in rows of no group, and in the next group's rows, stay where they are."""
    rng = np.random.default_rng(7)
    for sizes in ([5, 0, 20], [300, 270]):
        x, w, b, r, offsets = draw(rng, sizes, 136, 200, torch.float16, True, extra=40)
        live = int(offsets[-1])
        x[live:], r[live:] = float("inf"), float("nan")
        x[sizes[0]:live] = float("nan")
        y, z = run_nt(x, w, b, r, "gelu", offsets)
        want, off, zz = nt_ref(x[: sizes[0]], w, b, r[: sizes[0]], "gelu", torch.tensor([0, sizes[0]]))
        near(y[: sizes[0]].cpu(), want, rounded(torch.float16, want, off), "y")
        assert torch.isnan(y[sizes[0]:live]).all() and not y[live:].any() and not z[live:].any()
        d = eighths(rng, (live + 40, 136), torch.float16)
        d[live:], zk = float("inf"), torch.full((live + 40, 200), float("nan"), dtype=torch.float16)
        zk[: sizes[0]] = 0.5
        d[sizes[0]:live] = float("nan")
        dx, db = L.gemm_linear_nn(d.cuda(), w.cuda(), z=zk.cuda(), act="gelu", offsets=offsets.cuda(), bias_grad=True,
                                  workspace=buffer(len(sizes), live + 40, 136, 200))
        assert torch.isfinite(dx[: sizes[0]]).all() and torch.isfinite(db[0]).all() and not dx[live:].any()
        assert torch.isnan(db[-1]).all()
        dz, db = L.gemm_linear_grad(d.cuda(), z=torch.ones_like(d).cuda(), act="gelu", offsets=offsets.cuda(), bias_grad=True,
                                    workspace=buffer(len(sizes), live + 40, 136, 0))
        assert torch.isfinite(dz[: sizes[0]]).all() and torch.isfinite(db[0]).all() and not dz[live:].any()
        no_device_error()


def test_bad_offsets_reach_no_other_memory():
    rng = np.random.default_rng(8)
    rows, n, k = 90, 136, 200
    x, w, b, r, _ = draw(rng, [30, 30, 30], n, k, torch.float16, True)
    bad = torch.tensor([-5, 40, 20, 1 << 30], dtype=torch.int32)
    y, _ = run_nt(x, w, b, r, "silu", bad)
    want, off, _ = nt_ref(x, w, b, r, "silu", bad)
    near(y.cpu(), want, rounded(torch.float16, want, off), "y")
    dy, z = eighths(rng, (rows, n), torch.float16), torch.zeros((rows, n), dtype=torch.float16)
    dz, db = L.gemm_linear_grad(dy.cuda(), z=z.cuda(), act="silu", offsets=bad.cuda(), bias_grad=True, workspace=buffer(3, rows, n, 0))
    want, off, wb, wb_off = grad_ref(dy.double(), z, "silu", bad)
    near(dz.cpu(), want, rounded(torch.float16, want, off), "dz")
    near(db.cpu(), wb, wb_off + wb.abs() * 2.0 ** -24, "dbias")
    no_device_error()


def test_no_rows_and_no_columns():
    x, w = torch.empty((0, 64), device="cuda").half(), torch.randn(72, 64, device="cuda").half()
    y, z = L.gemm_linear_nt(x, w, act="gelu", keep=True)
    assert y.shape == z.shape == (0, 72)
    db = torch.full((64,), 5.0, device="cuda")
    L.gemm_linear_nn(torch.empty((0, 72), device="cuda").half(), w, bias_grad=True, dbias=db)
    assert not db.any()
    db = torch.full((3, 72), 5.0, device="cuda")
    L.gemm_linear_grad(torch.empty((0, 72), device="cuda").half(), offsets=torch.zeros(4, dtype=torch.int32, device="cuda"), bias_grad=True,
                       dbias=db)
    assert not db.any()
    no_device_error()


def test_workspace_sizes_of_nothing():
    for rows in (0, 5):
        for n, k in ((0, 0), (0, 64), (64, 0)):
            assert L.gemm_linear_workspace_size(3, rows, n, k) >= 0
    assert L.gemm_linear_workspace_size(1, 0, 64, 64) == 0
    empty = torch.empty((5, 0), device="cuda").half()
    assert L.gemm_linear_nt(torch.randn(5, 64, device="cuda").half(), torch.empty((0, 64), device="cuda").half()).shape == (5, 0)
    dz, db = L.gemm_linear_grad(empty, z=empty, act="gelu", bias_grad=True)
    assert dz.shape == (5, 0) and db.shape == (0,)


def test_as_many_groups_as_there_may_be():
    rng = np.random.default_rng(21)
    sizes = rng.integers(0, 3, 1024)
    check_nt(sizes, 64, 72, torch.float16, "silu", True, seed=1, extra=5, head=3)
    check_nn(sizes, 72, 64, torch.bfloat16, "gelu", True, seed=2, extra=5, head=3)
    check_grad(sizes, 264, torch.float16, "gelu", True, seed=3, extra=5, head=3)
    with pytest.raises(G.GemmError):
        check_grad([1] * 1025, 8, torch.float16, "gelu", True, seed=4)


def test_an_empty_contraction_is_refused():
    x, w = torch.empty((4, 0), device="cuda").half(), torch.empty((72, 0), device="cuda").half()
    with pytest.raises(G.GemmError):
        L.gemm_linear_nt(x, w)


def test_bias_gradient_needs_its_workspace():
    dy, w = torch.randn(300, 72, device="cuda").half(), torch.randn(72, 64, device="cuda").half()
    with pytest.raises(G.GemmError):
        L.gemm_linear_nn(dy, w, bias_grad=True)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(G.GemmError):
        L.gemm_linear_nn(dy, w, bias_grad=True, workspace=small)
    with pytest.raises(G.GemmError):
        L.gemm_linear_grad(dy, bias_grad=True)


def test_a_workspace_serves_fewer_rows():
    n, k = 520, 2056
    for groups in (1, 6):
        most = 3000
        need = L.gemm_linear_workspace_size(groups, most, n, k)
        only = L.gemm_linear_workspace_size(groups, most, n, 0)
        for rows in (1, 5, 64, 65, 129, 256, 257, 600, 1111, 2999):
            assert L.gemm_linear_workspace_size(groups, rows, n, k) <= need
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            off = None if groups == 1 else torch.linspace(0, rows, groups + 1, device="cuda").int()
            dy, z = torch.randn(rows, n, device="cuda").half(), torch.randn(rows, k, device="cuda").half()
            w = torch.randn(*(() if groups == 1 else (groups,)), n, k, device="cuda").half()
            L.gemm_linear_nn(dy, w, z=z, act="relu", offsets=off, bias_grad=True, workspace=ws)
            L.gemm_linear_grad(dy, z=dy, act="relu", offsets=off, bias_grad=True,
                               workspace=torch.empty(only, dtype=torch.uint8, device="cuda"))
    no_device_error()


def test_repeats_bit_for_bit():
    rng = np.random.default_rng(9)
    dy, w, z = (torch.randn(*s, device="cuda").bfloat16() for s in ((700, 520), (520, 1032), (700, 1032)))
    first = None
    for _ in range(3):
        ws = torch.from_numpy(rng.integers(0, 256, L.gemm_linear_workspace_size(1, 700, 520, 1032), dtype=np.uint8)).cuda()
        dx, db = L.gemm_linear_nn(dy, w, z=z, act="gelu", bias_grad=True, workspace=ws)
        dz, db2 = L.gemm_linear_grad(dx, z=z, act="gelu", bias_grad=True, workspace=ws)
        got = [t.clone() for t in (dx, db, dz, db2)]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
        first = got
    no_device_error()


def test_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(10)
    x, w, b, r, offsets = draw(rng, [200, 0, 130], 264, 328, torch.float16, True)
    xd, wd, bd, rd, od = (t.cuda() for t in (x, w, b, r, offsets))
    ws = buffer(3, 330, 264, 328)
    y, z = torch.empty_like(rd), torch.empty_like(rd)
    dx, db = torch.empty_like(xd), torch.empty((3, 328), device="cuda")

    def step(stream=None):
        L.gemm_linear_nt(xd, wd, bias=bd, residual=rd, act="gelu", offsets=od, keep=True, y=y, z=z, workspace=ws, stream=stream)
        dz = L.gemm_linear_grad(rd, z=z, act="gelu", offsets=od, stream=stream)
        L.gemm_linear_nn(dz, wd, z=xd, act="silu", offsets=od, bias_grad=True, dx=dx, dbias=db, workspace=ws, stream=stream)
        return dz

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, z, dx, db)]
    s = torch.cuda.Stream()
    for t in (y, z, dx, db):
        t.fill_(0)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        keep = step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y, z, dx, db)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        keep = step()
    for seed in range(2):
        xd.copy_(eighths(np.random.default_rng(seed), tuple(x.shape), torch.float16))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, z, dx, db)]
        for t in (y, z, dx, db):
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, z, dx, db)))
    del keep
    no_device_error()


def test_guard_bands():
    """Nothing is written outside the outputs."""
    rows, n, k = 77, 136, 200

    def banded(shape, kind):
        t = torch.full((shape[0] * shape[1] + 512,), 7.0, dtype=kind, device="cuda")
        return t, t[256:256 + shape[0] * shape[1]].view(shape)

    x, w, z0 = torch.randn(rows, k, device="cuda").half(), torch.randn(n, k, device="cuda").half(), torch.randn(rows, k, device="cuda").half()
    ty, y = banded((rows, n), torch.float16)
    tz, z = banded((rows, n), torch.float16)
    td, dx = banded((rows, k), torch.float16)
    tb, db = banded((1, k), torch.float32)
    ws = buffer(1, rows, n, k)
    L.gemm_linear_nt(x, w, act="gelu", keep=True, y=y, z=z, workspace=ws)
    L.gemm_linear_nn(y, w, z=z0, act="gelu", bias_grad=True, dx=dx, dbias=db.view(k), workspace=ws)
    no_device_error()
    for t in (ty, tz, td, tb):
        assert (t[:256] == 7).all() and (t[-256:] == 7).all()


@pytest.mark.parametrize("rows", [40, 2048])
@pytest.mark.parametrize("kind", sorted(KINDS))
def test_bias_gradient_of_a_long_contraction(rows, kind):
    """dbias stays a sum in 32 bits however long the contraction is.  All terms are positive, so no error cancels.  The tensor cores
    cut each sum of 16 products off, by less than 2^-23 of what it is: over a chain of 13 x 64 products, 52 sums that grow evenly, at
    most 26.5 x 2^-23 = 3.2e-6 of the chain's value (1024 sums, uncut, could lose 6.1e-5), and no more over chains of 20 and 9.
    At most 29 chains and 4 partials of a split tile are added to nearest, and most of them to less than half of the sum, 1.4e-6, and
    the columns' sums over 2048 rows, by 16 in a piece in pairs, 4 pieces, 2 sets and 8 tiles, half as much again where every
    rounding is at its worst: 6e-6."""
    n, k = 16384, 256
    gen = torch.Generator(device="cuda").manual_seed(rows)
    dy = (torch.rand(rows, n, generator=gen, device="cuda") + 0.5).to(KINDS[kind])
    w = (torch.rand(n, k, generator=gen, device="cuda") / 64 + 1 / 128).to(KINDS[kind])
    dx, db = L.gemm_linear_nn(dy, w, bias_grad=True, workspace=buffer(1, rows, n, k))
    no_device_error()
    want = (dy.double().sum(0)[None, :] @ w.double())[0]
    assert ((db.double() - want).abs() / want).max().item() < 6e-6


def test_a_workspace_that_captured_graphs_share():
    """Two graphs in turn in one workspace: what one of them leaves there means nothing to the other, whose parts lie elsewhere."""
    rng = np.random.default_rng(12)
    sizes = [(2500, 2304, 2048), (7, 1000, 4096), (1, 2304, 8192)]
    ws = torch.zeros(max(L.gemm_linear_workspace_size(1, *s) for s in sizes), dtype=torch.uint8, device="cuda")
    jobs = []
    for rows, n, k in sizes:
        x, w, b, _, _ = draw(rng, [rows], n, k, torch.bfloat16, False)
        xd, wd, bd = x.cuda(), w.cuda(), b.cuda()
        y, dx, db = (torch.empty((rows, n), dtype=torch.bfloat16, device="cuda"), torch.empty_like(xd), torch.empty(k, device="cuda"))

        def step(xd=xd, wd=wd, bd=bd, y=y, dx=dx, db=db):
            L.gemm_linear_nt(xd, wd, bias=bd, act="gelu", y=y, workspace=ws)
            L.gemm_linear_nn(y, wd, z=xd, act="silu", bias_grad=True, dx=dx, dbias=db, workspace=ws)

        step()
        torch.cuda.synchronize()
        outs = (y, dx, db)
        want = [t.clone() for t in outs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        jobs.append((graph, outs, want, step))
    for i in (0, 1, 0, 2, 1, 2, 0, 0, 1, 1, 2):
        graph, outs, want, _ = jobs[i]
        for t in outs:
            t.fill_(0)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
        jobs[(i + 1) % 3][3]()  # and one that is not captured between them
    no_device_error()
