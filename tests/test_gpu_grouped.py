"""Grouped products by expert and their gradients against a 64-bit host implementation.

Operands of integers over 8 make every product a multiple of 2^-6 and every sum here exact in fp32 in any
order, so a 16-bit result must be the exact sum rounded once, bit for bit, and an fp32 result the sum itself."""
import numpy as np
import pytest

from ragged_helpers import (HALF_STEP, KINDS, G, R, eighths, grouped_operands, grouped_ref, grouped_run, no_device_error,
                            offsets_of, require_gpu, torch)

pytestmark = pytest.mark.gpu

OPS = ["nt", "nn", "tn"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def check_exact(op, sizes, n, k, kind, seed, extra=0, head=0, dtype=None, workspace=True):
    rng = np.random.default_rng(seed)
    first, second = grouped_operands(op, rng, sizes, n, k, kind, extra=extra + head)
    offsets = offsets_of(sizes, head)
    ref = grouped_ref(op, first, second, offsets, len(sizes))
    got = grouped_run(op, first, second, offsets, dtype=dtype, workspace=workspace)
    want = ref.to(got.dtype)
    bad = torch.nonzero(got != want)
    assert bad.shape[0] == 0, "%d differ, first at %s: %s, want %s" % (
        bad.shape[0], bad[0].tolist(), got[tuple(bad[0])], want[tuple(bad[0])])


# few rows per group (single CTAs), many (CTA pairs), and both kinds of ragged: lengths around 16, 32, 64 and 256
SIZES = {
    "one row": [0, 1, 0],
    "few": [1, 0, 15, 16, 17, 31, 3, 0],
    "around 64": [63, 64, 65, 1],
    "wide": [255, 256, 257, 0, 90],
    "uneven": [700, 1, 33, 0, 128],
    "one group": [300],
}
SHAPES = [(8, 8), (64, 64), (136, 200), (264, 520), (1000, 72)]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("sizes", sorted(SIZES))
def test_exact(op, kind, n, k, sizes):
    check_exact(op, SIZES[sizes], n, k, KINDS[kind], seed=n * 1000 + k)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("sizes", ["few", "wide"])
def test_without_workspace(op, sizes):
    check_exact(op, SIZES[sizes], 264, 328, torch.float16, seed=5, workspace=False)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("sizes", sorted(SIZES))
def test_weight_gradient_in_fp32(kind, sizes):
    check_exact("tn", SIZES[sizes], 200, 136, KINDS[kind], seed=9, dtype=torch.float32)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("head,extra", [(0, 70), (5, 0), (13, 200)])
def test_rows_of_no_group(op, head, extra):
    """Rows before the first offset and after the last are zero in y and dx and take no part in dw."""
    check_exact(op, [20, 0, 41, 300], 136, 264, torch.float16, seed=11, extra=extra, head=head)
    check_exact(op, [1, 2, 0, 3], 136, 264, torch.bfloat16, seed=12, extra=extra, head=head)


@pytest.mark.parametrize("op", OPS)
def test_no_rows_at_all(op):
    check_exact(op, [0, 0, 0], 64, 72, torch.float16, seed=1, extra=50)
    first, second = grouped_operands(op, np.random.default_rng(0), [0, 0], 64, 72, torch.float16)
    got = grouped_run(op, first, second, offsets_of([0, 0]))
    assert got.numel() == (0 if op != "tn" else 2 * 64 * 72) and not got.any()


@pytest.mark.parametrize("op", OPS)
def test_many_groups(op):
    rng = np.random.default_rng(3)
    sizes = rng.integers(0, 4, size=1024).tolist()
    check_exact(op, sizes, 24, 40, torch.float16, seed=3)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("n,k", [(520, 600), (264, 1032), (448, 128), (1000, 72)])
def test_weight_gradient_of_many_ragged_groups(kind, n, k):
    """More tiles than the workers take in two turns: every group's rows end in tensor maps of its own."""
    rng = np.random.default_rng(n + k)
    sizes = rng.integers(0, 150, size=90).tolist()
    check_exact("tn", sizes, n, k, KINDS[kind], seed=n, extra=30)
    check_exact("tn", sizes, n, k, KINDS[kind], seed=k, head=3, dtype=torch.float32)


def test_own_maps_keep_other_groups_infinities_out():
    rng = np.random.default_rng(14)
    sizes = rng.integers(1, 70, size=100).tolist()
    dy, x = grouped_operands("tn", rng, sizes, 264, 520, torch.bfloat16)
    offsets = offsets_of(sizes)
    ref = grouped_ref("tn", dy, x, offsets, 100)
    ends = offsets.numpy()
    for g in range(1, 100, 2):  # every second group holds infinities and NaN
        dy[ends[g]:ends[g + 1]] = float("inf")
        x[ends[g]:ends[g + 1], ::2] = float("nan")
    got = grouped_run("tn", dy, x, offsets)
    assert torch.equal(got[::2], ref[::2].bfloat16())


@pytest.mark.parametrize("op", OPS)
def test_split_over_k_and_workers(op):
    """Few tiles with a long contraction: with a workspace a tile's K blocks lie on many workers."""
    check_exact(op, [3, 0, 2], 136 if op != "nn" else 4104, 4104 if op != "nn" else 136, torch.float16, seed=21)
    check_exact(op, [1], 264 if op != "nn" else 8200, 8200 if op != "nn" else 264, torch.bfloat16, seed=22)


@pytest.mark.parametrize("op", OPS)
def test_offsets_that_are_not_monotone_reach_no_other_memory(op):
    """They are clamped to [0, rows] and made monotone; the guard bands around the output stay."""
    rng = np.random.default_rng(8)
    n, k, rows = 64, 136, 100
    first, second = grouped_operands(op, rng, [25, 25, 25, 25], n, k, torch.float16)
    offsets = torch.tensor([-7, 40, 30, 2 ** 31 - 1, 90], dtype=torch.int32)
    ref = grouped_ref(op, first, second, offsets, 4)
    numel = ref.numel()
    band = 4096
    buf = torch.full((numel + 2 * band,), 7.0, dtype=torch.float16, device="cuda")
    out = buf[band:band + numel].view(ref.shape)
    got = grouped_run(op, first, second, offsets, out=out)
    assert torch.equal(got, ref.to(torch.float16))
    assert (buf[:band] == 7).all() and (buf[band + numel:] == 7).all()


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("sizes", [[30, 45, 2], [300, 270, 2], [1, 1, 1], [257, 0, 31]])
def test_other_groups_contents_never_reach_a_result(op, sizes):
    """Rows (and, forward, weights) of the other groups hold infinities and NaN."""
    rng = np.random.default_rng(4)
    n, k = 136, 200
    first, second = grouped_operands(op, rng, sizes, n, k, torch.float16)
    offsets = offsets_of(sizes)
    ref = grouped_ref(op, first, second, offsets, 3)
    lo, hi = int(offsets[0]), int(offsets[1])
    bad = torch.tensor([float("inf"), float("nan"), -float("inf")], dtype=torch.float16)
    first2, second2 = first.clone(), second.clone()
    first2[hi:] = bad[torch.arange(first2[hi:].numel()) % 3].view(first2[hi:].shape)
    if op == "tn":
        second2[hi:] = bad[torch.arange(second2[hi:].numel()) % 3].view(second2[hi:].shape)
    else:
        second2[1:] = bad[torch.arange(second2[1:].numel()) % 3].view(second2[1:].shape)
    got = grouped_run(op, first2, second2, offsets)
    if op == "tn":
        assert torch.equal(got[0], ref[0].to(torch.float16))
    else:
        assert torch.equal(got[lo:hi], ref[lo:hi].to(torch.float16))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("sizes", [[40, 0, 3, 21], [500, 130, 0, 260]])
def test_real_values(op, kind, sizes):
    """|error| <= half a step of the result plus the fp32 sums' error, at most (terms + 1) 2^-23 sum |a b|."""
    kind = KINDS[kind]
    rng = np.random.default_rng(17)

    def normal(rng, shape, kind):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(kind)

    n, k = 392, 520
    first, second = grouped_operands(op, rng, sizes, n, k, kind, draw=normal)
    offsets = offsets_of(sizes)
    ref = grouped_ref(op, first, second, offsets, 4)
    size = grouped_ref(op, first.abs(), second.abs(), offsets, 4)
    terms = {"nt": k, "nn": n, "tn": max(sizes)}[op]
    got = grouped_run(op, first, second, offsets).double()
    bound = HALF_STEP[kind] * 2 * ref.abs() + (terms + 1) * 2.0 ** -23 * size
    assert ((got - ref).abs() <= bound).all()


@pytest.mark.parametrize("op", OPS)
def test_repeats_bit_for_bit(op):
    rng = np.random.default_rng(5)
    sizes = [7, 0, 20, 3]
    first = torch.from_numpy(rng.standard_normal((30, 2056 if op != "tn" else 200)).astype(np.float32)).half()
    if op == "tn":
        second = torch.from_numpy(rng.standard_normal((30, 264)).astype(np.float32)).half()
    else:
        shape = (4, 200, 2056) if op == "nt" else (4, 2056, 200)
        second = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).half()
    runs = [grouped_run(op, first, second, offsets_of(sizes)) for _ in range(3)]
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


def test_data_gradient_against_differences():
    """sum(y c) changes by dx . v along v: exact here, since every value is a multiple of 2^-6."""
    rng = np.random.default_rng(6)
    sizes, n, k = [5, 0, 70], 64, 72
    x, w = grouped_operands("nt", rng, sizes, n, k, torch.float16)
    c, v = eighths(rng, (75, n), torch.float16), eighths(rng, (75, k), torch.float16)
    offsets = offsets_of(sizes)
    dx = grouped_ref("nn", c, w, offsets, 3)
    loss = [float((grouped_ref("nt", t, w, offsets, 3) * c.double()).sum()) for t in (x.double() + v.double(), x.double() - v.double())]
    assert abs((loss[0] - loss[1]) / 2 - float((dx * v.double()).sum())) <= 1e-9 * abs(loss[0]) + 1e-9
    assert torch.equal(grouped_run("nn", c, w, offsets), dx.half())
    dw = grouped_ref("tn", c, x, offsets, 3)
    u = eighths(rng, (3, n, k), torch.float16).double()
    loss = [float((grouped_ref("nt", x, t, offsets, 3) * c.double()).sum()) for t in (w.double() + u, w.double() - u)]
    assert abs((loss[0] - loss[1]) / 2 - float((dw * u).sum())) <= 1e-9 * abs(loss[0]) + 1e-9
    assert torch.equal(grouped_run("tn", c, x, offsets), dw.half())


def test_other_stream_and_graph():
    """A call on a stream of its own, and captured: replays follow new offsets and rows in the same buffers."""
    rng = np.random.default_rng(7)
    n, k, rows = 136, 1032, 40
    w = eighths(rng, (4, n, k), torch.float16)
    wd = w.cuda()
    xd = torch.zeros((rows, k), dtype=torch.float16, device="cuda")
    od = torch.zeros(5, dtype=torch.int32, device="cuda")
    y = torch.full((rows, n), float("nan"), dtype=torch.float16, device="cuda")
    ws = torch.zeros(R.gemm_grouped_workspace_size(4, rows, n, k), dtype=torch.uint8, device="cuda")
    R.gemm_grouped_nt(xd, wd, od, y=y, workspace=ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        R.gemm_grouped_nt(xd, wd, od, y=y, workspace=ws)
    for sizes in ([10, 10, 10, 10], [1, 0, 0, 0], [0, 40, 0, 0], [3, 9, 27, 1]):
        x = eighths(rng, (rows, k), torch.float16)
        offsets = offsets_of(sizes)
        xd.copy_(x)
        od.copy_(offsets)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), grouped_ref("nt", x, w, offsets, 4).half())
        with torch.cuda.stream(side):
            got = grouped_run("nt", x, w, offsets, stream=side)
        assert torch.equal(got, grouped_ref("nt", x, w, offsets, 4).half())
    no_device_error()


@pytest.mark.parametrize("mode,sizes", [(0, [3, 4]), (0, [300, 290]), (1, [3, 4]), (1, [300, 290]), (2, [300, 290])])
@pytest.mark.parametrize("skip", [0, 3])
def test_starved_wait_reports_timeout_and_recovers(mode, sizes, skip):
    """A ring fill that never comes: the waits run out, the kernel records it and returns, and the next call is right."""
    op = OPS[mode]
    rng = np.random.default_rng(2)
    first, second = grouped_operands(op, rng, sizes, 2056, 1544, torch.float16)  # CTA 0 has more than three fills
    offsets = offsets_of(sizes)
    ref = grouped_ref(op, first, second, offsets, 2).half()
    f, s, o = first.cuda(), second.cuda(), offsets.cuda()
    out = torch.zeros(ref.shape, dtype=torch.float16, device="cuda")
    ws = torch.zeros(R.gemm_grouped_workspace_size(2, sum(sizes), 2056, 1544), dtype=torch.uint8, device="cuda")
    no_device_error()
    st = R.gemm_grouped_stall_test(mode, f, s, o, out, ws, skip, 1 << 24)
    assert st == G.GEMM_OK
    st, code = G.gemm_f16_take_device_error()
    assert st == G.GEMM_ERR_TIMEOUT and (code & 0xFF) in range(1, 12)
    assert torch.equal(grouped_run(op, first, second, offsets), ref)


# Sizes at which single CTAs' tiles, and CTA pairs', are split over K.
SPLIT = {"single CTAs": ([3, 4], 264, 8200), "pairs": ([700], 2000, 8192), "pairs, two groups": ([290, 300], 1032, 8200)}


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("name", sorted(SPLIT))
@pytest.mark.parametrize("workspace", [True, False])
def test_split_tiles(op, name, workspace):
    sizes, other, long = SPLIT[name]
    check_exact(op, sizes, other if op == "nt" else long, long if op == "nt" else other, torch.bfloat16, seed=31, workspace=workspace)


def test_split_tiles_in_a_graph():
    """A partial sum's flag is spent by the launch that adds it: every replay, all of one number, waits for its own."""
    rng = np.random.default_rng(8)
    n, k, rows = 264, 8200, 7
    w = eighths(rng, (2, n, k), torch.float16)
    wd, od = w.cuda(), offsets_of([3, 4]).cuda()
    xd = torch.zeros((rows, k), dtype=torch.float16, device="cuda")
    ws = torch.full((R.gemm_grouped_workspace_size(2, rows, n, k),), 0x5A, dtype=torch.uint8, device="cuda")
    y = R.gemm_grouped_nt(xd, wd, od, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.gemm_grouped_nt(xd, wd, od, y=y, workspace=ws)
    for _ in range(4):
        x = eighths(rng, (rows, k), torch.float16)
        xd.copy_(x)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), grouped_ref("nt", x, w, offsets_of([3, 4]), 2).half())
    no_device_error()


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("name", ["single CTAs", "pairs"])
def test_starved_split_reports_timeout_and_recovers(mode, name):
    """The worker whose fill never comes publishes no partial sum: the one that waits for it gives up as well."""
    op = OPS[mode]
    rng = np.random.default_rng(3)
    sizes, other, long = SPLIT[name]
    n, k = (other, long) if op == "nt" else (long, other)
    first, second = grouped_operands(op, rng, sizes, n, k, torch.float16)
    offsets = offsets_of(sizes)
    ref = grouped_ref(op, first, second, offsets, len(sizes)).half()
    f, s, o = first.cuda(), second.cuda(), offsets.cuda()
    out = torch.zeros(ref.shape, dtype=torch.float16, device="cuda")
    ws = torch.zeros(R.gemm_grouped_workspace_size(len(sizes), sum(sizes), n, k), dtype=torch.uint8, device="cuda")
    no_device_error()
    assert R.gemm_grouped_stall_test(mode, f, s, o, out, ws, 0, 1 << 24) == G.GEMM_OK
    st, code = G.gemm_f16_take_device_error()
    assert st == G.GEMM_ERR_TIMEOUT and (code & 0xFF) in range(1, 12)
    call = R.gemm_grouped_nt if op == "nt" else R.gemm_grouped_nn
    assert torch.equal(call(f, s, o, workspace=ws).cpu(), ref)  # the same workspace, flags of the aborted launch in it
    no_device_error()


# Few tiles with many rows: the weight gradient's groups are cut into parts.
PARTS = {"one group": [6000], "uneven": [3000, 0, 700, 65, 1], "ends in a part": [1024, 255, 2049], "empty ends": [0, 4000, 0]}


@pytest.mark.parametrize("sizes", sorted(PARTS))
@pytest.mark.parametrize("n,k", [(8, 8), (200, 136), (264, 520)])
@pytest.mark.parametrize("dtype", [None, torch.float32])
@pytest.mark.parametrize("workspace", [True, False])
def test_weight_gradient_in_parts(sizes, n, k, dtype, workspace):
    check_exact("tn", PARTS[sizes], n, k, torch.bfloat16, seed=41, dtype=dtype, workspace=workspace)
    check_exact("tn", PARTS[sizes], n, k, torch.float16, seed=42, extra=90, head=7, dtype=dtype, workspace=workspace)


def test_parts_keep_other_groups_infinities_out():
    rng = np.random.default_rng(44)
    sizes = [1500, 1301, 700]
    dy, x = grouped_operands("tn", rng, sizes, 200, 136, torch.float16)
    offsets = offsets_of(sizes)
    ref = grouped_ref("tn", dy, x, offsets, 3)
    dy[1500:2801] = float("inf")
    x[1500:2801] = float("nan")
    got = grouped_run("tn", dy, x, offsets)
    assert torch.equal(got[::2], ref[::2].half()) and bool(torch.isnan(got[1]).all())


def test_parts_repeat_bit_for_bit_in_a_graph():
    rng = np.random.default_rng(45)
    dy = torch.from_numpy(rng.standard_normal((5000, 200)).astype(np.float32)).half().cuda()
    x = torch.from_numpy(rng.standard_normal((5000, 264)).astype(np.float32)).half().cuda()
    offsets = offsets_of([1800, 3200]).cuda()
    ws = torch.full((R.gemm_grouped_workspace_size(2, 5000, 200, 264),), 0xFF, dtype=torch.uint8, device="cuda")
    first = R.gemm_grouped_tn(dy, x, offsets, workspace=ws)
    out = torch.empty_like(first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            R.gemm_grouped_tn(dy, x, offsets, dw=out, workspace=ws)
    ws.fill_(0xFF)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    no_device_error()


def test_weight_gradients_of_groups_without_rows_are_zero():
    sizes = [0] * 30 + [1] + [0] * 40
    check_exact("tn", sizes, 264, 136, torch.float16, seed=47)
    check_exact("tn", sizes, 264, 136, torch.float16, seed=47, workspace=False)
