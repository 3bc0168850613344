"""Low-rank adapters beside a shared projection against a 64-bit host implementation.

Integer operands keep the inner product x a^T exact in the operands' type (checked below), so the result must
be the exact sum rounded once, bit for bit."""
import numpy as np
import pytest

from ragged_helpers import (HALF_STEP, KINDS, R, lora_ref, lora_run, no_device_error, require_gpu, small_ints, torch)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def operands(rng, rows, n, k, rank, adapters, kind):
    """x and a sparse enough that |x a^T| <= 128 (exact in bf16, twice it under a scale of 2 as well)."""
    x = small_ints(rng, (rows, k), kind, 2)
    a = small_ints(rng, (adapters, rank, k), kind, 1)
    a[torch.from_numpy(rng.random((adapters, rank, k)) < max(0.0, 1 - 48.0 / k))] = 0
    b = small_ints(rng, (adapters, n, rank), kind, 2)
    w = small_ints(rng, (n, k), kind, 2)
    scale = torch.from_numpy(2.0 ** rng.integers(-1, 2, size=adapters)).float()
    u = torch.einsum("tk,lrk->tlr", x.double(), a.double())
    assert u.abs().max() <= 64
    return x, w, a, b, scale


def check(rows, n, k, rank, adapters, ids, kind, seed, scaled=True):
    rng = np.random.default_rng(seed)
    x, w, a, b, scale = operands(rng, rows, n, k, rank, adapters, kind)
    ids = torch.from_numpy(np.asarray(ids).astype(np.int32))
    scale = scale if scaled else None
    ref = lora_ref(x, w, a, b, ids, scale)
    got = lora_run(x, w, a, b, ids, scale)
    bad = torch.nonzero(got != ref.to(kind))
    assert bad.shape[0] == 0, "%d differ, first at %s: %s, want %s" % (
        bad.shape[0], bad[0].tolist(), got[tuple(bad[0])], ref[tuple(bad[0])])


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rows", [1, 2, 17, 63, 64, 65, 200, 256, 257, 600])
@pytest.mark.parametrize("n,k,rank", [(8, 8, 8), (136, 200, 16), (264, 520, 64), (1000, 72, 40), (200, 264, 128), (72, 136, 72)])
def test_rows_with_adapters_of_their_own(kind, rows, n, k, rank):
    """Every row draws an adapter, none among them, in any order."""
    rng = np.random.default_rng(rows)
    check(rows, n, k, rank, 9, rng.integers(-1, 9, size=rows), KINDS[kind], seed=rows + n)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("ends", [[100, 300, 301, 700], [256, 512], [1, 2, 3, 64], [40, 600]])
def test_requests_in_runs(kind, ends):
    ids = np.repeat([3, 0, -1, 2][: len(ends)], np.diff([0] + ends))
    check(ends[-1], 264, 328, 24, 4, ids, KINDS[kind], seed=len(ends))


@pytest.mark.parametrize("rows", [16, 32, 33])
@pytest.mark.parametrize("n,k,rank", [(1032, 2056, 8), (136, 1096, 24), (2200, 72, 32), (1032, 8, 40)])
def test_few_rows_where_the_adapters_kernels_change(rows, n, k, rank):
    rng = np.random.default_rng(rows * rank)
    check(rows, n, k, rank, 40, rng.integers(-2, 42, size=rows), torch.bfloat16, seed=rows + rank)


@pytest.mark.parametrize("rows,n,k,rank", [(64, 8200, 1096, 16), (30, 2056, 4104, 72), (2000, 4104, 648, 40)])
def test_many_tiles_with_long_contractions(rows, n, k, rank):
    """Several tiles for every worker, and K blocks that go round the ring more than twice before the adapters'."""
    check(rows, n, k, rank, 20, np.random.default_rng(2).integers(-1, 20, size=rows), torch.bfloat16, seed=13)
    check(rows, n, k, rank, 20, np.arange(rows) * 3 // rows, torch.float16, seed=14)


def test_more_rows_than_one_pass_takes():
    """The row tiles of one pass fit a table; 70000 rows take two passes."""
    check(70000, 64, 72, 8, 2, np.arange(70000) // 9000 % 3 - 1, torch.float16, seed=15)


@pytest.mark.parametrize("rows", [1, 64, 200])
def test_every_row_another_adapter(rows):
    check(rows, 136, 264, 16, rows, np.random.default_rng(1).permutation(rows), torch.float16, seed=3)


@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("ids", [-1, 4, 2 ** 31 - 1, -2 ** 31])
def test_no_row_has_an_adapter(rows, ids):
    check(rows, 136, 264, 16, 4, np.full(rows, ids), torch.bfloat16, seed=4)


@pytest.mark.parametrize("rows", [5, 300])
def test_no_scale(rows):
    check(rows, 136, 264, 16, 4, np.arange(rows) % 5 - 1, torch.float16, seed=5, scaled=False)


@pytest.mark.parametrize("adapters,rank", [(0, 16), (3, 0)])
@pytest.mark.parametrize("rows", [5, 300])
def test_no_adapters_or_no_rank(adapters, rank, rows):
    rng = np.random.default_rng(6)
    x, w = small_ints(rng, (rows, 264), torch.float16, 2), small_ints(rng, (136, 264), torch.float16, 2)
    a, b = torch.zeros((adapters, rank, 264)).half(), torch.zeros((adapters, 136, rank)).half()
    got = lora_run(x, w, a, b, torch.zeros(rows, dtype=torch.int32))
    assert torch.equal(got, (x.double() @ w.double().T).half())


def test_empty_sizes():
    half = torch.float16
    y = lora_run(torch.zeros((0, 64), dtype=half), torch.zeros((72, 64), dtype=half), torch.zeros((2, 8, 64), dtype=half),
                 torch.zeros((2, 72, 8), dtype=half), torch.zeros(0, dtype=torch.int32))
    assert y.shape == (0, 72)
    y = lora_run(torch.zeros((5, 0), dtype=half), torch.zeros((72, 0), dtype=half), torch.zeros((2, 8, 0), dtype=half),
                 torch.zeros((2, 72, 8), dtype=half), torch.zeros(5, dtype=torch.int32))
    assert y.shape == (5, 72) and not y.any()


@pytest.mark.parametrize("rows", [20, 300])
def test_other_adapters_contents_never_reach_a_row(rows):
    """Adapters that a row does not have hold infinities and NaN, and a row without one keeps the projection."""
    rng = np.random.default_rng(7)
    x, w, a, b, scale = operands(rng, rows, 136, 264, 24, 3, torch.float16)
    ids = torch.from_numpy((np.arange(rows) % 4 - 1).astype(np.int32))
    ref = lora_ref(x, w, a, b, ids, scale).half()
    a[2], b[2] = float("nan"), float("inf")
    got = lora_run(x, w, a, b, ids, scale)
    keep = ids != 2
    assert torch.equal(got[keep], ref[keep])


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rows,n", [(20, 136), (300, 136), (64, 2056), (600, 1000)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_one_bad_value_of_b_spoils_its_own_column_and_rows(kind, rows, n, bad):
    rng = np.random.default_rng(12)
    x, w, a, b, scale = operands(rng, rows, n, 264, 72, 3, KINDS[kind])
    ids = torch.from_numpy((np.arange(rows) % 4 - 1).astype(np.int32))
    ref = lora_ref(x, w, a, b, ids, scale).to(KINDS[kind])
    spots = [(1, 5, 3), (2, n - 1, 71), (2, 0, 64)]
    for i, col, r in spots:
        b[i, col, r] = bad
    got = lora_run(x, w, a, b, ids, scale)
    hit = torch.zeros(got.shape, dtype=torch.bool)
    for i, col, _ in spots:
        hit[ids == i, col] = True
    assert not torch.isfinite(got[hit]).any()
    assert torch.equal(got[~hit], ref[~hit])


@pytest.mark.parametrize("rows", [20, 300])
def test_other_rows_contents_never_reach_a_row(rows):
    rng = np.random.default_rng(8)
    x, w, a, b, scale = operands(rng, rows, 136, 264, 24, 3, torch.bfloat16)
    ids = torch.from_numpy((np.arange(rows) % 4 - 1).astype(np.int32))
    ref = lora_ref(x, w, a, b, ids, scale).bfloat16()
    x[::5] = float("inf")
    x[1::5] = float("nan")
    got = lora_run(x, w, a, b, ids, scale)
    keep = torch.arange(rows) % 5 > 1
    assert torch.equal(got[keep], ref[keep])


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rows", [33, 400])
def test_real_values(kind, rows):
    """Half a step of the result, half a step of every u that enters it, and the fp32 sums' error,
    at most (terms + 1) 2^-23 of the sum of magnitudes."""
    kind = KINDS[kind]
    rng = np.random.default_rng(9)

    def normal(shape, scale=1.0):
        return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(kind)

    n, k, rank, adapters = 264, 520, 48, 5
    x, w, a, b = normal((rows, k)), normal((n, k)), normal((adapters, rank, k), k ** -0.5), normal((adapters, n, rank))
    scale = torch.rand(adapters) + 0.5
    ids = torch.from_numpy(rng.integers(-1, adapters, size=rows).astype(np.int32))
    ref = lora_ref(x, w, a, b, ids, scale)
    base = lora_ref(x.abs(), w.abs(), a[:0], b[:0], ids, None)
    delta = lora_ref(x, torch.zeros_like(w), a, b.abs(), ids, scale)  # for the shape
    u = torch.zeros((rows, rank), dtype=torch.float64)
    mag = torch.zeros((rows, rank), dtype=torch.float64)
    mine = torch.zeros_like(delta)
    fuzz = torch.zeros_like(delta)
    for i in range(adapters):
        at = ids == i
        u[at] = float(scale[i]) * (x[at].double() @ a[i].double().T)
        mag[at] = float(scale[i]) * (x[at].abs().double() @ a[i].abs().double().T)
        mine[at] = u[at].abs() @ b[i].abs().double().T
        fuzz[at] = ((k + 1) * 2.0 ** -23 * mag[at]) @ b[i].abs().double().T
    half = 2 * HALF_STEP[kind]
    bound = half * ref.abs() + half * 1.01 * mine + 2 * fuzz + (k + rank + 1) * 2.0 ** -23 * (base + 2 * mine)
    got = lora_run(x, w, a, b, ids, scale).double()
    assert ((got - ref).abs() <= bound).all()


def test_repeats_on_another_stream():
    rng = np.random.default_rng(10)
    x = torch.from_numpy(rng.standard_normal((48, 1032)).astype(np.float32)).half()
    w = torch.from_numpy(rng.standard_normal((200, 1032)).astype(np.float32)).half()
    a = torch.from_numpy(rng.standard_normal((6, 16, 1032)).astype(np.float32)).half()
    b = torch.from_numpy(rng.standard_normal((6, 200, 16)).astype(np.float32)).half()
    ids = torch.from_numpy(rng.integers(-1, 6, size=48).astype(np.int32))
    first = lora_run(x, w, a, b, ids)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert torch.equal(lora_run(x, w, a, b, ids, stream=side), first)
    assert torch.equal(lora_run(x, w, a, b, ids), first)
    no_device_error()


def test_captured_in_a_graph_follows_new_inputs():
    rng = np.random.default_rng(11)
    rows, n, k, rank, adapters = 24, 136, 520, 16, 4
    x, w, a, b, scale = operands(rng, rows, n, k, rank, adapters, torch.float16)
    xd, wd, ad, bd, sd = (t.cuda() for t in (x, w, a, b, scale))
    idd = torch.zeros(rows, dtype=torch.int32, device="cuda")
    y = torch.zeros((rows, n), dtype=torch.float16, device="cuda")
    ws = torch.zeros(R.gemm_lora_workspace_size(rows, n, k, rank, adapters), dtype=torch.uint8, device="cuda")
    R.gemm_lora_nt(xd, wd, ad, bd, idd, sd, y=y, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.gemm_lora_nt(xd, wd, ad, bd, idd, sd, y=y, workspace=ws)
    for seed in range(4):
        ids = torch.from_numpy(np.random.default_rng(seed).integers(-1, adapters, size=rows).astype(np.int32))
        idd.copy_(ids)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), lora_ref(x, w, a, b, ids, scale).half())
    no_device_error()
