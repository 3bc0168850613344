"""The adapters as K blocks of the projection, on the tensor cores, against a 64-bit host implementation.

Which way a call takes goes by its sizes, so every case here takes the shortest contraction that sends it there, and
asserts it.  Integer operands keep the inner product x a^T small and whole, so the result must be the exact sum rounded
once, bit for bit."""
import numpy as np
import pytest

from ragged_helpers import KINDS, R, lora_ref, lora_run, no_device_error, require_gpu, small_ints, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def k_for(rows, n, rank, adapters, least=72):
    """The shortest contraction, of a whole number of eights and no whole number of K blocks, that takes the tensor cores."""
    def there(k):
        return R.gemm_lora_way(rows, n, k, rank, adapters) == R.LORA_TENSOR_CORES
    lo, hi = least // 8, 1 << 14
    assert there(8 * hi)
    while lo < hi:
        mid = (lo + hi) // 2
        if there(8 * mid):
            hi = mid
        else:
            lo = mid + 1
    k = 8 * lo
    return k if k % 64 else k + 8


def operands(rng, rows, n, k, rank, adapters, kind, ids):
    """x and a sparse enough that |x a^T| <= 64, whole numbers that both types hold exactly, under a scale of up to 2 as well."""
    x = small_ints(rng, (rows, k), kind, 2)
    a = small_ints(rng, (adapters, rank, k), kind, 1)
    a[torch.from_numpy(rng.random((adapters, rank, k)) < max(0.0, 1 - 48.0 / k))] = 0
    b = small_ints(rng, (adapters, n, rank), kind, 2)
    w = small_ints(rng, (n, k), kind, 2)
    w[torch.from_numpy(rng.random((n, k)) < max(0.0, 1 - 2048.0 / k))] = 0
    scale = torch.from_numpy(2.0 ** rng.integers(-1, 2, size=adapters)).float()
    for i in range(adapters):
        at = ids == i
        if at.any():
            assert (x[at].double() @ a[i].double().T).abs().max() <= 64
    return x, w, a, b, scale


def made(rows, n, rank, adapters, ids, kind, seed, least=72):
    k = k_for(rows, n, rank, adapters, least)
    assert R.gemm_lora_way(rows, n, k, rank, adapters) == R.LORA_TENSOR_CORES
    ids = torch.from_numpy(np.asarray(ids).astype(np.int32))
    return operands(np.random.default_rng(seed), rows, n, k, rank, adapters, kind, ids) + (ids,)


def check(rows, n, rank, adapters, ids, kind, seed, scaled=True, least=72):
    x, w, a, b, scale, ids = made(rows, n, rank, adapters, ids, kind, seed, least)
    scale = scale if scaled else None
    ref = lora_ref(x, w, a, b, ids, scale)
    got = lora_run(x, w, a, b, ids, scale)
    bad = torch.nonzero(got != ref.to(kind))
    assert bad.shape[0] == 0, "%d differ, first at %s: %s, want %s" % (
        bad.shape[0], bad[0].tolist(), got[tuple(bad[0])], ref[tuple(bad[0])])


# one row tile (split over the workers) up to 256 rows, several above; one half of a pair without columns at n = 8
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rows", [65, 200, 256, 257, 600])
@pytest.mark.parametrize("n,rank", [(8, 128), (136, 64), (264, 72), (1000, 120), (392, 40)])
def test_rows_with_adapters_of_their_own(kind, rows, n, rank):
    ids = np.random.default_rng(rows).integers(-1, 4, size=rows)
    check(rows, n, rank, 4, ids, KINDS[kind], seed=rows + n)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rank", [8, 16, 24, 32])
def test_low_ranks(kind, rank):
    ids = np.random.default_rng(rank).integers(-1, 3, size=900)
    check(900, 136, rank, 3, ids, KINDS[kind], seed=rank)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("ends", [[100, 300, 301, 700], [256, 512], [1, 2, 3, 200], [40, 600]])
def test_requests_in_runs(kind, ends):
    ids = np.repeat([3, 0, -1, 2][: len(ends)], np.diff([0] + ends))
    check(ends[-1], 264, 104, 4, ids, KINDS[kind], seed=len(ends))


@pytest.mark.parametrize("rows", [256, 500])
@pytest.mark.parametrize("rank", [64, 128])
def test_many_adapters_in_a_row_tile(rows, rank):
    """More adapter blocks than the projection has K blocks."""
    ids = np.random.default_rng(1).permutation(np.arange(rows) % 60)
    check(rows, 6000, rank, 60, ids, torch.bfloat16, seed=3)


@pytest.mark.parametrize("rows", [100, 300])
@pytest.mark.parametrize("ids", [-1, 4, 2 ** 31 - 1, -2 ** 31])
def test_no_row_has_an_adapter(rows, ids):
    check(rows, 136, 128, 4, np.full(rows, ids), torch.bfloat16, seed=4)


@pytest.mark.parametrize("rows", [100, 300])
def test_no_scale(rows):
    check(rows, 136, 128, 4, np.arange(rows) % 5 - 1, torch.float16, seed=5, scaled=False)


@pytest.mark.parametrize("rows", [100, 300])
def test_no_adapters(rows):
    check(rows, 136, 128, 0, np.zeros(rows), torch.float16, seed=6)


@pytest.mark.parametrize("rows", [200, 300])
def test_other_adapters_contents_never_reach_a_row(rows):
    """Adapters that a row does not have hold infinities and NaN, and a row without one keeps the projection."""
    x, w, a, b, scale, ids = made(rows, 136, 104, 3, np.arange(rows) % 4 - 1, torch.float16, seed=7)
    ref = lora_ref(x, w, a, b, ids, scale).half()
    a[2], b[2] = float("nan"), float("inf")
    got = lora_run(x, w, a, b, ids, scale)
    keep = ids != 2
    assert torch.equal(got[keep], ref[keep])
    assert not torch.isfinite(got[~keep]).any()


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rows,n", [(200, 136), (256, 2056), (300, 136), (1100, 1000)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_one_bad_value_of_b_spoils_its_own_column_and_rows(kind, rows, n, bad):
    x, w, a, b, scale, ids = made(rows, n, 72, 3, np.arange(rows) % 4 - 1, KINDS[kind], seed=12)
    ref = lora_ref(x, w, a, b, ids, scale).to(KINDS[kind])
    spots = [(1, 5, 3), (2, n - 1, 71), (2, 0, 64), (0, 130, 33)]
    for i, col, r in spots:
        b[i, col, r] = bad
    got = lora_run(x, w, a, b, ids, scale)
    hit = torch.zeros(got.shape, dtype=torch.bool)
    for i, col, _ in spots:
        hit[ids == i, col] = True
    assert not torch.isfinite(got[hit]).any()
    assert torch.equal(got[~hit], ref[~hit])


def test_bad_values_in_some_row_tiles_only():
    """The table of b's rows that hold an infinity is made anew for every tile: those after a spoilt one are whole."""
    rows, n = 2000, 1000
    ids = np.arange(rows) * 8 // rows
    x, w, a, b, scale, ids = made(rows, n, 72, 8, ids, torch.bfloat16, seed=16)
    ref = lora_ref(x, w, a, b, ids, scale).bfloat16()
    hit = torch.zeros(ref.shape, dtype=torch.bool)
    for i in (1, 4, 6):
        for col in (0, 127, 128, 500 + i, n - 1):
            b[i, col, 9 * i] = float("nan")
            hit[ids == i, col] = True
    got = lora_run(x, w, a, b, ids, scale)
    assert torch.isnan(got[hit]).all()
    assert torch.equal(got[~hit], ref[~hit])


@pytest.mark.parametrize("rows", [200, 300])
def test_other_rows_contents_never_reach_a_row(rows):
    x, w, a, b, scale, ids = made(rows, 136, 104, 3, np.arange(rows) % 4 - 1, torch.bfloat16, seed=8)
    ref = lora_ref(x, w, a, b, ids, scale).bfloat16()
    x[::5] = float("inf")
    x[1::5] = float("nan")
    got = lora_run(x, w, a, b, ids, scale)
    keep = torch.arange(rows) % 5 > 1
    assert torch.equal(got[keep], ref[keep])


def real(rng, kind, shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(kind)


def test_repeats_bit_for_bit_on_another_stream():
    rng = np.random.default_rng(10)
    for rows in (130, 700):
        k = k_for(rows, 200, 96, 6)
        x, w = real(rng, torch.float16, (rows, k)), real(rng, torch.float16, (200, k))
        a, b = real(rng, torch.float16, (6, 96, k), k ** -0.5), real(rng, torch.float16, (6, 200, 96))
        ids = torch.from_numpy(rng.integers(-1, 6, size=rows).astype(np.int32))
        first = lora_run(x, w, a, b, ids)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            assert torch.equal(lora_run(x, w, a, b, ids, stream=side), first)
        assert torch.equal(lora_run(x, w, a, b, ids), first)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rows,rank", [(130, 128), (600, 24), (600, 64), (900, 104)])
def test_the_inner_product_is_not_rounded_to_the_type(kind, rows, rank):
    """u = s x a^T of up to 16 significant bits, more than either type holds, and sums that fp32 holds exactly: the result
    is the exact sum rounded once."""
    kind = KINDS[kind]
    n, adapters = 264, 3
    k = k_for(rows, n, rank, adapters)
    assert R.gemm_lora_way(rows, n, k, rank, adapters) == R.LORA_TENSOR_CORES
    rng = np.random.default_rng(17)
    x, w = small_ints(rng, (rows, k), kind, 100), small_ints(rng, (n, k), kind, 1)
    a, b = small_ints(rng, (adapters, rank, k), kind, 7), small_ints(rng, (adapters, n, rank), kind, 2)
    w[torch.from_numpy(rng.random((n, k)) < 1 - 8.0 / k)] = 0
    a[torch.from_numpy(rng.random((adapters, rank, k)) < 1 - 48.0 / k)] = 0
    scale = torch.tensor([2.0 ** -5, 2.0 ** -4, 2.0 ** -5])
    ids = torch.from_numpy(rng.integers(-1, adapters, size=rows).astype(np.int32))
    most = torch.stack([(x.double() @ a[i].double().T).abs().max() for i in range(adapters)]).max()
    assert 2 ** 11 < most < 2 ** 16
    ref = lora_ref(x, w, a, b, ids, scale)
    assert ref.abs().max() < 65504
    got = lora_run(x, w, a, b, ids, scale)
    bad = torch.nonzero(got != ref.to(kind))
    assert bad.shape[0] == 0, "%d of %d differ" % (bad.shape[0], got.numel())


@pytest.mark.parametrize("rows", [200, 600])
def test_captured_in_a_graph_follows_new_inputs(rows):
    n, rank, adapters = 136, 72, 4
    x, w, a, b, scale, ids = made(rows, n, rank, adapters, np.zeros(rows), torch.float16, seed=11)
    k = x.shape[1]
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
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), lora_ref(x, w, a, b, ids, scale).half())
    no_device_error()
