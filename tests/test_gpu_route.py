"""The experts' router against a 64-bit host implementation: whole numbers equal, weights and gradients within
a bound from their formulas (exp to 2 units in the last place, sums of up to 1024 terms in fp32)."""
import numpy as np
import pytest

from ragged_helpers import G, R, grouped_ref, no_device_error, require_gpu, route_ref, route_run, torch

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# a weight is a quotient of an exp (2 ulp, and |z - m| 2^-24 from the subtraction) and a sum of at most 1024 of
# them added in 32 lanes and five steps: (2 + 40 + 32 + 5 + 1) 2^-24 with |z - m| <= 40, rounded up
WEIGHT = 100 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def check(logits, top, renorm):
    want = route_ref(logits, top, renorm)
    got = route_run(logits, top, renorm)
    for name in ("ids", "offsets", "order", "position"):
        g = getattr(got, name).cpu().numpy()
        assert np.array_equal(g, want[name]), "%s: %s" % (name, np.argwhere(g != want[name])[:3].tolist())
    w = got.weights.cpu().double().numpy()
    assert np.array_equal(np.isnan(w), np.isnan(want["weights"]))
    fine = ~np.isnan(w)
    assert (np.abs(w - want["weights"])[fine] <= WEIGHT * want["weights"][fine] + 2.0 ** -126).all()
    return got, want


def draw(rows, experts, kind, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((1.5 * rng.standard_normal((rows, experts))).astype(np.float32)).to(TYPES[kind])


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("rows", [1, 2, 63, 64, 65, 300])
@pytest.mark.parametrize("experts,top", [(1, 1), (8, 2), (31, 8), (64, 8), (65, 5), (128, 8), (256, 8), (500, 6), (1024, 32)])
def test_choice(kind, rows, experts, top, renorm):
    check(draw(rows, experts, kind, rows + experts), top, renorm)


@pytest.mark.parametrize("rows,experts,top", [(5000, 64, 8), (2500, 7, 7), (4100, 200, 1)])
def test_many_rows(rows, experts, top):
    check(draw(rows, experts, "bf16", 1), top, True)


def test_ties_go_to_the_lowest_index():
    z = torch.zeros((70, 40))
    z[1] = -0.0
    z[2, ::2] = -0.0
    z[3, 5:] = 1.0
    z[4] = torch.finfo(torch.float32).min
    check(z, 8, True)
    check(z.half().clamp(-65504, 65504), 8, False)


@pytest.mark.parametrize("rows", [6, 70])
def test_masked_experts(rows):
    """-infinity is never chosen: rows with fewer experts than choices, and with none."""
    z = draw(rows, 24, "f32", 3)
    z[0] = -float("inf")
    z[1, 3:] = -float("inf")
    z[2, :] = -float("inf")
    z[2, 23] = -1e30
    z[3, ::2] = -float("inf")
    z[4] = torch.finfo(torch.float32).min
    got, _ = check(z, 8, True)
    check(z, 8, False)
    live = int((got.ids >= 0).sum())
    assert int(got.offsets[-1]) == live and (got.order[live:] == -1).all()


def test_every_row_masked():
    check(torch.full((130, 9), -float("inf")), 4, False)


@pytest.mark.parametrize("renorm", [False, True])
def test_nan_and_infinity(renorm):
    z = draw(70, 24, "f32", 4)
    z[0, 5] = float("nan")
    z[1] = float("nan")
    z[2, 3] = float("inf")
    z[3, :20] = -float("inf")
    z[3, 21] = float("nan")
    want = route_ref(z, 8, renorm)
    got = route_run(z, 8, renorm)
    assert np.array_equal(got.ids.cpu().numpy(), want["ids"])
    w = got.weights.cpu().numpy()
    assert np.isnan(w[0]).all() and np.isnan(w[1]).all() and np.isnan(w[2]).all()
    assert np.isnan(w[3, :4]).all() and not w[3, 4:].any()
    assert not np.isnan(w[4:]).any()


def test_no_rows():
    r = route_run(torch.zeros((0, 16)), 4)
    assert r.ids.shape == (0, 4) and not r.offsets.any()


def grad_ref(z, ids, w, dw, renorm):
    z = z.double().numpy()
    dl = np.zeros_like(z)
    inner = (w * dw).sum(1)
    m = z.max(1, keepdims=True)
    with np.errstate(all="ignore"):
        p = np.exp(z - m)
        p = np.where(np.isfinite(m), p / p.sum(1, keepdims=True), 0.0)
    for t in range(z.shape[0]):
        for j in range(ids.shape[1]):
            if ids[t, j] < 0:
                continue
            dl[t, ids[t, j]] += w[t, j] * (dw[t, j] - inner[t]) if renorm else p[t, ids[t, j]] * dw[t, j]
        if not renorm:
            dl[t] -= p[t] * inner[t]
    return dl


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("rows,experts,top", [(1, 8, 2), (65, 64, 8), (300, 300, 6), (9, 1024, 32), (5, 1, 1)])
def test_gradient(kind, rows, experts, top, renorm):
    """Against the formula: each entry is p times a difference, off by at most 2 WEIGHT p (|dw| + sum w |dw|)."""
    z = draw(rows, experts, kind, experts)
    if experts > 8:
        z[0] = -float("inf")
        z[-1, 4:] = -float("inf")
    want = route_ref(z, top, renorm)
    rng = np.random.default_rng(5)
    dw = rng.standard_normal((rows, top)).astype(np.float32)
    r = route_run(z, top, renorm)
    got = R.gemm_route_topk_grad(z.cuda(), r.ids, r.weights, torch.from_numpy(dw).cuda(), renorm=renorm).cpu().double().numpy()
    ref = grad_ref(z, want["ids"], want["weights"], dw.astype(np.float64), renorm)
    size = grad_ref(z, want["ids"], want["weights"], np.abs(dw).astype(np.float64), False)
    reach = np.abs(dw).max() * 2
    bound = 2 * WEIGHT * (np.abs(ref) + np.abs(size) + reach * np.where(ref != 0, 1.0, 0.0) * np.exp(0)) + 2.0 ** -126
    assert (np.abs(got - ref) <= bound).all()
    assert not got[ref == 0].any() or renorm is False


@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(renorm):
    """sum(w c) moves by dlogits . v along v; central differences of the 64-bit forward with h = 1e-5 are off by
    O(h^2) of third derivatives bounded by 6 |c|."""
    rng = np.random.default_rng(6)
    z = draw(20, 30, "f32", 7)
    c = rng.standard_normal((20, 5))
    r = route_run(z, 5, renorm)
    dl = R.gemm_route_topk_grad(z.cuda(), r.ids, r.weights, torch.from_numpy(c).float().cuda(), renorm=renorm)
    v = rng.standard_normal((20, 30))
    h = 1e-5
    side = [route_ref(z.double() + s * h * torch.from_numpy(v), 5, renorm) for s in (1, -1)]
    assert np.array_equal(side[0]["ids"], side[1]["ids"])
    slope = (((side[0]["weights"] - side[1]["weights"]) * c).sum(1)) / (2 * h)
    got = (dl.cpu().double().numpy() * v).sum(1)
    assert (np.abs(got - slope) <= 1e-5 * (1 + np.abs(c).sum(1) * np.abs(v).max(1))).all()


def test_route_then_experts():
    """The offsets and the order feed the grouped product as they are."""
    rng = np.random.default_rng(8)
    rows, experts, top, n, k = 90, 12, 3, 64, 136
    z = draw(rows, experts, "f32", 9)
    z[:, 4] = -float("inf")
    x = torch.from_numpy(rng.integers(-8, 9, size=(rows, k)).astype(np.float32) / 8).half()
    w = torch.from_numpy(rng.integers(-8, 9, size=(experts, n, k)).astype(np.float32) / 8).half()
    r = route_run(z, top)
    xs = x.cuda()[(r.order // top).long()]
    y = R.gemm_grouped_nt(xs, w.cuda(), r.offsets)
    no_device_error()
    assert torch.equal(y.cpu(), grouped_ref("nt", xs.cpu(), w, r.offsets, experts).half())
    assert G.gemm_f16_take_device_error()[0] == G.GEMM_OK


def test_very_many_rows():
    """More blocks than one sums by itself: the counts are scanned by a kernel of their own."""
    check(draw(40000, 16, "bf16", 2), 4, False)
