"""The router with scores, a bias and groups against a 64-bit host implementation: whole numbers equal, also where two scores
differ by less than 32 bits hold, weights and gradients within bounds from their formulas."""
import numpy as np
import pytest

from ragged_helpers import G, R, grouped_ref, no_device_error, require_gpu, torch

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# A weight in units of 2^-24: an exponential of l - m (4, and |l - m| <= 40 from the subtraction) over a sum of exponentials (4 and
# twice their mean argument, below 7, each; up to 37 additions) with a quotient and the scale: 4 + 40 + 18 + 37 + 3; less for a sigmoid.
WEIGHT = 120 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def scores(z, score):
    """s of every logit in float64, rows of a softmax with NaN or +infinity NaN."""
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z)))) + 0 * np.where(np.isnan(z), z, 0)
        m = z.max(1, keepdims=True)
        p = np.where(z == -np.inf, 0.0, np.exp(z - np.where(np.isfinite(m), m, 0)))
        p = p / np.where(p.sum(1, keepdims=True) == 0, 1, p.sum(1, keepdims=True))
        return np.where(np.isnan(m) | (m == np.inf), np.nan, p)


def ref(logits, top, score="sigmoid", bias=None, groups=1, top_groups=None, group_top=2, renorm=True, scale=1.0):
    z = logits.double().numpy()
    rows, experts = z.shape
    top_groups = groups if top_groups is None else top_groups
    b = np.zeros(experts) if bias is None else bias.double().numpy()
    s = scores(z, score)
    with np.errstate(all="ignore"):
        c = s + b
    if bias is None:  # the logits' order; NaN throughout a row whose softmax is none
        by = np.where(np.isnan(s), np.nan, z)
    else:
        by = c
    off = (z == -np.inf) | (b == -np.inf)

    def rank(v, masked):  # sortable: what cannot be chosen, NaN, the others
        return (0, 0.0) if masked else (1, 0.0) if np.isnan(v) else (2, v)

    size = experts // groups
    ids = np.full((rows, top), -1, dtype=np.int32)
    w = np.zeros((rows, top))
    for t in range(rows):
        keys = [rank(by[t, e], off[t, e]) for e in range(experts)]
        if groups > 1:
            sums = []
            for g in range(groups):
                mine = sorted(range(g * size, (g + 1) * size), key=lambda e: keys[e], reverse=True)
                mine = [e for e in mine if keys[e][0]][:group_top]
                if not mine:
                    sums.append((0, 0.0))
                elif group_top == 1 and bias is None:
                    sums.append(keys[mine[0]])
                else:
                    v = c[t, mine].sum()
                    sums.append(rank(v, False))
            order = sorted(range(groups), key=lambda g: (-sums[g][0], -sums[g][1], g))[:top_groups]
            keys = [k if e // size in order else (0, 0.0) for e, k in enumerate(keys)]
        pick = sorted((e for e in range(experts) if keys[e][0]), key=lambda e: (-keys[e][0], -keys[e][1], e))[:top]
        ids[t, : len(pick)] = pick
        if pick:
            total = s[t, pick].sum() if renorm else 1.0
            w[t, : len(pick)] = scale * s[t, pick] / total if total != 0 else 0.0
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat < 0, experts, flat), kind="stable").astype(np.int32)
    live = int((flat >= 0).sum())
    position = np.full(rows * top, -1, dtype=np.int32)
    position[order[:live]] = np.arange(live)
    order[live:] = -1
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=experts))]).astype(np.int32)
    return {"ids": ids, "weights": w, "offsets": offsets, "order": order, "position": position.reshape(rows, top)}


def run(logits, top, bias=None, stream=None, **how):
    rows, experts = logits.shape
    ws = torch.full((max(1, R.gemm_route_workspace_size(rows, experts, top)),), 0xA5, dtype=torch.uint8, device="cuda")
    r = R.gemm_route_scored(logits.cuda(), top, bias=None if bias is None else bias.cuda(), workspace=ws, stream=stream, **how)
    no_device_error(stream)
    return r


def check(logits, top, **how):
    want, got = ref(logits, top, **how), run(logits, top, **how)
    for name in ("ids", "offsets", "order", "position"):
        g = getattr(got, name).cpu().numpy()
        assert np.array_equal(g, want[name]), "%s: %s" % (name, np.argwhere(g != want[name])[:3].tolist())
    w = got.weights.cpu().double().numpy()
    assert np.array_equal(np.isnan(w), np.isnan(want["weights"]))
    fine = ~np.isnan(w)
    assert (np.abs(w - want["weights"])[fine] <= WEIGHT * np.abs(want["weights"][fine]) + 2.0 ** -126).all()
    return got, want


def draw(rows, experts, kind, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((1.5 * rng.standard_normal((rows, experts))).astype(np.float32)).to(TYPES[kind])


def draw_bias(experts, seed, size=0.05):
    return torch.from_numpy((size * np.random.default_rng(seed).standard_normal(experts)).astype(np.float32))


FORMS = [  # experts, groups, top_groups, top
    (1, 1, 1, 1), (8, 1, 1, 2), (31, 1, 1, 8), (65, 1, 1, 5), (256, 8, 4, 8), (256, 1, 1, 8), (160, 8, 3, 6), (64, 16, 5, 8), (12, 4, 2, 6),
    (32, 32, 7, 7), (40, 8, 8, 3), (10, 2, 1, 5), (512, 16, 4, 8), (1024, 4, 2, 32), (1024, 1, 1, 32), (384, 1, 1, 8), (96, 32, 20, 10),
]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("rows", [1, 9, 30, 64, 65])
@pytest.mark.parametrize("experts,groups,top_groups,top", FORMS)
def test_choice(experts, groups, top_groups, top, rows, kind, score):
    z = draw(rows, experts, kind, rows + experts)
    bias = draw_bias(experts, experts)
    for i, (b, group_top, renorm) in enumerate([(bias, 2, True), (bias, 1, False), (None, 1, True), (None, 2, False)]):
        check(z, top, score=score, bias=b, groups=groups, top_groups=top_groups, group_top=group_top, renorm=renorm, scale=(1.0, 2.5)[i % 2])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_many_rows(score):
    check(draw(3000, 256, "bf16", 1), 8, score=score, bias=draw_bias(256, 2), groups=8, top_groups=4, scale=2.5)
    check(draw(2100, 40, "f16", 2), 3, score=score, bias=draw_bias(40, 3), groups=4, top_groups=2, group_top=1, renorm=False)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [1, 8])
def test_scores_closer_than_32_bits(score, groups):
    """Biases that make the chosen experts' c of a row equal but for the bias's own rounding: their order is that of the 64-bit sums.
    All rows have the row's logits in another order, so that it is the same c with other neighbours."""
    rng = np.random.default_rng(11)
    experts, rows, top = 64, 80, 6
    z = np.tile((1.5 * rng.standard_normal(experts)).astype(np.float32), (rows, 1))
    s = scores(z.astype(np.float64), score)[0]
    bias = (s.max() + 0.25 - s).astype(np.float32)  # c = the same for all, within 2^-25 or so
    gaps = np.diff(np.sort(s + bias.astype(np.float64)))
    assert gaps.min() > 1e-13 and gaps.max() < 1e-6
    got, want = check(torch.from_numpy(z), top, score=score, bias=torch.from_numpy(bias), groups=groups, top_groups=max(1, groups // 2))
    assert len(set(want["ids"][0].tolist())) == top
    # a logit moved by its last bits changes who is first
    for t in range(rows):
        z[t, t % experts] = np.nextafter(z[t, t % experts], np.float32(10), dtype=np.float32)
    check(torch.from_numpy(z), top, score=score, bias=torch.from_numpy(bias), groups=groups, top_groups=max(1, groups // 2))


def test_groups_closer_than_32_bits():
    """Groups whose two largest differ, with sums that are equal but for their last bits."""
    rng = np.random.default_rng(12)
    groups, size, rows = 8, 8, 70
    z = np.full((rows, groups * size), -9.0, dtype=np.float32)
    bias = np.zeros(groups * size, dtype=np.float32)
    first = rng.uniform(0.2, 0.4, groups).astype(np.float32)
    low = scores(np.full((1, 1), -9.0), "sigmoid")[0, 0]
    for g in range(groups):  # c: first[g] + low and (1 - first[g]) + low, with first[g] rounded to fp32
        bias[g * size + g] = first[g]
        bias[g * size + (g + 3) % size] = np.float32(1.0) - first[g] * np.float32(1 + (g % 3) * 2.0 ** -23)
    assert low > 0
    check(torch.from_numpy(z), 5, bias=torch.from_numpy(bias), groups=groups, top_groups=3)
    for t in range(rows):
        z[t, rng.integers(0, groups * size)] += rng.uniform(0, 1e-5)
    check(torch.from_numpy(z), 5, bias=torch.from_numpy(bias), groups=groups, top_groups=3)


@pytest.mark.parametrize("bias", [None, 0.0, 0.5])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_go_to_the_lowest_index(score, bias):
    z = torch.zeros((70, 40))
    z[1] = -0.0
    z[2, ::2] = -0.0
    z[3, 5:] = 1.0
    z[4] = -80.0
    z[5, 7:20] = 2.0
    b = None if bias is None else torch.full((40,), bias)
    for group_top in (1, 2):
        check(z, 8, score=score, bias=b, groups=4, top_groups=2, group_top=group_top)
        check(z.half(), 8, score=score, bias=b, group_top=group_top)
        check(z.bfloat16(), 8, score=score, bias=b, groups=8, top_groups=3, group_top=group_top, renorm=False)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_many_equal_scores(score):
    """More experts with one score than a warp's lanes, alone, with one just beside them, and in groups."""
    z = torch.full((70, 256), 0.75)
    for t in range(1, 70):
        z[t, (37 * t) % 256] = float(np.nextafter(np.float32(0.75), np.float32(1 if t % 2 else 0)))
    for b in (None, torch.full((256,), 0.125)):
        check(z, 8, score=score, bias=b)
        for group_top in (1, 2):
            check(z, 8, score=score, bias=b, groups=8, top_groups=4, group_top=group_top)
            check(z.bfloat16(), 30, score=score, bias=b, groups=8, top_groups=1, group_top=group_top)


def test_coarse_logits_with_an_even_bias():
    """bf16 logits repeat within a row; a bias that is the same for all, as at the start of a training, keeps their order."""
    z = draw(500, 256, "bf16", 13)
    for b in (torch.zeros(256), torch.full((256,), -0.3)):
        check(z, 8, bias=b, groups=8, top_groups=4)
        check(z, 8, bias=b)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("rows", [8, 70])
def test_masked_experts(rows, score):
    """-infinity among logits or biases is never chosen: rows, and groups, with fewer experts than choices, and with none."""
    z = draw(rows, 24, "f32", 3)
    z[0] = -float("inf")
    z[1, 3:] = -float("inf")
    z[2, :] = -float("inf")
    z[2, 23] = -30.0
    z[3, ::2] = -float("inf")
    z[4, 6:12] = -float("inf")
    z[5, :18] = -float("inf")
    z[6, 1:] = -float("inf")
    b = draw_bias(24, 4)
    for bias in (None, b, torch.where(torch.arange(24) % 5 == 0, -float("inf"), b)):
        for group_top in (1, 2):
            got, _ = check(z, 8, score=score, bias=bias, groups=4, top_groups=2, group_top=group_top)
            live = int((got.ids >= 0).sum())
            assert int(got.offsets[-1]) == live and (got.order[live:] == -1).all()
            check(z, 8, score=score, bias=bias, groups=1, group_top=group_top, renorm=False)


def test_every_expert_masked():
    check(torch.full((130, 8), -float("inf")), 4, bias=draw_bias(8, 1))
    check(draw(70, 8, "f32", 1), 2, bias=torch.full((8,), -float("inf")), groups=2, top_groups=1)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_nan_and_infinity(score, renorm):
    z = draw(70, 24, "f32", 4)
    z[0, 5] = float("nan")
    z[1] = float("nan")
    z[2, 3] = float("inf")
    z[3, :20] = -float("inf")
    z[3, 21] = float("nan")
    z[4, :12] = float("nan")
    b = draw_bias(24, 5)
    infinite = b.clone()
    infinite[2], infinite[9], infinite[20] = float("inf"), float("inf"), float("nan")
    for bias in (None, b, infinite):
        for groups, top_groups, group_top in ((1, 1, 2), (4, 3, 1), (4, 2, 2)):
            check(z, 8, score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top, renorm=renorm)


def test_scores_that_underflow():
    """Scores too small for 32 bits keep their ratio, as in 64."""
    z = torch.full((3, 16), -200.0)
    z[1] = torch.linspace(-80, -60, 16)
    z[2, 3] = 200.0
    check(z, 4, score="sigmoid")
    check(z, 4, score="softmax", bias=torch.arange(16.0))
    dw = torch.randn(3, 4)
    for score, bias in (("sigmoid", None), ("softmax", torch.arange(16.0))):
        r = run(z, 4, score=score, bias=bias)
        got = R.gemm_route_scored_grad(z.cuda(), r.ids, dw.cuda(), score=score)
        want, size = grad_ref(z, r.ids.cpu().numpy(), dw.double().numpy(), score, True, 1.0)
        assert (np.abs(got.cpu().double().numpy() - want) <= 2 * WEIGHT * size + 2.0 ** -120).all()


def test_no_rows():
    r = run(torch.zeros((0, 16)), 4, groups=2)
    assert r.ids.shape == (0, 4) and not r.offsets.any()


@pytest.mark.parametrize("top,how", [(5, {"groups": 3}), (5, {"groups": 8, "top_groups": 1}), (2, {"groups": 4, "top_groups": 5}), (0, {}),
                                     (2, {"group_top": 3}), (2, {"score": "tanh"}), (2, {"bias": torch.zeros(15)})])
def test_refusals(top, how):
    how = {name: v.cuda() if name == "bias" else v for name, v in how.items()}
    with pytest.raises(ValueError):
        R.gemm_route_scored(torch.zeros((3, 16), device="cuda"), top, **how)


def test_groups_that_are_no_power_of_two_are_refused():
    with pytest.raises(G.GemmError):
        run(torch.zeros((3, 18)), 2, groups=6, top_groups=2)


def grad_ref(z, ids, dw, score, renorm, scale):
    """dlogits by the formula, and the sum of the magnitudes of its terms."""
    z = z.double().numpy()
    s = scores(z, score)
    dl, size = np.zeros_like(z), np.zeros_like(z)
    for t in range(z.shape[0]):
        at = ids[t][ids[t] >= 0]
        d = dw[t][ids[t] >= 0] * scale
        if len(at) == 0:
            continue
        total = s[t, at].sum() if renorm else 1.0
        if score == "sigmoid":
            slope = s[t, at] * scores(-z[t:t + 1, at], "sigmoid")[0]
            g, m = (d - (d * s[t, at]).sum() / total, np.abs(d) + (np.abs(d) * s[t, at]).sum() / total) if renorm else (d, np.abs(d))
            dl[t, at], size[t, at] = slope * g / total, slope * m / total
        elif renorm:
            v = s[t, at] / total
            dl[t, at], size[t, at] = v * (d - (d * v).sum()), v * (np.abs(d) + (np.abs(d) * v).sum())
        else:
            dp, mp = np.zeros(z.shape[1]), np.zeros(z.shape[1])
            dp[at], mp[at] = d, np.abs(d)
            dl[t], size[t] = s[t] * (dp - (dp * s[t]).sum()), s[t] * (mp + (mp * s[t]).sum())
    return dl, size


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("rows,experts,groups,top_groups,top", [(1, 8, 1, 1, 2), (65, 64, 8, 3, 6), (300, 300, 4, 2, 6), (9, 1024, 1, 1, 32), (5, 1, 1, 1, 1)])
def test_gradient(rows, experts, groups, top_groups, top, kind, renorm, score):
    """Each term is a product of weights and dw: off by at most 2 WEIGHT of the terms' magnitudes."""
    z = draw(rows, experts, kind, experts)
    if experts > 8:
        z[0] = -float("inf")
        z[-1, 4:] = -float("inf")
    dw = np.random.default_rng(5).standard_normal((rows, top)).astype(np.float32)
    r = run(z, top, score=score, bias=draw_bias(experts, 6), groups=groups, top_groups=top_groups, renorm=renorm, scale=2.5)
    got = R.gemm_route_scored_grad(z.cuda(), r.ids, torch.from_numpy(dw).cuda(), score=score, renorm=renorm, scale=2.5)
    want, size = grad_ref(z, r.ids.cpu().numpy(), dw.astype(np.float64), score, renorm, 2.5)
    assert (np.abs(got.cpu().double().numpy() - want) <= 2 * WEIGHT * size + 2.0 ** -120).all()
    no_device_error()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    """sum(w c) moves by dlogits . v along v; central differences of the 64-bit forward with h = 1e-5 are off by O(h^2)."""
    rng = np.random.default_rng(6)
    how = dict(score=score, bias=draw_bias(32, 7), groups=4, top_groups=2, renorm=renorm, scale=1.5)
    z = draw(20, 32, "f32", 7)
    c = rng.standard_normal((20, 5))
    r = run(z, 5, **how)
    dl = R.gemm_route_scored_grad(z.cuda(), r.ids, torch.from_numpy(c).float().cuda(), score=score, renorm=renorm, scale=1.5)
    v = rng.standard_normal((20, 32))
    h = 1e-5
    side = [ref(z.double() + s * h * torch.from_numpy(v), 5, **how) for s in (1, -1)]
    assert np.array_equal(side[0]["ids"], side[1]["ids"])
    slope = (((side[0]["weights"] - side[1]["weights"]) * c).sum(1)) / (2 * h)
    got = (dl.cpu().double().numpy() * v).sum(1)
    assert (np.abs(got - slope) <= 1e-5 * (1 + np.abs(c).sum(1) * np.abs(v).max(1))).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_ids_given_twice_and_of_none(score, renorm):
    """The same expert twice adds up; ids outside the experts take no part."""
    z = draw(4, 40, "f32", 8)
    ids = torch.tensor([[3, 3, 7, -1], [3, 40, 1 << 30, 5], [-7, -1, 40, 99], [9, 9, 9, 9]], dtype=torch.int32)
    dw = torch.from_numpy(np.random.default_rng(9).standard_normal((4, 4)).astype(np.float32))
    got = R.gemm_route_scored_grad(z.cuda(), ids.cuda(), dw.cuda(), score=score, renorm=renorm).cpu().double()
    s = torch.from_numpy(scores(z.double().numpy(), score))
    want = torch.zeros((4, 40), dtype=torch.float64)
    size = torch.zeros_like(want)
    for t in range(4):
        on = [(int(e), float(d)) for e, d in zip(ids[t], dw[t]) if 0 <= e < 40]
        total = sum(float(s[t, e]) for e, _ in on) if renorm else 1.0
        mean = sum(d * float(s[t, e]) for e, d in on) / total if renorm and on else 0.0
        ds = torch.zeros(40, dtype=torch.float64)
        for e, d in on:
            ds[e] += (d - mean) / total
        want[t] = ds * s[t] * (1 - s[t]) if score == "sigmoid" else s[t] * (ds - (ds * s[t]).sum())
        size[t] = (s[t] * sum(abs(d) for _, d in on) * 2 / total) if on else 0.0
    assert (torch.abs(got - want) <= 8 * WEIGHT * size + 2.0 ** -120).all()
    no_device_error()


def test_as_the_softmax_router():
    """Without bias, groups and scale a softmax router chooses as gemm_route_topk does."""
    z = draw(200, 64, "bf16", 10)
    for renorm in (False, True):
        a = run(z, 8, score="softmax", renorm=renorm)
        ws = torch.empty(R.gemm_route_workspace_size(200, 64, 8), dtype=torch.uint8, device="cuda")
        b = R.gemm_route_topk(z.cuda(), 8, renorm=renorm, workspace=ws)
        for name in ("ids", "offsets", "order", "position"):
            assert torch.equal(getattr(a, name), getattr(b, name))
        assert torch.allclose(a.weights, b.weights, rtol=2 * WEIGHT, atol=0)


def test_on_another_stream_in_a_graph_and_again():
    z = draw(700, 256, "bf16", 14).cuda()
    bias = draw_bias(256, 15).cuda()
    dw = torch.randn(700, 8, device="cuda")
    ws = torch.empty(R.gemm_route_workspace_size(700, 256, 8), dtype=torch.uint8, device="cuda")
    out = R.gemm_route_scored(z, 8, bias=bias, groups=8, top_groups=4, workspace=ws)
    dl = torch.empty(700, 256, device="cuda")

    def step(stream=None):
        R.gemm_route_scored(z, 8, bias=bias, groups=8, top_groups=4, out=out, workspace=ws, stream=stream)
        R.gemm_route_scored_grad(z, out.ids, dw, dlogits=dl, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*out, dl)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for t in (*out, dl):
        t.fill_(0)
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (*out, dl)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (16, 17):
        z.copy_(draw(700, 256, "bf16", seed))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (*out, dl)]
        for t in (*out, dl):
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (*out, dl)))
    no_device_error()


def test_very_many_rows():
    """More blocks than one sums by itself: the counts are scanned by a kernel of their own."""
    z = draw(20000, 16, "bf16", 2)
    got = run(z, 4, bias=draw_bias(16, 1), groups=4, top_groups=2)
    few = run(z[:64], 4, bias=draw_bias(16, 1), groups=4, top_groups=2)
    assert torch.equal(got.ids[:64], few.ids) and torch.equal(got.weights[:64], few.weights)
    flat = got.ids.flatten().long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(order.int(), got.order) and int(got.offsets[-1]) == flat.numel()


def test_route_then_experts():
    """The offsets and the order feed the grouped product as they are."""
    rng = np.random.default_rng(8)
    rows, experts, top, n, k = 90, 16, 3, 64, 136
    z = draw(rows, experts, "f32", 9)
    x = torch.from_numpy(rng.integers(-8, 9, size=(rows, k)).astype(np.float32) / 8).half()
    w = torch.from_numpy(rng.integers(-8, 9, size=(experts, n, k)).astype(np.float32) / 8).half()
    r = run(z, top, bias=draw_bias(experts, 1), groups=4, top_groups=2)
    xs = x.cuda()[(r.order // top).long()]
    y = R.gemm_grouped_nt(xs, w.cuda(), r.offsets)
    no_device_error()
    assert torch.equal(y.cpu(), grouped_ref("nt", xs.cpu(), w, r.offsets, experts).half())


def test_outputs_are_tensors_of_their_own():
    """The outputs lie in one allocation: what is written to one, and what lives on, reaches no other."""
    z = draw(70, 24, "f32", 18)
    r = run(z, 5, bias=draw_bias(24, 1))
    want = [t.clone() for t in r]
    kept = r.offsets
    for i, t in enumerate(r):
        assert t.is_contiguous() and not t.requires_grad and t.data_ptr() % 16 == 0
        t.fill_(3)
        for j, o in enumerate(r):
            if j != i:
                assert torch.equal(o, want[j]) or j < i
    del r, t, o
    junk = [torch.full((100000,), 7, device="cuda", dtype=torch.int32) for _ in range(20)]
    assert (kept == 3).all() and kept.shape == (25,)
    assert (torch.cat([kept, kept]).cpu() == 3).all() and len(junk) == 20
