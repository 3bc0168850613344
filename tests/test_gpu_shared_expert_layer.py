"""The expert layer with a shared expert against the same layer written in 64-bit torch with automatic differentiation: the
router with scores, the products with an epilogue and their gradients together, with rows that have fewer experts than choices."""
import pytest

from ragged_helpers import no_device_error, require_gpu, torch

from dense_fp16_gemm_03_gb300 import expert_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def build(rows, width, hidden, experts, top, shared, groups, top_groups, masked=False):
    layer = expert_layer.SharedExpertLayer(width, hidden, experts, top, rows, shared, groups=groups, top_groups=top_groups, scale=1.5)
    layer.balance.normal_(0.0, 0.05, generator=torch.Generator(device="cuda").manual_seed(3))
    if masked:  # groups of which two experts are left
        layer.balance[: experts // 2][torch.arange(experts // 2) % 4 != 0] = -float("inf")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=gen, device="cuda").bfloat16()
    dout = torch.randn(rows, width, generator=gen, device="cuda").bfloat16()
    return layer, x, dout


def reference(layer, x, dout, ids):
    leaf = [t.double().requires_grad_() for t in (x, layer.router, layer.up, layer.down, layer.w1, layer.b1, layer.w2, layer.b2)]
    xd, router, up, down, w1, b1, w2, b2 = leaf
    have = ids >= 0
    at = ids.clamp(min=0).long()
    s = torch.where(have, torch.gather(torch.sigmoid(xd @ router.T), 1, at), 0.0)
    w = layer.scale * s / s.sum(1, keepdim=True)
    h = torch.einsum("tk,tjnk->tjn", xd, up[at])
    y = torch.einsum("tjn,tjkn->tjk", torch.relu(h).square(), down[at])
    want = (w[:, :, None] * y).sum(1) + torch.nn.functional.gelu(xd @ w1.T + b1) @ w2.T + b2
    want.backward(dout.double())
    return want.detach(), [t.grad for t in leaf]


NAMES = ("x", "router", "up", "down", "w1", "b1", "w2", "b2")


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("rows,width,hidden,experts,top,shared,groups,top_groups",
                         [(1, 64, 128, 8, 2, 136, 2, 1), (37, 72, 136, 16, 3, 72, 4, 2), (700, 128, 264, 32, 4, 520, 8, 3)])
def test_layer_and_its_gradients(rows, width, hidden, experts, top, shared, groups, top_groups, masked):
    """Every stored intermediate is rounded to bf16 (half a step is at most 2^-8 of a value): h, a, y, the routed sum, s, z, dz, da, dh on
    the way, of which a square doubles one, so norms are off by at most some 10 roundings of 2^-8, spread evenly a third of that
    each; the bound takes 10 * 2^-8 whole."""
    layer, x, dout = build(rows, width, hidden, experts, top, shared, groups, top_groups, masked)
    out, saved = layer.forward(x)
    grads = layer.backward(dout, saved)
    no_device_error()
    ids = saved[2].ids
    if masked:
        assert not torch.isin(ids, torch.nonzero(torch.isinf(layer.balance)).flatten().int()).any()
    want, refs = reference(layer, x, dout, ids)
    for name, got, ref in [("out", out, want)] + list(zip(NAMES, grads, refs)):
        off = float((got.double() - ref).norm() / ref.norm())
        assert off <= 10 * 2.0 ** -8, (name, off)


def test_a_captured_training_step():
    """Forward, backward and the bias's step in a graph: replays on new inputs give what eager calls give."""
    layer, x, dout = build(300, 128, 264, 16, 4, 264, 4, 2)
    start = layer.balance.clone()

    def step():
        out, saved = layer.forward(x)
        grads = layer.backward(dout, saved)
        layer.rebalance(saved[2])
        return [out, *grads]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (5, 6):
        x.copy_(torch.randn(300, 128, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        layer.balance.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        after = layer.balance.clone()
        got = [t.clone() for t in captured]
        layer.balance.copy_(start)
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(after, layer.balance)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    no_device_error()


def test_rebalance_moves_the_bias_by_the_counts():
    layer, x, _ = build(200, 64, 72, 16, 2, 72, 4, 2)
    _, saved = layer.forward(x)
    before, counts = layer.balance.clone(), torch.bincount(saved[2].ids.flatten().long(), minlength=16).float()
    layer.rebalance(saved[2], rate=0.25)
    assert torch.equal(layer.balance, before + 0.25 * torch.sign(counts.mean() - counts))
    no_device_error()


def test_the_command_runs(monkeypatch, capsys):
    argv = "expert_layer --rows 80 --width 64 --hidden 72 --experts 16 --top 2 --groups 4 --top-groups 2 --shared 72"
    monkeypatch.setattr("sys.argv", argv.split())
    expert_layer.main()
    assert "with a shared expert, backward" in capsys.readouterr().out


def test_no_rows():
    layer = expert_layer.SharedExpertLayer(64, 128, 8, 2, 32, 96, groups=4, top_groups=2)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    out, saved = layer.forward(x)
    grads = layer.backward(torch.empty_like(out), saved)
    no_device_error()
    assert out.shape == grads[0].shape == (0, 64)
    for g, like in zip(grads[1:], (layer.router, layer.up, layer.down, layer.w1, layer.b1, layer.w2, layer.b2)):
        assert g.shape == like.shape and not g.any()
