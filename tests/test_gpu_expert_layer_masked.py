"""The expert layer where rows have fewer experts than choices."""
import pytest

from ragged_helpers import no_device_error, require_gpu, torch

from dense_fp16_gemm_03_gb300 import expert_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def masked_layer(rows, width=64, hidden=128, experts=6, top=4, live=2):
    """Experts from `live` on have a logit of -infinity for every row of positive numbers."""
    layer = expert_layer.ExpertLayer(width, hidden, experts, top, rows)
    layer.router[live:] = -float("inf")
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = (torch.rand(rows, width, generator=gen, device="cuda") + 0.1).bfloat16()
    return layer, x


@pytest.mark.parametrize("rows", [5, 100])
def test_a_missing_choice_takes_nothing_from_another_row(rows):
    """Row 0 stands first among the rows sorted by expert, and its result is infinite: no other row's is."""
    layer, x = masked_layer(rows)
    x[0] = 1e30
    out, saved = layer.forward(x)
    no_device_error()
    ids, position = saved[2].ids, saved[2].position
    assert (ids[:, 2:] == -1).all() and (ids[:, :2] >= 0).all() and int(position[0].min()) == -1
    assert 0 in position[0].tolist()
    assert not torch.isfinite(out[0]).all()
    assert torch.isfinite(out[1:]).all()
    assert torch.equal(out[1:], layer.forward(x[1:].contiguous())[0])


@pytest.mark.parametrize("live", [2, 6])
def test_a_training_step_is_captured_and_repeats_bit_for_bit(live):
    """Forward and backward in a graph, which a wait for the GPU would break; replays follow new rows."""
    rows = 200
    layer, x = masked_layer(rows, live=live)
    gen = torch.Generator(device="cuda").manual_seed(6)
    if live == 2:
        layer.router[live:] = -1e30  # (of no row's choice beside the others; finite, so the gradient of x is)
    dout = torch.randn(rows, layer.width, generator=gen, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            layer.backward(dout, layer.forward(x)[1])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, saved = layer.forward(x)
        grads = layer.backward(dout, saved)
    for scale in (1.0, 0.5):
        x.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        no_device_error()
        first = [t.clone() for t in (out,) + grads]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (out,) + grads))
        want = layer.forward(x)
        assert torch.equal(first[0], want[0])
        for got, ref in zip(first[1:], layer.backward(dout, want[1])):
            assert torch.isfinite(got).all() and torch.equal(got, ref)


def test_gradients_of_rows_with_missing_choices():
    """Two of three choices: the gradients are those of a layer of two choices of the live experts.  The weights differ only
    in rounding (the same softmax over two logits); what is stored in bf16 is off by the same steps."""
    rows = 60
    layer, x = masked_layer(rows, experts=4, top=3, live=2)
    two = expert_layer.ExpertLayer(64, 128, 2, 2, rows)
    two.router, two.up, two.down = layer.router[:2].clone(), layer.up[:2].clone(), layer.down[:2].clone()
    dout = torch.randn(rows, 64, device="cuda").bfloat16()
    out, saved = layer.forward(x)
    ref, ref_saved = two.forward(x)
    assert torch.equal(saved[2].ids[:, :2], ref_saved[2].ids)
    layer.router[2:] = 0.0  # (the backward product with the router: 0 * -inf would be NaN; their dlogits are 0)
    _, drouter, dup, ddown = layer.backward(dout, saved)
    _, drouter2, dup2, ddown2 = two.backward(dout, ref_saved)
    dx, dx2 = layer.backward(dout, saved)[0], two.backward(dout, ref_saved)[0]
    no_device_error()
    assert not dup[2:].any() and not ddown[2:].any() and not drouter[2:].any()
    for a, b in ((out, ref), (dx, dx2), (drouter[:2], drouter2), (dup[:2], dup2), (ddown[:2], ddown2)):
        off = float((a.double() - b.double()).norm() / b.double().norm())
        assert off <= 2 * 8 * 2.0 ** -9, off
