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
