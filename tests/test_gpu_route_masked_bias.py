"""A bias of -infinity masks an expert whatever its score is: also where that is NaN, by its own logit or, through a softmax, by
another one's."""
import pytest

from ragged_helpers import require_gpu, torch
from test_gpu_route_scored import check, draw, draw_bias

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [8, 70])
@pytest.mark.parametrize("experts,top", [(24, 8), (256, 32), (1024, 32), (40, 40 // 2)])
def test_masked_experts_of_rows_that_hold_nan(experts, top, rows, kind, score, renorm):
    z = draw(rows, experts, kind, seed=experts)
    masked = torch.arange(experts) % 3 != 1
    bias = torch.where(masked, -INF, draw_bias(experts, 5))
    z[0, 0], z[1, 1], z[2, 2], z[3, 4] = NAN, NAN, INF, INF       # masked, not masked
    z[4] = NAN
    z[5, masked] = NAN
    z[6, ~masked] = -INF
    z[6, masked] = NAN
    z[7, ::2] = -INF
    z[7, 1::4] = NAN
    for groups, top_groups, group_top in ((1, 1, 2), (4, 4, 1), (8, 8, 2), (4, 2, 2), (8, 3, 1)):
        most = min(top, top_groups * (experts // groups))
        got, want = check(z, most, score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top, renorm=renorm)
        ids = got.ids.cpu().long()
        assert not masked[ids.clamp(min=0)][ids >= 0].any()
        check(z, most, score=score, bias=torch.where(torch.arange(experts) == 1, NAN, bias), groups=groups, top_groups=top_groups,
              group_top=group_top, renorm=renorm)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_every_expert_masked_in_rows_that_hold_nan(score):
    z = torch.full((70, 16), NAN)
    z[1] = INF
    got, _ = check(z, 4, score=score, bias=torch.full((16,), -INF), groups=4, top_groups=2)
    assert (got.ids == -1).all() and not got.weights.any() and not got.offsets.any()
