"""The last of as many choices as a row may have, beside the first expert that is not chosen: scores closer than a key holds, with
all others well apart, so that nothing but that border tells of a close call."""
import numpy as np
import pytest

from ragged_helpers import R, require_gpu, torch
from test_gpu_route_scored import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def border(rows, experts, top, seed, equal=False):
    """fp32 logits, in every row `top` - 1 clear choices and two at 0.5 and the next number, the larger one behind the other."""
    rng = np.random.default_rng(seed)
    two = np.float32([0.5, 0.5 if equal else np.nextafter(np.float32(0.5), np.float32(1))])
    z = np.empty((rows, experts), dtype=np.float32)
    for t in range(rows):
        at = rng.permutation(experts)
        low, high = sorted(at[:2])
        z[t, at[2:top + 1]] = np.linspace(1, 4, top - 1)
        z[t, at[top + 1:]] = np.linspace(-6, -1, experts - top - 1)
        z[t, [low, high]] = two
    return torch.from_numpy(z)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("rows", [5, 70])
@pytest.mark.parametrize("experts", [33, 64, 256, 1024])
@pytest.mark.parametrize("top", [31, 32])
def test_border(top, experts, rows, bias, score):
    assert R.MAX_TOP == 32
    b = torch.zeros(experts) if bias else None
    z = border(rows, experts, top, seed=experts + rows)
    check(z, top, score=score, bias=b)
    check(border(rows, experts, top, seed=experts, equal=True), top, score=score, bias=b)
    if experts % 4 == 0:
        check(z, top, score=score, bias=b, groups=4, top_groups=4, group_top=1)


def test_border_with_masks_and_infinities():
    """A row that holds what is no number, or what cannot be chosen, has the same border."""
    z = border(70, 256, 32, seed=3)
    away = z < 0
    z[::3] = torch.where(away[::3], -float("inf"), z[::3])
    z[1, int(z[1].argmin())] = float("nan")
    z[2, int(z[2].argmax())] = float("inf")
    for b in (None, torch.zeros(256)):
        check(z, 32, bias=b)
        check(z, 32, score="softmax", bias=b)


def test_many_random_rows():
    """Random rows have such a border by chance: 1024 experts, the 32 best."""
    rng = np.random.default_rng(4)
    z = torch.from_numpy((1.5 * rng.standard_normal((20000, 1024))).astype(np.float32))
    bias = torch.from_numpy((0.05 * rng.standard_normal(1024)).astype(np.float32))
    for b in (None, bias):
        ws = torch.empty(R.gemm_route_workspace_size(20000, 1024, 32), dtype=torch.uint8, device="cuda")
        got = R.gemm_route_scored(z.cuda(), 32, bias=None if b is None else b.cuda(), workspace=ws).ids.cpu().long()
        c = z.double() if b is None else torch.sigmoid(z.double()) + b.double()
        want = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :32]
        assert torch.equal(got, want)
