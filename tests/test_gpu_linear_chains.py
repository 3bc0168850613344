"""Column sums of contractions that are cut into few chains, of which the first is a large part."""
import pytest

from linear_helpers import KINDS, L, buffer, no_device_error, require_gpu, torch

pytestmark = pytest.mark.gpu

ROWS, COLS = 4096, 5120  # 320 tiles of 256 x 256: most of them whole, not split between workers


def mean_error(kind, blocks):
    """Relative error of dbias, the mean over all columns.  All terms are positive: what the tensor cores cut off adds up, while
    the roundings to nearest of all other sums cancel in the mean."""
    gen = torch.Generator(device="cuda").manual_seed(blocks)
    n = 64 * blocks
    dy = (torch.rand(ROWS, n, generator=gen, device="cuda") + 0.5).to(kind)
    w = (torch.rand(n, COLS, generator=gen, device="cuda") / 64 + 1 / 128).to(kind)
    _, db = L.gemm_linear_nn(dy, w, bias_grad=True, workspace=buffer(1, ROWS, n, COLS))
    no_device_error()
    want = dy.double().sum(0) @ w.double()
    return ((db.double() - want) / want).mean().item()


@pytest.mark.parametrize("blocks", [14, 20, 21, 29, 30, 39, 40, 64])
@pytest.mark.parametrize("kind", sorted(KINDS))
def test_no_more_than_the_longest_chain(kind, blocks):
    """In a chain that grows evenly each step cuts an even share off, so what is lost, relative to the chain, goes with its length;
    relative to the sum it is at most that of the longest chain, 20 K blocks, 20/13 of what a contraction of 13 blocks, one
    chain, loses (one chain of 39 would lose three times that).  2^-23 for what the roundings to nearest leave of a mean."""
    require_gpu()
    one = abs(mean_error(KINDS[kind], 13))
    assert one < 1e-5
    assert abs(mean_error(KINDS[kind], blocks)) <= 20 / 13 * one + 2.0 ** -23
