"""Replays of a captured launch, all of one stamp, after one of them was aborted: no partial sum's flag is left over, so a
replay never adds a sum that an earlier one published."""
import numpy as np
import pytest

from ragged_helpers import G, R, eighths, grouped_operands, grouped_ref, no_device_error, offsets_of, require_gpu, torch

pytestmark = pytest.mark.gpu

# sizes at which single CTAs' tiles, and CTA pairs', are split over K
SPLIT = {"single CTAs": ([3, 4], 264, 8200), "pairs": ([700], 2000, 8192), "pairs, two groups": ([290, 300], 1032, 8200)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("name", sorted(SPLIT))
@pytest.mark.parametrize("skip", [0, 3])
def test_replays_after_an_aborted_one(mode, name, skip):
    """The hook leaves a fill undone while the error word is clear: of the replays, the first is aborted and those before
    the error is taken run through."""
    op = ("nt", "nn")[mode]
    rng = np.random.default_rng(skip)
    sizes, other, long = SPLIT[name]
    n, k = (other, long) if op == "nt" else (long, other)
    first, w = grouped_operands(op, rng, sizes, n, k, torch.float16)
    offsets = offsets_of(sizes)
    groups = len(sizes)
    fd, wd, od = first.cuda(), w.cuda(), offsets.cuda()
    out = torch.zeros((sum(sizes), n if op == "nt" else k), dtype=torch.float16, device="cuda")
    ws = torch.full((R.gemm_grouped_workspace_size(groups, sum(sizes), n, k),), 0x5A, dtype=torch.uint8, device="cuda")
    call = R.gemm_grouped_nt if op == "nt" else R.gemm_grouped_nn
    call(fd, wd, od, workspace=ws)
    no_device_error()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert R.gemm_grouped_stall_test(mode, fd, wd, od, out, ws, skip, 1 << 24) == G.GEMM_OK
    for _ in range(2):
        fd.copy_(eighths(rng, tuple(first.shape), torch.float16))
        graph.replay()  # aborted
        torch.cuda.synchronize()
        for _ in range(2):
            x = eighths(rng, tuple(first.shape), torch.float16)
            fd.copy_(x)
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out.cpu(), grouped_ref(op, x, w, offsets, groups).half())
        st, code = G.gemm_f16_take_device_error()
        assert st == G.GEMM_ERR_TIMEOUT and (code & 0xFF) in range(1, 12)
    assert torch.equal(call(fd, wd, od, workspace=ws).cpu(), grouped_ref(op, x, w, offsets, groups).half())
    no_device_error()
