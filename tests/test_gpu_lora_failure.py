"""Failure detection of the adapters' products: a ring fill that never comes makes the waits run out, the kernel records it
and returns, and the next call, or the next replay of the captured one, is right."""
import numpy as np
import pytest

from ragged_helpers import G, R, lora_ref, no_device_error, require_gpu, small_ints, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# the way, rows, n, k, rank, adapters: beside the projection (whole and split tiles), and on the tensor cores (whole tiles,
# and one row tile, split), there with an adapter's K block in every place but the first of a tile
CASES = {
    "beside": (R.LORA_BESIDE, 40, 264, 1096, 16, 5),
    "beside, split": (R.LORA_BESIDE, 20, 264, 8200, 16, 5),
    "tensor cores": (R.LORA_TENSOR_CORES, 500, 6000, 584, 72, 60),
    "tensor cores, split": (R.LORA_TENSOR_CORES, 256, 6000, 648, 128, 60),
}


@pytest.mark.parametrize("name", sorted(CASES))
@pytest.mark.parametrize("skip", [0, 1, 3])
def test_starved_wait_reports_timeout_and_recovers(name, skip):
    way, rows, n, k, rank, adapters = CASES[name]
    assert R.gemm_lora_way(rows, n, k, rank, adapters) == way
    rng = np.random.default_rng(skip)
    half = torch.float16
    x, w = small_ints(rng, (rows, k), half, 1), small_ints(rng, (n, k), half, 1)
    a, b = small_ints(rng, (adapters, rank, k), half, 1), small_ints(rng, (adapters, n, rank), half, 1)
    a[torch.from_numpy(rng.random((adapters, rank, k)) < 1 - 48.0 / k)] = 0
    ids = torch.from_numpy((np.arange(rows) % (adapters + 1) - 1).astype(np.int32))
    ref = lora_ref(x, w, a, b, ids, None).half()
    dev = [t.cuda() for t in (x, w, a, b, ids)]
    y = torch.zeros((rows, n), dtype=half, device="cuda")
    ws = torch.full((R.gemm_lora_workspace_size(rows, n, k, rank, adapters),), 0xA5, dtype=torch.uint8, device="cuda")
    no_device_error()
    assert R.gemm_lora_stall_test(*dev, y, ws, skip, 1 << 24) == G.GEMM_OK
    st, code = G.gemm_f16_take_device_error()
    assert st == G.GEMM_ERR_TIMEOUT and (code & 0xFF) in range(1, 12)
    assert torch.equal(R.gemm_lora_nt(*dev, workspace=ws).cpu(), ref)
    no_device_error()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert R.gemm_lora_stall_test(*dev, y, ws, skip, 1 << 24) == G.GEMM_OK
    graph.replay()  # aborted
    torch.cuda.synchronize()
    dev[0].copy_(-x)
    for _ in range(2):  # the error word is set: nothing is skipped
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), -ref)
    assert G.gemm_f16_take_device_error()[0] == G.GEMM_ERR_TIMEOUT
    no_device_error()


def test_refusals():
    z = torch.zeros(0, dtype=torch.float16, device="cuda")
    x, a, b = z.view(0, 8), z.view(0, 8, 8), z.view(0, 8, 8)
    w = torch.zeros((8, 8), dtype=torch.float16, device="cuda")
    ids = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert R.gemm_lora_stall_test(x, w, a, b, ids, z.view(0, 8), None, 0, 0) == G.GEMM_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        R.gemm_lora_stall_test(x, w, a, b, ids, z.view(0, 8)[:, :4], None, 0, 1)
