"""The expert layer against the same layer written in 64-bit torch with automatic differentiation: the operators
together, forward and backward, with rows that have fewer experts than choices."""
import numpy as np
import pytest

from ragged_helpers import no_device_error, require_gpu, torch

from dense_fp16_gemm_03_gb300 import expert_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("rows,width,hidden,experts,top", [(1, 64, 128, 8, 2), (37, 72, 136, 8, 3), (700, 128, 264, 20, 4)])
def test_layer_and_its_gradients(rows, width, hidden, experts, top):
    """Every stored intermediate is rounded to bf16 (half a step 2^-9): five of them on the longest way (h, a, y, da, dh,
    with the square doubling h's), so an entry is off by at most some 8 * 2^-9 of the sum of its terms' magnitudes; the
    sums' norms are bounded by 8 * 2^-9 = 0.016 of the gradient's norm times the terms' spread, taken as 2."""
    layer = expert_layer.ExpertLayer(width, hidden, experts, top, rows)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=gen, device="cuda").bfloat16()
    dout = torch.randn(rows, width, generator=gen, device="cuda").bfloat16()
    out, saved = layer.forward(x)
    grads = layer.backward(dout, saved)
    no_device_error()

    leaf = [t.double().requires_grad_() for t in (x, layer.router, layer.up, layer.down)]
    xd, router, up, down = leaf
    p = torch.softmax(xd @ router.T, 1)
    ids = saved[2].ids.long()
    w = torch.gather(p, 1, ids)
    w = w / w.sum(1, keepdim=True)
    h = torch.einsum("tk,tjnk->tjn", xd, up[ids])
    y = torch.einsum("tjn,tjkn->tjk", torch.relu(h).square(), down[ids])
    want = (w[:, :, None] * y).sum(1)
    want.backward(dout.double())
    for name, got, ref in [("out", out, want.detach())] + [(n, g, t.grad) for n, g, t in zip(("x", "router", "up", "down"), grads, leaf)]:
        off = float((got.double() - ref).norm() / ref.norm())
        assert off <= 2 * 8 * 2.0 ** -9, (name, off)


def test_two_streams_with_workspaces_of_their_own():
    """Split products that overlap on the GPU wait only for workers before them, so neither holds the other up."""
    from dense_fp16_gemm_03_gb300 import ragged as R
    rng = np.random.default_rng(3)
    n, k, rows = 264, 4104, 24
    w = torch.from_numpy(rng.integers(-8, 9, size=(6, n, k)).astype(np.float32) / 8).half().cuda()
    x = torch.from_numpy(rng.integers(-8, 9, size=(rows, k)).astype(np.float32) / 8).half().cuda()
    offsets = torch.tensor([0, 5, 5, 9, 20, 23, 24], dtype=torch.int32, device="cuda")
    size = R.gemm_grouped_workspace_size(6, rows, n, k)
    want = R.gemm_grouped_nt(x, w, offsets)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(want) for _ in streams]
    spaces = [torch.zeros(max(1, size), dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(50):
        for s, o, ws in zip(streams, outs, spaces):
            R.gemm_grouped_nt(x, w, offsets, y=o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    no_device_error()
    assert all(torch.equal(o, want) for o in outs)


def test_a_workspace_for_the_most_rows_serves_fewer():
    """Sizes never fall with the rows, and calls of fewer rows take the larger buffer, whichever kernels they run."""
    from dense_fp16_gemm_03_gb300 import ragged as R
    steps = [1, 2, 63, 64, 65, 100, 256, 257, 300, 512, 1000, 1024, 2048, 5000, 20000, 66000]
    for n, k, rank, adapters in [(64, 72, 8, 2), (4096, 4096, 16, 64), (8192, 4096, 64, 16), (1000, 4104, 128, 300)]:
        sizes = [R.gemm_lora_workspace_size(r, n, k, rank, adapters) for r in steps]
        assert sizes == sorted(sizes)
        for groups in (1, 8, 1000):
            sizes = [R.gemm_grouped_workspace_size(groups, r, n, k) for r in steps]
            assert sizes == sorted(sizes)
        sizes = [R.gemm_route_workspace_size(r, 128, 8) for r in steps]
        assert sizes == sorted(sizes)
    n, k, rank, adapters, most = 264, 4104, 16, 40, 700
    ws = torch.zeros(R.gemm_lora_workspace_size(most, n, k, rank, adapters), dtype=torch.uint8, device="cuda")
    gs = torch.zeros(R.gemm_grouped_workspace_size(3, most, n, k), dtype=torch.uint8, device="cuda")
    w = torch.zeros((n, k), dtype=torch.float16, device="cuda")
    a, b = torch.zeros((adapters, rank, k), device="cuda").half(), torch.zeros((adapters, n, rank), device="cuda").half()
    wg = torch.ones((3, n, k), device="cuda").half()
    for rows in range(1, most + 1, 37):
        x = torch.ones((rows, k), device="cuda").half()
        ids = torch.arange(rows, dtype=torch.int32, device="cuda") % adapters
        assert not R.gemm_lora_nt(x, w, a, b, ids, workspace=ws).any()
        offsets = torch.tensor([0, rows // 3, rows // 2, rows], dtype=torch.int32, device="cuda")
        assert (R.gemm_grouped_nt(x, wg, offsets, workspace=gs) == k).all()
        dy = torch.ones((rows, n), device="cuda").half()
        assert (R.gemm_grouped_nn(dy, wg, offsets, workspace=gs) == n).all()
        dw = R.gemm_grouped_tn(dy, x, offsets, workspace=gs)
        assert [float(dw[g].min()) for g in range(3)] == [float(v) for v in torch.diff(offsets).tolist()]
    no_device_error()
