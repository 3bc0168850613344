"""The README's example of the ragged products and the router runs as it stands, above the router's 64 rows of one block."""
import os
import re

import pytest

from ragged_helpers import no_device_error, require_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [20, 100])
def test_example_runs(rows):
    require_gpu()
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    code = [c for c in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "gemm_route_topk" in c]
    assert len(code) == 1
    experts, n, k, rank, adapters, half = 16, 72, 136, 16, 4, torch.float16

    def rand(*shape, dtype=half):
        return torch.randn(*shape, device="cuda").to(dtype)

    names = {"torch": torch, "rows": rows, "experts": experts, "n": n, "k": k, "rank": rank, "adapters": adapters,
             "logits": rand(rows, experts, dtype=torch.float32), "tokens": rand(rows, k), "w": rand(experts, n, k),
             "dy": rand(8 * rows, n), "dweights": rand(rows, 8, dtype=torch.float32), "h": rand(rows, k), "shared": rand(n, k),
             "a": rand(adapters, rank, k), "b": rand(adapters, n, rank),
             "ids": torch.arange(rows, dtype=torch.int32, device="cuda") % (adapters + 1) - 1,
             "scale": torch.ones(adapters, device="cuda")}
    exec(code[0], names)
    no_device_error()
    assert names["dx"].shape == (8 * rows, k) and names["dw"].shape == (experts, n, k)
    assert names["dlogits"].shape == (rows, experts) and names["y"].shape == (rows, n)
