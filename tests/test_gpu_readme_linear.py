"""The README's example of the products with an epilogue and the scored router runs as it stands."""
import os
import re

import pytest

from ragged_helpers import no_device_error, require_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [20, 100])
def test_example_runs(rows):
    require_gpu()
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    code = [c for c in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "gemm_linear_nt" in c]
    assert len(code) == 1
    experts, n, k = 64, 72, 136

    def rand(*shape, dtype=torch.float16):
        return torch.randn(*shape, device="cuda").to(dtype)

    f32 = torch.float32
    names = {"torch": torch, "experts": experts, "n": n, "k": k, "x": rand(rows, k), "w": rand(n, k), "bias": rand(n), "dy": rand(rows, n),
             "z_below": rand(rows, k), "logits": rand(rows, experts, dtype=f32), "balance": rand(experts, dtype=f32) / 16,
             "dweights": rand(rows, 8, dtype=f32), "experts_w": rand(experts, n, k)}
    exec(code[0], names)
    no_device_error()
    assert names["y"].shape == names["dz"].shape == (rows, n) and names["dx"].shape == (rows, k)
    assert names["dbias"].shape == (n,) and names["dbelow"].shape == (k,)
    assert names["dlogits"].shape == (rows, experts) and names["h"].shape == names["hz"].shape == (8 * rows, n)
