"""A binding that was built for another PyTorch or Python is built again, and refused where it is loaded all the same."""
import os

import pytest

from dense_fp16_gemm_03_gb300 import _binding
from dense_fp16_gemm_03_gb300 import build as B
from test_build_host import tree  # noqa: F401


@pytest.fixture
def built(tree, monkeypatch):  # noqa: F811
    if B.binding_lacks():
        pytest.skip("no binding here: %s is missing" % B.binding_lacks())
    B.build()
    monkeypatch.setattr(_binding, "_native", None)
    return tree


def test_the_target_names_this_pytorch():
    torch = pytest.importorskip("torch")
    assert torch.__version__ in B.binding_target()


def test_built_again_for_another_version(built, monkeypatch):
    first = B.binding_built_for()
    assert first == B.binding_target() and not B._stale_binding()
    monkeypatch.setattr(B, "binding_target", lambda: "PyTorch '0.0', other")
    assert B._stale_binding()
    with pytest.raises(RuntimeError, match="was built for PyTorch"):
        _binding.native()
    os.utime(B.BINDING, (1, 1))
    B.build()
    assert os.path.getmtime(B.BINDING) > 1 and B.binding_built_for() == "PyTorch '0.0', other" and not B._stale_binding()


def test_a_binding_without_a_note_is_not_loaded(built):
    os.remove(B.BINDING + ".for")
    with pytest.raises(RuntimeError, match="another version"):
        _binding.native()
    B.build()
    assert B.binding_built_for() == B.binding_target()
    assert not [f for f in os.listdir(B.OUT_DIR) if ".tmp" in f]
