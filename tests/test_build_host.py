"""The build on machines that lack what the Python binding needs, or where it does not compile: the C library is built all the
same.  The sources are stand-ins of a line each."""
import ctypes
import os
import subprocess

import pytest

from dense_fp16_gemm_03_gb300 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build.py with sources and outputs of its own; the binding's source compiles without any headers."""
    if not os.path.exists(B.NVCC):
        pytest.skip("no nvcc")
    source, binding = tmp_path / "lib.cu", tmp_path / "binding.cpp"
    source.write_text('extern "C" int answer() { return 42; }\n')
    binding.write_text('extern "C" int bound() { return 7; }\n')
    out = tmp_path / "_build"
    for name, value in {"OUT_DIR": str(out), "LIB": str(out / "libgemm_f16.so"), "BINDING": str(out / "gemm_binding.so"),
                        "SOURCES": [str(source)], "DEPS": [str(source)], "BINDING_SOURCE": str(binding)}.items():
        monkeypatch.setattr(B, name, value)
    return tmp_path


def answers():
    return ctypes.CDLL(B.LIB).answer() == 42


def test_both(tree):
    if B.binding_lacks():
        pytest.skip("no binding here: %s is missing" % B.binding_lacks())
    assert B.build() == B.LIB and answers() and os.path.exists(B.BINDING)
    first = os.path.getmtime(B.BINDING)
    B.build()
    assert os.path.getmtime(B.BINDING) == first
    assert not [f for f in os.listdir(B.OUT_DIR) if ".tmp" in f]


def test_a_binding_that_does_not_compile_leaves_the_library(tree):
    if B.binding_lacks():
        pytest.skip("no binding here: %s is missing" % B.binding_lacks())
    with open(B.BINDING_SOURCE, "w") as f:
        f.write("this is no C++\n")
    for _ in range(2):  # and says so again
        with pytest.raises(subprocess.CalledProcessError):
            B.build()
        assert answers() and not os.path.exists(B.BINDING)


def test_a_library_that_does_not_compile(tree):
    with open(B.SOURCES[0], "w") as f:
        f.write("this is no C++\n")
    with pytest.raises(subprocess.CalledProcessError):
        B.build()
    assert not os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


@pytest.mark.parametrize("what", ["PyTorch", "CUDA libraries of PyTorch", "Python.h", "compiler"])
def test_what_the_binding_lacks(tree, what, monkeypatch, capfd):
    """A clean end with the library; a binding of earlier sources is taken away."""
    if what == "PyTorch":
        monkeypatch.setattr(B, "_torch_dir", lambda: None)
    elif what == "CUDA libraries of PyTorch":
        real = os.path.exists
        monkeypatch.setattr(B.os.path, "exists", lambda f: not str(f).endswith("libc10_cuda.so") and real(f))
    elif what == "Python.h":
        monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": str(tree)})
    else:
        monkeypatch.setattr(B, "CXX", "no-such-compiler")
    os.makedirs(B.OUT_DIR)
    with open(B.BINDING, "w") as f:
        f.write("old")
    os.utime(B.BINDING, (1, 1))
    assert B.binding_lacks() is not None
    assert B.build() == B.LIB and answers() and not os.path.exists(B.BINDING)
    assert "left out" in capfd.readouterr().err
    assert B.build() == B.LIB


def test_what_is_missing_is_named_at_the_call(monkeypatch, tree):
    from dense_fp16_gemm_03_gb300 import _binding
    monkeypatch.setattr(_binding, "_native", None)
    monkeypatch.setattr(B, "binding_lacks", lambda: "Python.h")
    with pytest.raises(RuntimeError, match="Python.h is missing"):
        _binding.native()
