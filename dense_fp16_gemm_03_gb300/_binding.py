"""Loads the native part of the Python binding (csrc/binding.cpp, built by build.py)."""
import importlib.machinery
import importlib.util
import os

from . import build as _build
from . import gemm as _gemm

_native = None


def native():
    """The module gemm_binding; raises if it is not built."""
    global _native
    if _native is None:
        if not os.path.exists(_build.BINDING):
            lacks = _build.binding_lacks()
            raise RuntimeError("gemm_binding.so is not built (%s); %srun __graft_entry__.build()" % (
                _build.BINDING, "%s is missing here: install it and " % lacks if lacks else ""))
        if _build.binding_built_for() != _build.binding_target():
            raise RuntimeError("gemm_binding.so was built for %s, and this is %s; run __graft_entry__.build()" % (
                _build.binding_built_for() or "another version", _build.binding_target()))
        _gemm._tm()   # PyTorch's libraries first, and the product's
        _gemm.lib()
        loader = importlib.machinery.ExtensionFileLoader("gemm_binding", _build.BINDING)
        module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("gemm_binding", _build.BINDING, loader=loader))
        loader.exec_module(module)
        _native = module
    return _native


def checked(result, where):
    """What a call gave, or its refusal as an error."""
    if type(result) is int:
        raise _gemm.GemmError(result, where)
    return result
