"""Host-side checks of the products with an epilogue that need no GPU: exports, limits, and every argument validated before a
device is touched."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

from dense_fp16_gemm_03_gb300 import build as pkg_build  # noqa: E402
from dense_fp16_gemm_03_gb300 import gemm as G  # noqa: E402
from dense_fp16_gemm_03_gb300 import linear as LN  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20       # an aligned address that is never dereferenced
INVALID, ALIGN, SHAPE = G.GEMM_ERR_INVALID_ARG, G.GEMM_ERR_ALIGNMENT, G.GEMM_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def L():
    pkg_build.build()
    return LN.lib()


def _header():
    return open(os.path.join(ROOT, "include", "gemm_linear.h")).read()


def test_every_declared_symbol_is_exported(L):
    names = set(re.findall(r"\b(gemm_linear_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", _header(), flags=re.S)))
    assert names == set(LN.EXPORTED)
    for name in names:
        assert hasattr(L, name)


def test_activations_match_the_header():
    found = {name.lower(): int(v) for name, v in re.findall(r"GEMM_ACT_(\w+) = (\d+)", _header())}
    assert found == {a: v for a, v in LN.ACTS.items() if a is not None}


def nt(L, dtype=0, act=3, groups=1, rows=10, n=64, k=72, offsets=None, x=P, w=P, bias=P, residual=P, z=P, y=P):
    return L.gemm_linear_nt(dtype, act, groups, rows, n, k, offsets, x, w, bias, residual, z, y, None, 0, None)


def nn(L, dtype=0, act=3, groups=1, rows=10, n=64, k=72, offsets=None, dy=P, w=P, z=P, dx=P, dbias=P):
    return L.gemm_linear_nn(dtype, act, groups, rows, n, k, offsets, dy, w, z, dx, dbias, None, 0, None)


def grad(L, dtype=0, act=3, groups=1, rows=10, n=64, offsets=None, dy=P, z=P, dz=P, dbias=P):
    return L.gemm_linear_grad(dtype, act, groups, rows, n, offsets, dy, z, dz, dbias, None, 0, None)


CALLS = {"nt": nt, "nn": nn, "grad": grad}
COMMON = [
    ({"groups": 0}, INVALID), ({"groups": -1}, INVALID), ({"rows": -1}, INVALID), ({"n": -8}, INVALID), ({"groups": 2}, INVALID),
    ({"groups": 1025, "offsets": P}, SHAPE), ({"rows": 1 << 31}, SHAPE), ({"n": 12}, SHAPE), ({"n": 1 << 31}, SHAPE),
    ({"dtype": 2}, INVALID), ({"dtype": -1}, INVALID), ({"act": 6}, INVALID), ({"act": -1}, INVALID), ({"offsets": P + 2}, ALIGN),
]
OWN = {
    "nt": [({"k": 71}, SHAPE), ({"k": -8}, INVALID), ({"k": 0}, SHAPE), ({"x": None}, INVALID), ({"w": None}, INVALID), ({"y": None}, INVALID),
           ({"x": P + 8}, ALIGN), ({"w": P + 2}, ALIGN), ({"y": P + 4}, ALIGN), ({"bias": P + 2}, ALIGN), ({"residual": P + 8}, ALIGN),
           ({"z": P + 8}, ALIGN)],
    "nn": [({"k": 71}, SHAPE), ({"n": 0}, SHAPE), ({"dy": None}, INVALID), ({"w": None}, INVALID), ({"z": None}, INVALID),
           ({"dx": None}, INVALID), ({"dy": P + 8}, ALIGN), ({"z": P + 8}, ALIGN), ({"dx": P + 2}, ALIGN), ({"dbias": P + 4}, ALIGN)],
    "grad": [({"dy": None}, INVALID), ({"z": None}, INVALID), ({"dz": None}, INVALID), ({"dy": P + 8}, ALIGN), ({"z": P + 8}, ALIGN),
             ({"dz": P + 2}, ALIGN), ({"dbias": P + 4}, ALIGN)],
}


@pytest.mark.parametrize("op,change,status", [(op, c, s) for op in CALLS for c, s in COMMON + OWN[op]])
def test_refusals(L, op, change, status):
    assert CALLS[op](L, **change) == status


@pytest.mark.parametrize("op", sorted(CALLS))
def test_nothing_to_do(L, op):
    none = {"nt": {"x": None, "w": None, "y": None, "bias": None, "residual": None, "z": None},
            "nn": {"dy": None, "w": None, "z": None, "dx": None, "dbias": None},
            "grad": {"dy": None, "z": None, "dz": None, "dbias": None}}[op]
    assert CALLS[op](L, rows=0, **none) == G.GEMM_OK


def test_workspace_size_refusals(L):
    import ctypes
    b = ctypes.c_size_t()
    for args, status in (((0, 10, 64, 64), INVALID), ((1, -1, 64, 64), INVALID), ((1025, 10, 64, 64), SHAPE), ((1, 10, 60, 64), SHAPE)):
        assert L.gemm_linear_workspace_size(*args, ctypes.byref(b)) == status
    assert L.gemm_linear_workspace_size(1, 10, 64, 64, None) == INVALID


def test_stall_hook_refusals(L):
    args = (0, 0, 1, 10, 64, 72, None, P, P, P, P, None, None, 0, 0)
    assert L.gemm_linear_stall_test(2, *args, 1000, None) == INVALID
    assert L.gemm_linear_stall_test(-1, *args, 1000, None) == INVALID
    assert L.gemm_linear_stall_test(0, *args, 0, None) == INVALID


def test_binding_refuses_before_the_call(L):
    x, w = torch.zeros((4, 8), dtype=torch.float16), torch.zeros((16, 8), dtype=torch.float16)
    with pytest.raises(ValueError):
        LN.gemm_linear_nt(x, w)  # host tensors
    with pytest.raises(ValueError):
        LN.gemm_linear_nt(x, w, act="tanh")
    with pytest.raises(ValueError):
        LN.gemm_linear_nn(x, w, act="gelu")
    with pytest.raises(ValueError):
        LN.gemm_linear_grad(x, act="gelu")
