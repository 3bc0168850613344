"""Host-side checks of the ragged products and the router that need no GPU: the library exports what the header
declares, and every argument is validated before a device is touched."""
import ctypes
import os
import re

import pytest

from dense_fp16_gemm_03_gb300 import build as pkg_build
from dense_fp16_gemm_03_gb300 import gemm as G
from dense_fp16_gemm_03_gb300 import ragged as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20       # an aligned address that is never dereferenced
INVALID, ALIGN, SHAPE = G.GEMM_ERR_INVALID_ARG, G.GEMM_ERR_ALIGNMENT, G.GEMM_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def L():
    pkg_build.build()
    return R.lib()


def test_every_declared_symbol_is_exported(L):
    text = open(os.path.join(ROOT, "include", "gemm_ragged.h")).read()
    names = set(re.findall(r"\b(gemm_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(R.EXPORTED)
    for name in names:
        assert hasattr(L, name)


def test_limits_match_the_header():
    text = open(os.path.join(ROOT, "include", "gemm_ragged.h")).read()
    for name, value in (("GEMM_GROUPED_MAX_GROUPS", R.MAX_GROUPS), ("GEMM_LORA_MAX_RANK", R.MAX_RANK),
                        ("GEMM_ROUTE_MAX_EXPERTS", R.MAX_EXPERTS), ("GEMM_ROUTE_MAX_TOP", R.MAX_TOP)):
        assert int(re.search(r"#define %s (\d+)" % name, text).group(1)) == value
    for name, value in (("F16", R.DTYPE_F16), ("BF16", R.DTYPE_BF16), ("F32", R.DTYPE_F32)):
        assert int(re.search(r"GEMM_DTYPE_%s = (\d+)" % name, text).group(1)) == value


def grouped(L, op="nt", dtype=0, out=0, groups=4, rows=10, n=64, k=72, offsets=P, first=P, second=P, result=P):
    if op == "tn":
        return L.gemm_grouped_tn(dtype, out, groups, rows, n, k, offsets, first, second, result, None, 0, None)
    f = L.gemm_grouped_nt if op == "nt" else L.gemm_grouped_nn
    return f(dtype, groups, rows, n, k, offsets, first, second, result, None, 0, None)


@pytest.mark.parametrize("op", ["nt", "nn", "tn"])
@pytest.mark.parametrize("change,status", [
    ({"groups": -1}, INVALID), ({"rows": -1}, INVALID), ({"n": -8}, INVALID), ({"k": -8}, INVALID),
    ({"groups": 1025}, SHAPE), ({"rows": 1 << 31}, SHAPE), ({"n": 12}, SHAPE), ({"k": 71}, SHAPE), ({"n": 1 << 31}, SHAPE),
    ({"dtype": 2}, INVALID), ({"dtype": 7}, INVALID), ({"dtype": -1}, INVALID),
    ({"offsets": None}, INVALID), ({"first": None}, INVALID), ({"second": None}, INVALID), ({"result": None}, INVALID),
    ({"offsets": P + 2}, ALIGN), ({"first": P + 8}, ALIGN), ({"second": P + 2}, ALIGN), ({"result": P + 4}, ALIGN),
])
def test_grouped_refusals(L, op, change, status):
    assert grouped(L, op, **change) == status


def test_grouped_tn_output_types(L):
    assert grouped(L, "tn", dtype=0, out=1) == INVALID
    assert grouped(L, "tn", dtype=1, out=0) == INVALID
    assert grouped(L, "tn", dtype=1, out=3) == INVALID


def test_grouped_without_output_is_a_no_op(L):
    for op in ("nt", "nn"):
        assert grouped(L, op, rows=0, offsets=None, first=None, second=None, result=None) == G.GEMM_OK
    assert grouped(L, "nt", n=0, second=None, result=None) == G.GEMM_OK
    assert grouped(L, "nn", k=0, second=None, result=None) == G.GEMM_OK
    assert grouped(L, "tn", groups=0, result=None) == G.GEMM_OK
    assert grouped(L, "tn", n=0, first=None, result=None) == G.GEMM_OK


def lora(L, dtype=0, rows=10, n=64, k=72, rank=16, adapters=3, x=P, w=P, a=P, b=P, ids=P, scale=P, y=P):
    return L.gemm_lora_nt(dtype, rows, n, k, rank, adapters, x, w, a, b, ids, scale, y, None, 0, None)


@pytest.mark.parametrize("change,status", [
    ({"rows": -1}, INVALID), ({"adapters": -1}, INVALID), ({"rank": -8}, INVALID), ({"dtype": 2}, INVALID),
    ({"rank": 136}, SHAPE), ({"rank": 12}, SHAPE), ({"n": 9}, SHAPE), ({"k": 9}, SHAPE), ({"rows": 1 << 31}, SHAPE),
    ({"x": None}, INVALID), ({"w": None}, INVALID), ({"a": None}, INVALID), ({"b": None}, INVALID), ({"ids": None}, INVALID),
    ({"y": None}, INVALID), ({"x": P + 8}, ALIGN), ({"a": P + 2}, ALIGN), ({"b": P + 2}, ALIGN), ({"scale": P + 2}, ALIGN),
    ({"ids": P + 1}, ALIGN),
])
def test_lora_refusals(L, change, status):
    assert lora(L, **change) == status


def test_lora_without_output_is_a_no_op(L):
    assert lora(L, rows=0, x=None, ids=None, y=None) == G.GEMM_OK
    assert lora(L, n=0, w=None, b=None, y=None) == G.GEMM_OK


def route(L, dtype=2, rows=10, experts=16, top=4, logits=P, ids=P, weights=P, offsets=P, order=P, position=P):
    return L.gemm_route_topk(dtype, rows, experts, top, 1, logits, ids, weights, offsets, order, position, None, 0, None)


@pytest.mark.parametrize("change,status", [
    ({"dtype": 3}, INVALID), ({"rows": -1}, INVALID), ({"experts": 0}, INVALID), ({"top": 0}, INVALID), ({"top": 17}, INVALID),
    ({"experts": 1025}, SHAPE), ({"experts": 64, "top": 33}, SHAPE), ({"rows": 1 << 29}, SHAPE),
    ({"logits": None}, INVALID), ({"ids": None}, INVALID), ({"weights": None}, INVALID), ({"offsets": None}, INVALID),
    ({"order": None}, INVALID), ({"position": None}, INVALID), ({"logits": P + 4}, ALIGN), ({"order": P + 1}, ALIGN),
])
def test_route_refusals(L, change, status):
    assert route(L, **change) == status


@pytest.mark.parametrize("at", range(5))
def test_route_grad_refusals(L, at):
    args = [P] * 5
    args[at] = None
    assert L.gemm_route_topk_grad(2, 10, 16, 4, 1, *args, None) == INVALID
    args[at] = P + 2
    assert L.gemm_route_topk_grad(2, 10, 16, 4, 1, *args, None) == ALIGN
    assert L.gemm_route_topk_grad(2, 0, 16, 4, 1, None, None, None, None, None, None) == G.GEMM_OK


def test_stall_test_refusals(L):
    args = (0, 4, 10, 64, 72, P, P, P, P, None, 0, 0)
    assert L.gemm_grouped_stall_test(3, *args, 1000, None) == INVALID
    assert L.gemm_grouped_stall_test(-1, *args, 1000, None) == INVALID
    assert L.gemm_grouped_stall_test(0, *args, 0, None) == INVALID


def test_workspace_queries_refuse(L):
    b = ctypes.c_size_t()
    assert L.gemm_grouped_workspace_size(1, 1, 8, 8, None) == INVALID
    assert L.gemm_grouped_workspace_size(1, 1, 7, 8, ctypes.byref(b)) == SHAPE
    assert L.gemm_grouped_workspace_size(2000, 1, 8, 8, ctypes.byref(b)) == SHAPE
    assert L.gemm_lora_workspace_size(1, 8, 8, 256, 1, ctypes.byref(b)) == SHAPE
    assert L.gemm_route_workspace_size(1, 8, 9, ctypes.byref(b)) == INVALID
    assert L.gemm_route_workspace_size(64, 128, 8, ctypes.byref(b)) == G.GEMM_OK and b.value == 0
    assert L.gemm_route_workspace_size(65, 128, 8, ctypes.byref(b)) == G.GEMM_OK and b.value == 4 * 128 * 4


def test_binding_checks_tensors():
    """Wrong shapes, types, devices and layouts are ValueErrors before any call."""
    torch = pytest.importorskip("torch")
    half = torch.float16
    x, w, off = torch.zeros((4, 16), dtype=half), torch.zeros((2, 8, 16), dtype=half), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        R.gemm_grouped_nt(x, w, off)          # host tensors
    with pytest.raises(ValueError):
        R.gemm_grouped_tn(x, x, off)
    with pytest.raises(ValueError):
        R.gemm_lora_nt(x, w[0], w, w, off)
    with pytest.raises(ValueError):
        R.gemm_route_topk(x, 2)
    with pytest.raises(ValueError):
        R._dtype(torch.float32)
    with pytest.raises(ValueError):
        R._dtype(torch.int8, f32=True)
    assert R._dtype(torch.bfloat16) == R.DTYPE_BF16
