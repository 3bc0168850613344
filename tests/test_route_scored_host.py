"""Host-side checks of the router with scores that need no GPU: every argument is validated before a device is touched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from dense_fp16_gemm_03_gb300 import build as pkg_build  # noqa: E402
from dense_fp16_gemm_03_gb300 import gemm as G  # noqa: E402
from dense_fp16_gemm_03_gb300 import ragged as R  # noqa: E402

P = 1 << 20       # an aligned address that is never dereferenced
INVALID, ALIGN, SHAPE = G.GEMM_ERR_INVALID_ARG, G.GEMM_ERR_ALIGNMENT, G.GEMM_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def L():
    pkg_build.build()
    return R.lib()


def scored(L, dtype=2, score=1, rows=10, experts=64, top=4, groups=8, top_groups=3, group_top=2, renorm=1, logits=P, bias=P, ids=P, weights=P,
           offsets=P, order=P, position=P):
    return L.gemm_route_scored(dtype, score, rows, experts, top, groups, top_groups, group_top, renorm, ctypes.c_float(1.0), logits, bias, ids,
                               weights, offsets, order, position, None, 0, None)


def grad(L, dtype=2, score=1, rows=10, experts=64, top=4, renorm=1, logits=P, ids=P, dweights=P, dlogits=P):
    return L.gemm_route_scored_grad(dtype, score, rows, experts, top, renorm, ctypes.c_float(1.0), logits, ids, dweights, dlogits, None)


@pytest.mark.parametrize("change,status", [
    ({"rows": -1}, INVALID), ({"experts": 0}, INVALID), ({"experts": 1032}, SHAPE), ({"top": 0}, INVALID), ({"top": 65}, INVALID),
    ({"experts": 512, "top": 33}, SHAPE), ({"rows": 1 << 31}, SHAPE), ({"dtype": 3}, INVALID), ({"score": 2}, INVALID), ({"score": -1}, INVALID),
    ({"groups": 0}, INVALID), ({"groups": 7}, INVALID), ({"experts": 60, "groups": 6}, SHAPE), ({"groups": 64}, SHAPE),
    ({"top_groups": 0}, INVALID), ({"top_groups": 9}, INVALID), ({"group_top": 0}, INVALID), ({"group_top": 3}, INVALID),
    ({"top": 25}, INVALID), ({"logits": None}, INVALID), ({"logits": P + 8}, ALIGN), ({"bias": P + 2}, ALIGN), ({"ids": None}, INVALID),
    ({"weights": None}, INVALID), ({"offsets": None}, INVALID), ({"order": P + 2}, ALIGN), ({"position": None}, INVALID),
])
def test_refusals(L, change, status):
    assert scored(L, **change) == status


@pytest.mark.parametrize("change,status", [
    ({"rows": -1}, INVALID), ({"top": 0}, INVALID), ({"dtype": -1}, INVALID), ({"score": 5}, INVALID), ({"logits": None}, INVALID),
    ({"ids": None}, INVALID), ({"dweights": P + 2}, ALIGN), ({"dlogits": None}, INVALID),
])
def test_grad_refusals(L, change, status):
    assert grad(L, **change) == status


def test_grad_of_no_rows(L):
    assert grad(L, rows=0, logits=None, ids=None, dweights=None, dlogits=None) == G.GEMM_OK


def test_limits_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gemm_ragged.h")).read()
    assert int(re.search(r"#define GEMM_ROUTE_MAX_GROUPS (\d+)", text).group(1)) == R.MAX_ROUTE_GROUPS
    for name, value in R.ROUTE_SCORES.items():
        assert int(re.search(r"GEMM_ROUTE_%s = (\d+)" % name.upper(), text).group(1)) == value
