"""Which way the adapters run, from sizes alone (pure host code, no GPU)."""
import ctypes

import pytest

from dense_fp16_gemm_03_gb300 import build as pkg_build
from dense_fp16_gemm_03_gb300 import gemm as G
from dense_fp16_gemm_03_gb300 import ragged as R

SMS = 152


@pytest.fixture(scope="module")
def L():
    pkg_build.build()
    return R.lib()


def items(rows, n, rank):
    """What the two kernels beside the projection count: four of a row's u's, 128 of its columns."""
    return max(rows * (rank // 4), rows * -(-n // 128))


@pytest.mark.parametrize("rows,n,k,rank,adapters", [
    (1 << 27, 8, 8, 128, 256),              # 2^32 items: the count itself would be zero
    ((1 << 27) - 1, 8, 8, 128, 256),        # the step past the last one would wrap
    ((1 << 27) - 300, 8, 8, 128, 1000),
    (1 << 29, 8, 8, 32, 256),
    ((1 << 31) - 1, 8, 8, 8, 1000),
    ((1 << 31) - 1, 8, 8, 128, 1000),
])
def test_items_are_never_more_than_32_bits_count(L, rows, n, k, rank, adapters):
    most_step = 16 * SMS * 4
    assert R.gemm_lora_way(rows, n, k, rank, adapters, SMS) == R.LORA_TENSOR_CORES or items(rows, n, rank) + most_step < 1 << 32
    # the last rows that run beside, by bisection
    lo, hi = 64, rows
    if R.gemm_lora_way(hi, n, k, rank, adapters, SMS) == R.LORA_BESIDE:
        return
    while hi - lo > 1:
        mid = (lo + hi) // 2
        if R.gemm_lora_way(mid, n, k, rank, adapters, SMS) == R.LORA_BESIDE:
            lo = mid
        else:
            hi = mid
    assert items(lo, n, rank) + most_step < 1 << 32


def test_few_rows_run_beside_and_many_of_few_adapters_on_the_tensor_cores(L):
    for rows in (1, 2, 32, 64):
        assert R.gemm_lora_way(rows, 8192, 4096, 16, 64, SMS) == R.LORA_BESIDE
    assert R.gemm_lora_way(8192, 8192, 4096, 64, 16, SMS) == R.LORA_TENSOR_CORES
    assert R.gemm_lora_way(64, (1 << 31) - 8, 8, 8, 1, SMS) == R.LORA_BESIDE


def test_refusals(L):
    way = ctypes.c_int32()
    ref = ctypes.byref(way)
    assert L.gemm_lora_way(1, 8, 8, 8, 1, SMS, None) == G.GEMM_ERR_INVALID_ARG
    for sms in (-1, 1):
        assert L.gemm_lora_way(1, 8, 8, 8, 1, sms, ref) == G.GEMM_ERR_INVALID_ARG
    assert L.gemm_lora_way(-1, 8, 8, 8, 1, SMS, ref) == G.GEMM_ERR_INVALID_ARG
    assert L.gemm_lora_way(1, 9, 8, 8, 1, SMS, ref) == G.GEMM_ERR_UNSUPPORTED_SHAPE
    assert L.gemm_lora_way(1, 8, 8, 136, 1, SMS, ref) == G.GEMM_ERR_UNSUPPORTED_SHAPE
    assert L.gemm_lora_way(1 << 31, 8, 8, 8, 1, SMS, ref) == G.GEMM_ERR_UNSUPPORTED_SHAPE
