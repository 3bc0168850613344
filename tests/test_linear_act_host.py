"""The normal distribution function of the epilogues: the errors that linear_act.cuh states, from its own coefficients."""
import os
import re

import numpy as np
import pytest

log_ndtr = pytest.importorskip("scipy.special").log_ndtr

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_fp16_gemm_03_gb300", "csrc", "linear_act.cuh")
F = np.float32


def coefficients():
    text = open(SOURCE).read()
    body = text[text.index("normal_cdf(Two z"):text.index("// P(-|z|)")]
    found = [F(v) for v in re.findall(r"two\((-?0\.\d{10,})f\)", body)]
    assert len(found) == 8 and "two(0.3f)" in body
    return found


def points(low, high):
    return np.linspace(low, high, 400001).astype(F).astype(np.float64)


def test_the_form_in_64_bits():
    x = points(0, 14)
    t = 1 / (1 + np.float64(F(0.3)) * x)
    q = np.zeros_like(x)
    for c in coefficients():
        q = q * t + np.float64(c)
    assert np.abs(q * t * np.exp(-x * x / 2 - log_ndtr(-x)) - 1).max() < 1.7e-7


@pytest.mark.parametrize("low,high,most", [(0, 2, 6e-7), (2, 5, 1.6e-6), (5, 12.8, 8e-6)])
def test_the_function_in_fp32(low, high, most):
    """Each step rounded to fp32, a multiplication with its addition once, the exponential and the reciprocal exact before
    their own rounding (the hardware's add 2^-22 each)."""
    x = points(low, high)
    x32 = x.astype(F)
    t = (1 / (x * np.float64(F(0.3)) + 1).astype(F).astype(np.float64)).astype(F)
    e = np.exp2((x32 * x32 * F(-0.5 * 1.4426950408889634)).astype(np.float64)).astype(F)
    q = np.zeros_like(x32)
    for c in coefficients():
        q = (q.astype(np.float64) * t + c).astype(F)
    q = q * (t * e)
    assert np.abs(q / np.exp(log_ndtr(-x)) - 1).max() < most
