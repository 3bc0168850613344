// Activations and their derivatives, in fp32, as the epilogues of the linear
// products and their gradients apply them.
//
//   relu       max(z, 0), NaN kept             1 where z > 0, else 0 (also for NaN)
//   relu2      relu(z)^2                       2 relu(z)
//   gelu       z P(z), P the normal            P(z) + z p(z), p the density
//              distribution function
//   gelu_tanh  z s(2u), u = sqrt(2/pi)         s(2u) + z s(2u) (1 - s(2u)) 2u'
//              (z + 0.044715 z^3), as 0.5 z (1 + tanh u)
//   silu       z s(z), s(z) = 1 / (1 + e^-z)   s(z) + z s(z) (1 - s(z))
//
// P(-x) for x >= 0 is e^(-x^2/2) t Q(t) with t = 1 / (1 + 0.3 x): the form
// of Abramowitz and Stegun 7.1.26 with a polynomial of degree 7 fitted here
// (weighted least squares on Chebyshev points until the relative error is even:
// below 1.5e-7 for x up to 14, past which P(-x) is 0 in fp32).  It shares the
// exponential with the density and has no cancellation in the tail.
// Exponentials and reciprocals are the hardware's approximate ones (relative
// error some 2^-22, which 16-bit results do not see).
#pragma once

#include <stdint.h>

#include "gemm_linear.h"

namespace gemm_f16 {
namespace act {

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-x); 0 for -infinity
__device__ __forceinline__ float sigmoid(float x)
{
    return rcp(1.0f + ex2(-kLog2e * x));
}

// P(z), and e^(-z^2/2) in `*e`
__device__ __forceinline__ float normal_cdf(float z, float *e)
{
    const float x = fabsf(z);
    const float t = rcp(fmaf(0.3f, x, 1.0f));
    const float g = ex2(z * z * (-0.5f * kLog2e));
    float q = 0.03567477688193321f;
    q = fmaf(q, t, -0.15720310807228088f);
    q = fmaf(q, t, 0.20635353028774261f);
    q = fmaf(q, t, -0.05368367210030556f);
    q = fmaf(q, t, 0.12856164574623108f);
    q = fmaf(q, t, 0.09991348534822464f);
    q = fmaf(q, t, 0.12075395882129669f);
    q = fmaf(q, t, 0.11962930113077164f);
    q *= t * g;  // P(-x)
    *e = g;
    return z > 0.0f ? 1.0f - q : q;
}

constexpr float kTanh1 = 1.5957691216057308f;             // 2 sqrt(2/pi)
constexpr float kTanh3 = 1.5957691216057308f * 0.044715f;

// s(2u)
__device__ __forceinline__ float tanh_gate(float z)
{
    return sigmoid(z * fmaf(kTanh3, z * z, kTanh1));
}

template <int ACT>
__device__ __forceinline__ float apply(float z)
{
    if constexpr (ACT == GEMM_ACT_RELU) return z <= 0.0f ? 0.0f : z;
    if constexpr (ACT == GEMM_ACT_RELU2) {
        const float r = z <= 0.0f ? 0.0f : z;
        return r * r;
    }
    if constexpr (ACT == GEMM_ACT_GELU) {
        float e;
        return z * normal_cdf(z, &e);
    }
    if constexpr (ACT == GEMM_ACT_GELU_TANH) return z * tanh_gate(z);
    if constexpr (ACT == GEMM_ACT_SILU) return z * sigmoid(z);
    return z;
}

// d f'(z)
template <int ACT>
__device__ __forceinline__ float apply_grad(float d, float z)
{
    if constexpr (ACT == GEMM_ACT_RELU) return z > 0.0f ? d : 0.0f;
    if constexpr (ACT == GEMM_ACT_RELU2) return d * (2.0f * (z <= 0.0f ? 0.0f : z));
    if constexpr (ACT == GEMM_ACT_GELU) {
        float e;
        const float p = normal_cdf(z, &e);
        return d * fmaf(z * 0.3989422804014327f, e, p);
    }
    if constexpr (ACT == GEMM_ACT_GELU_TANH) {
        const float s = tanh_gate(z);
        // (where z^2 would be infinite, 1 - s is 0)
        return d * fmaf(z * s * (1.0f - s), fmaf(3.0f * kTanh3, fminf(z * z, 1e30f), kTanh1), s);
    }
    if constexpr (ACT == GEMM_ACT_SILU) {
        const float s = sigmoid(z);
        return d * fmaf(z * s, 1.0f - s, s);
    }
    return d;
}

// f(Kind<a>()): one branch for a whole piece of work
template <int ACT>
struct Kind {
    static constexpr int value = ACT;
};

template <class F>
__device__ __forceinline__ void with_kind(uint32_t a, F &&f)
{
    switch (a) {
    case GEMM_ACT_RELU: f(Kind<GEMM_ACT_RELU>()); break;
    case GEMM_ACT_RELU2: f(Kind<GEMM_ACT_RELU2>()); break;
    case GEMM_ACT_GELU: f(Kind<GEMM_ACT_GELU>()); break;
    case GEMM_ACT_GELU_TANH: f(Kind<GEMM_ACT_GELU_TANH>()); break;
    case GEMM_ACT_SILU: f(Kind<GEMM_ACT_SILU>()); break;
    default: f(Kind<GEMM_ACT_NONE>()); break;
    }
}

}  // namespace act
}  // namespace gemm_f16
