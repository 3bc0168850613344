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
// below 1.7e-7 in 64 bits with the coefficients as they stand in fp32, for x up to
// 14, past which P(-x) is 0 in fp32).  It shares the exponential with the density
// and has no cancellation in the tail.
// Exponentials and reciprocals are the hardware's approximate ones, with a relative
// error of some 2^-22.  The exponential's argument is rounded before: one of size a
// adds up to a 2^-23, so P(-x) in fp32 is off by 6e-7 up to x = 2, 1.6e-6 up to 5 and
// 8e-6 at the end of its range, and by what the hardware's two add.  Results in 16
// bits do not see that; in a bias gradient, a sum in fp32, the tail weighs as little
// as it is small.
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

// Two values side by side: sm_100 and later multiply and add them in one instruction, and with two values' exponentials and
// reciprocals that is most of an activation (16384 x 4096 through gelu's derivative: 26 instructions a value one by one,
// some 15 in pairs, where the bytes leave room for 30).
struct Two {
    uint64_t v;
};

__device__ __forceinline__ Two two(float a, float b)
{
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ Two two(float a)
{
    return two(a, a);
}

__device__ __forceinline__ float2 apart(Two a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}

__device__ __forceinline__ Two operator*(Two a, Two b)
{
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ Two operator+(Two a, Two b)
{
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ Two fma(Two a, Two b, Two c)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

__device__ __forceinline__ Two ex2(Two a)
{
    const float2 x = apart(a);
    return two(ex2(x.x), ex2(x.y));
}

__device__ __forceinline__ Two rcp(Two a)
{
    const float2 x = apart(a);
    return two(rcp(x.x), rcp(x.y));
}

__device__ __forceinline__ Two sigmoid(Two x)
{
    return rcp(two(1.0f) + ex2(x * two(-kLog2e)));
}

// P(z), and e^(-z^2/2) in `*e`
__device__ __forceinline__ Two normal_cdf(Two z, Two *e)
{
    const float2 s = apart(z);
    const Two t = rcp(fma(two(0.3f), two(fabsf(s.x), fabsf(s.y)), two(1.0f)));
    const Two g = ex2(z * z * two(-0.5f * kLog2e));
    Two q = two(0.03567477688193321f);
    q = fma(q, t, two(-0.15720310807228088f));
    q = fma(q, t, two(0.20635353028774261f));
    q = fma(q, t, two(-0.05368367210030556f));
    q = fma(q, t, two(0.12856164574623108f));
    q = fma(q, t, two(0.09991348534822464f));
    q = fma(q, t, two(0.12075395882129669f));
    q = fma(q, t, two(0.11962930113077164f));
    q = q * (t * g);  // P(-|z|)
    *e = g;
    const float2 low = apart(q), high = apart(fma(q, two(-1.0f), two(1.0f)));
    return two(s.x > 0.0f ? high.x : low.x, s.y > 0.0f ? high.y : low.y);
}

constexpr float kTanh1 = 1.5957691216057308f;             // 2 sqrt(2/pi)
constexpr float kTanh3 = 1.5957691216057308f * 0.044715f;

// s(2u), and z^2 in `*square`
__device__ __forceinline__ Two tanh_gate(Two z, Two *square)
{
    *square = z * z;
    return sigmoid(z * fma(two(kTanh3), *square, two(kTanh1)));
}

__device__ __forceinline__ float relu(float z)
{
    return z <= 0.0f ? 0.0f : z;
}

template <int ACT>
__device__ __forceinline__ Two apply(Two z)
{
    const float2 s = apart(z);
    if constexpr (ACT == GEMM_ACT_RELU) return two(relu(s.x), relu(s.y));
    if constexpr (ACT == GEMM_ACT_RELU2) {
        const Two r = two(relu(s.x), relu(s.y));
        return r * r;
    }
    if constexpr (ACT == GEMM_ACT_GELU) {
        Two e;
        return z * normal_cdf(z, &e);
    }
    if constexpr (ACT == GEMM_ACT_GELU_TANH) {
        Two square;
        return z * tanh_gate(z, &square);
    }
    if constexpr (ACT == GEMM_ACT_SILU) return z * sigmoid(z);
    return z;
}

// d f'(z)
template <int ACT>
__device__ __forceinline__ Two apply_grad(Two d, Two z)
{
    const float2 s = apart(z);
    if constexpr (ACT == GEMM_ACT_RELU) {
        const float2 g = apart(d);
        return two(s.x > 0.0f ? g.x : 0.0f, s.y > 0.0f ? g.y : 0.0f);
    }
    if constexpr (ACT == GEMM_ACT_RELU2) return d * (two(relu(s.x), relu(s.y)) * two(2.0f));
    if constexpr (ACT == GEMM_ACT_GELU) {
        Two e;
        const Two p = normal_cdf(z, &e);
        return d * fma(z * two(0.3989422804014327f), e, p);
    }
    if constexpr (ACT == GEMM_ACT_GELU_TANH) {
        Two square;
        const Two p = tanh_gate(z, &square);
        // (where z^2 would be infinite, 1 - p is 0)
        const float2 sq = apart(square);
        const Two slope = fma(two(3.0f * kTanh3), two(fminf(sq.x, 1e30f), fminf(sq.y, 1e30f)), two(kTanh1));
        return d * fma(z * p * fma(p, two(-1.0f), two(1.0f)), slope, p);
    }
    if constexpr (ACT == GEMM_ACT_SILU) {
        const Two p = sigmoid(z);
        return d * fma(z * p, fma(p, two(-1.0f), two(1.0f)), p);
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
