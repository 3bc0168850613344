// The experts' router with scores, a bias for the choice, and groups of experts:
//
//   s = softmax(l) or 1 / (1 + e^-l);  c = s + bias
//   a group's score: the largest, or the sum of the two largest, of its c
//   ids = the `top` largest c in the `top_groups` best groups, ties to the lowest index
//   w = scale s[ids], divided by the sum of s[ids] if renorm
//
// and the gradient of the logits.  What a choice comes to (offsets, order,
// position) is the top-k router's, in route_kernel.cuh.
//
// One warp per row.  A group's experts lie in 32 / groups neighbouring lanes, in
// runs of experts / 32 (rounded up), so a group's best are found in the lane and by
// a few shuffles, and a lane's logits are neighbours in memory.
//
// The choice is that of the exact c.  Rounded to 32 bits, close ones could change
// places, and which do would depend on the exponential's last bits.  So c in fp32,
// whose error is bounded below, decides only where what it compares is further apart
// than that: between neighbours of the chosen ones, the first one not chosen, and the
// last group kept and the best one dropped.  A row with a closer call (some 1 in 500 of
// 256 experts with normal logits) is chosen again in 64 bits by route_exact.
// Without a bias, and unless groups go by sums, c has the logits' order, and the
// logits themselves are compared, which is exact.
//
// Error of c, in units of 2^-24, all exponentials and reciprocals the hardware's (2^-22
// and 2^-23 relative) of arguments x with two roundings (2 |x|), |x| e^-x < 0.37:
//   sigmoid   4.4 for s (s (1 - s) is at most 1/4, |x| s (1 - s) at most 0.23), and c's
//             rounding, (1 + |bias|) / 2: below 6 + |bias|
//   softmax   with P the row's largest: 5.2 P from the exponential, the sum's relative
//             error (18 from the exponentials, 37 from adding up to 32 in a lane and 5
//             shuffles) and the quotient's 3, and c's rounding: below 65 P + |bias|
// Two c that are compared are off by twice that, two sums of two by four times that and
// a rounding more.
//
// Bound by issued instructions, as the top-k router: 1032 a row of 256 experts, the eight best of the four best of eight
// groups, at 61% of the issue slots; 16384 rows 33.4 us with the rows' places, the gradient 6.8, in a graph.
#pragma once

#include "gemm_ragged.h"
#include "linear_act.cuh"
#include "ragged_kernel.cuh"
#include "route_kernel.cuh"

namespace gemm_f16 {

struct RouteScoredParams : RouteParams {
    const float *bias;     // [experts], or null
    uint32_t sigmoid;      // else softmax
    uint32_t groups, top_groups, group_top;
    uint32_t size;         // experts of a group
    uint32_t run;          // experts of a lane
    uint32_t spread;       // a group has 2^spread lanes
    uint32_t by_logit;     // c has the logits' order
    float scale;
};

// Which experts a lane has: [first, first + count).
struct RouteLane {
    uint32_t lanes, group, first, count;
    __device__ __forceinline__ explicit RouteLane(const RouteScoredParams &p)
    {
        const uint32_t lane = threadIdx.x & 31u;
        lanes = 1u << p.spread;
        group = lane >> p.spread;
        const uint32_t from = (lane & (lanes - 1u)) * p.run;
        first = group * p.size + from;
        count = from < p.size ? min(p.run, p.size - from) : 0u;
    }
};

__device__ __forceinline__ float route_logit(const RouteParams &p, size_t at)
{
    if (p.dtype == 2u) return static_cast<const float *>(p.logits)[at];
    const uint16_t v = static_cast<const uint16_t *>(p.logits)[at];
    return p.dtype == 1u ? __uint_as_float(uint32_t(v) << 16) : __half2float(__ushort_as_half(v));
}

// A lane's logits of a row (-infinity where it has none): all loads before the first conversion.
template <int VPT>
__device__ __forceinline__ void route_load_run(const RouteScoredParams &p, size_t row, const RouteLane &at, bool live, float (&f)[VPT])
{
    if (p.dtype == 2u) {
        const float *from = static_cast<const float *>(p.logits) + row * p.experts + at.first;
        if (VPT >= 4 && p.run == uint32_t(VPT) && at.count == uint32_t(VPT) && p.experts % 4u == 0u && p.size % 4u == 0u) {
#pragma unroll
            for (int i = 0; i < VPT / 4; ++i) {
                const float4 v = live ? reinterpret_cast<const float4 *>(from)[i] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                f[4 * i] = v.x;
                f[4 * i + 1] = v.y;
                f[4 * i + 2] = v.z;
                f[4 * i + 3] = v.w;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) f[i] = (live && uint32_t(i) < at.count) ? from[i] : -INFINITY;
        return;
    }
    const uint32_t none = p.dtype == 1u ? 0xFF80u : 0xFC00u;  // -infinity
    const uint16_t *from = static_cast<const uint16_t *>(p.logits) + row * p.experts + at.first;
    uint32_t raw[VPT];
    if (VPT >= 8 && p.run == uint32_t(VPT) && at.count == uint32_t(VPT) && p.experts % 8u == 0u && p.size % 8u == 0u) {
#pragma unroll
        for (int i = 0; i < VPT / 8; ++i) {
            const uint4 v = live ? reinterpret_cast<const uint4 *>(from)[i] : make_uint4(none * 0x10001u, none * 0x10001u, none * 0x10001u, none * 0x10001u);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                raw[8 * i + 2 * j] = w[j] & 0xFFFFu;
                raw[8 * i + 2 * j + 1] = w[j] >> 16;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) raw[i] = (live && uint32_t(i) < at.count) ? uint32_t(from[i]) : none;
    }
    if (p.dtype == 1u) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) f[i] = __uint_as_float(raw[i] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) f[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(raw[i])));
    }
}

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// The choice of one row in 64 bits: the id of choice `lane`, or -1.  Run by a whole warp, for few rows: nothing here is
// made fast.  c that cannot be chosen is -infinity; NaN comes after all others.
template <int VPT>
__device__ __noinline__ int32_t route_exact(const RouteScoredParams &p, size_t row)
{
    const RouteLane at(p);
    const uint32_t lane = threadIdx.x & 31u;
    const double last = -1.7e308;
    double c[VPT];
    float most = -INFINITY;
    bool nan = false;
    for (int i = 0; i < VPT; ++i) {
        const float f = uint32_t(i) < at.count ? route_logit(p, row * p.experts + at.first + i) : -INFINITY;
        c[i] = f;
        most = fmaxf(most, f);
        nan = nan || f != f;
    }
    for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    const bool bad = __any_sync(0xffffffffu, nan) || most == INFINITY;
    double sum = 0.0;
    if (!p.sigmoid) {
        for (int i = 0; i < VPT; ++i)
            if (c[i] != -INFINITY) sum += exp(c[i] - double(most));
        sum = warp_sum(sum);
    }
    double one = -INFINITY, two = -INFINITY;  // the lane's two largest
    for (int i = 0; i < VPT; ++i) {
        if (c[i] == -INFINITY) continue;
        double v = p.by_logit ? c[i] : p.sigmoid ? 1.0 / (1.0 + exp(-c[i])) : exp(c[i] - double(most)) / sum;
        if (!p.sigmoid && bad) v = NAN;
        if (p.bias) v = p.bias[at.first + i] == -INFINITY ? -INFINITY : v + double(p.bias[at.first + i]);
        if (v != v) v = last;
        c[i] = v;
        if (v > one) {
            two = one;
            one = v;
        } else if (v > two) {
            two = v;
        }
    }
    if (p.groups > 1u) {
        for (uint32_t d = at.lanes / 2u; d > 0u; d >>= 1) {
            const double o1 = __shfl_xor_sync(0xffffffffu, one, d), o2 = __shfl_xor_sync(0xffffffffu, two, d);
            two = fmax(fmin(one, o1), fmax(two, o2));
            one = fmax(one, o1);
        }
        double score = one;
        if (p.group_top == 2u && two != -INFINITY) score = (one == last || two == last) ? last : one + two;
        uint32_t rank = 0;
        for (uint32_t g = 0; g < p.groups; ++g) {
            const double o = __shfl_sync(0xffffffffu, score, g * at.lanes);
            rank += (o > score || (o == score && g < at.group)) ? 1u : 0u;
        }
        if (rank >= p.top_groups)
            for (int i = 0; i < VPT; ++i) c[i] = -INFINITY;
    }
    int32_t id = -1;
    for (uint32_t j = 0; j < p.top; ++j) {
        double best = -INFINITY;
        uint32_t e = 0xffffffffu;
        for (int i = 0; i < VPT; ++i)
            if (c[i] > best) {
                best = c[i];
                e = at.first + i;
            }
        for (int d = 16; d > 0; d >>= 1) {
            const double ob = __shfl_xor_sync(0xffffffffu, best, d);
            const uint32_t oe = __shfl_xor_sync(0xffffffffu, e, d);
            if (ob > best || (ob == best && oe < e)) {
                best = ob;
                e = oe;
            }
        }
        if (best == -INFINITY) break;
        if (lane == j) id = int32_t(e);
        for (int i = 0; i < VPT; ++i)
            if (at.first + i == e && uint32_t(i) < at.count) c[i] = -INFINITY;
    }
    return id;
}

__device__ __forceinline__ float route_top(float l)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l = fmaxf(l, __shfl_xor_sync(0xffffffffu, l, d));
    return l;
}

// e^-from / (1 + e^-l) for from <= 0 and l <= from or from = 0: scores that are divided by their sum keep their ratio where
// they themselves are too small for 32 bits.
__device__ __forceinline__ float route_sigmoid(float l, float from)
{
    const float e = act::ex2(-act::kLog2e * fabsf(l));
    const float over = act::rcp(1.0f + e);
    return l < 0.0f ? act::ex2(act::kLog2e * (l - from)) * over : over;
}

// c of an expert in 64 bits, for a row whose softmax has its largest logit `most` and the sum `sum` of its exponentials.
__device__ __noinline__ double route_score64(const RouteScoredParams &p, size_t row, uint32_t e, float most, double sum)
{
    const double l = route_logit(p, row * p.experts + e);
    const double s = p.by_logit ? l : p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - double(most)) / sum;
    return p.bias ? s + double(p.bias[e]) : s;
}

// A warp's part of the choice's shared memory: its picks, and its lanes' keys but the first.
template <int VPT>
constexpr uint32_t kRouteListBytes = 256u + 128u * VPT;

// A key is the ordered bits of c, its last ones replaced by the place in the lane, the first place the largest: a lane's keys
// differ and are sorted by a maximum and a minimum each, and the choice needs no index beside them.  0: never chosen; NaN
// has the smallest value of all others.
template <int VPT>
struct RouteKey {
    static constexpr int kBits = VPT <= 1 ? 0 : VPT <= 2 ? 1 : VPT <= 4 ? 2 : VPT <= 8 ? 3 : VPT <= 16 ? 4 : 5;
    static constexpr uint32_t kMask = (1u << kBits) - 1u;
    static __device__ __forceinline__ uint32_t finite(float c, int i)
    {
        const uint32_t u = __float_as_uint(c + 0.0f);  // (-0 is 0)
        return ((u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u)) & ~kMask) | (kMask - uint32_t(i));
    }
    static __device__ __forceinline__ uint32_t any(float c, int i)  // NaN and infinities too
    {
        return c == -INFINITY ? 0u : c != c ? (1u << kBits) | (kMask - uint32_t(i)) : finite(c, i);
    }
    static __device__ __forceinline__ float value(uint32_t key)  // of a number
    {
        key &= ~kMask;
        return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
    }
};

// Whether two experts of a row have the same logit and the same bias, and with them the same c.
__device__ __forceinline__ bool route_same(const RouteScoredParams &p, size_t row, int32_t a, int32_t b)
{
    return route_logit(p, row * p.experts + a) == route_logit(p, row * p.experts + b) && (!p.bias || p.bias[a] == p.bias[b]);
}

// A lane's keys in falling order (Batcher's odd-even merge sort).
template <int N>
__device__ __forceinline__ void route_sort(uint32_t (&key)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t x = key[i + j], y = key[i + j + k];
                        key[i + j] = max(x, y);
                        key[i + j + k] = min(x, y);
                    }
}

// What the choice needs to know of the biases: how large the finite ones are, and whether this lane's others are -infinity or
// worse.  (The biases themselves are read again for each row: in registers they would cost more than they spare.)
struct RouteBias {
    float widest;
    bool plain, masks;  // none is +infinity or NaN; one is -infinity (this lane's)
    __device__ __forceinline__ RouteBias(const RouteScoredParams &p, const RouteLane &at) : widest(0.0f), plain(true), masks(false)
    {
        if (p.bias)
            for (uint32_t i = 0; i < at.count; ++i) {
                const float b = p.bias[at.first + i];
                if (fabsf(b) < INFINITY) widest = fmaxf(widest, fabsf(b));
                plain = plain && b < INFINITY;
                masks = masks || b == -INFINITY;
            }
        widest = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(widest)));
    }
};

// A lane's biases (0 without), as route_load_run has its logits.
template <int VPT>
__device__ __forceinline__ void route_load_bias(const RouteScoredParams &p, const RouteLane &at, bool full, float (&b)[VPT])
{
    if (p.bias == nullptr) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) b[i] = 0.0f;
        return;
    }
    const float *from = p.bias + at.first;
    if (VPT >= 4 && full && (reinterpret_cast<uintptr_t>(p.bias) & 15u) == 0u) {
#pragma unroll
        for (int i = 0; i < VPT / 4; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(from)[i];
            b[(4 * i) % VPT] = v.x;
            b[(4 * i + 1) % VPT] = v.y;
            b[(4 * i + 2) % VPT] = v.z;
            b[(4 * i + 3) % VPT] = v.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) b[i] = uint32_t(i) < at.count ? from[i] : 0.0f;
}

// What a row's weights need besides the chosen logits.
struct RouteRow {
    float most, sum;  // softmax: the largest logit, the sum of the exponentials
    bool bad;         // a softmax of NaN or +infinity: every score is NaN
};

// The sum of a softmax's exponentials in 64 bits, for the scores that are compared so.
__device__ __noinline__ double route_sum64(const RouteScoredParams &p, size_t row, float most)
{
    if (p.sigmoid || p.by_logit) return 1.0;
    const RouteLane at(p);
    double sum = 0.0;
#pragma unroll 1
    for (uint32_t i = 0; i < at.count; ++i) sum += exp(double(route_logit(p, row * p.experts + at.first + i)) - double(most));
    return warp_sum(sum);
}

// Close calls.  They are few, and what they cost is mostly the instructions' way from memory (a row that went through a second
// copy of the whole choice held its block up by 13 us), so the code is short.
//
// Whether all experts of a row have the same logit and the same bias, as before a training's first step: then their order, and
// the groups', is that of the indices.
__device__ __noinline__ bool route_even(const RouteScoredParams &p, size_t row)
{
    bool same = true;
#pragma unroll 1
    for (uint32_t e = threadIdx.x & 31u; e < p.experts; e += 32u) same = same && route_same(p, row, 0, int32_t(e));
    return __all_sync(0xffffffffu, same);
}

// Rank of this lane's group by its score in 64 bits.  `one`, `two`: the lane's experts that may be among the group's largest
// (-1 for none).
__device__ __noinline__ uint32_t route_rank64(const RouteScoredParams &p, size_t row, float most, bool sums, int32_t one, int32_t two)
{
    const uint32_t lane = threadIdx.x & 31u, lanes = 1u << p.spread;
    const double sum = route_sum64(p, row, most);
    double first = -INFINITY, second = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int32_t e = i ? two : one;
        if (!__any_sync(0xffffffffu, e >= 0)) break;
        const double v = e >= 0 ? route_score64(p, row, uint32_t(e), most, sum) : -INFINITY;
        second = fmax(second, fmin(first, v));
        first = fmax(first, v);
    }
#pragma unroll 1
    for (uint32_t d = lanes / 2u; d > 0u; d >>= 1) {
        const double o1 = __shfl_xor_sync(0xffffffffu, first, d), o2 = __shfl_xor_sync(0xffffffffu, second, d);
        second = fmax(fmin(first, o1), fmax(second, o2));
        first = fmax(first, o1);
    }
    const double score = sums && second != -INFINITY ? first + second : first;
    uint32_t rank = 0;
#pragma unroll 1
    for (uint32_t g = 0; g < p.groups; ++g) {
        const double o = __shfl_sync(0xffffffffu, score, g << p.spread);
        rank += (o > score || (o == score && g < (lane >> p.spread))) ? 1u : 0u;
    }
    return rank;
}

// The experts in `id` (of the first `count` lanes) in the order of their scores in 64 bits, the `top` first ones.
__device__ __noinline__ int32_t route_order64(const RouteScoredParams &p, size_t row, float most, int32_t id, uint32_t count)
{
    const uint32_t lane = threadIdx.x & 31u;
    const double sum = route_sum64(p, row, most);
    const double v = lane < count ? route_score64(p, row, uint32_t(id), most, sum) : -INFINITY;
    uint32_t rank = 0;
#pragma unroll 1
    for (uint32_t i = 0; i < count; ++i) {
        const double o = __shfl_sync(0xffffffffu, v, i);
        const int32_t e = __shfl_sync(0xffffffffu, id, i);
        rank += (o > v || (o == v && e < id)) ? 1u : 0u;
    }
    int32_t chosen = -1;
#pragma unroll 1
    for (uint32_t i = 0; i < count; ++i) {
        const uint32_t r = __shfl_sync(0xffffffffu, rank, i);
        const int32_t e = __shfl_sync(0xffffffffu, id, i);
        if (r == lane) chosen = e;
    }
    return lane < p.top ? chosen : -1;
}

// The choice of one row: the id of choice `lane`, or -1.  `keep`: a lane's keys but the first, one behind another at a step
// of 32 words, `pick`: 32 pairs of words, both the warp's own.
template <int VPT>
__device__ __forceinline__ int32_t route_choose(const RouteScoredParams &p, size_t row, const RouteLane &at, const RouteBias &bias,
                                                uint32_t *keep, uint2 *pick, RouteRow *r)
{
    using Key = RouteKey<VPT>;
    const uint32_t lane = threadIdx.x & 31u;
    const bool full = p.run == uint32_t(VPT) && p.run << p.spread == p.size;  // every lane has VPT experts
    const bool sums = p.groups > 1u && p.group_top == 2u;
    const bool exact_keys = p.by_logit && p.dtype != 2u;  // (16 bits fit)
    // a key loses less than this of c (at most 1 + widest)
    float tol = (16.0f + 4.0f * bias.widest) * 0x1p-24f + (1.0f + bias.widest) * float(Key::kMask + 1u) * 0x1p-23f;
    float most = -INFINITY, sum = 0.0f;
    bool bad = false, numbers = bias.plain;  // numbers: no logit or bias is +infinity or NaN
    uint32_t key[VPT];
    {
        float f[VPT];
        route_load_run<VPT>(p, row, at, true, f);
        // and none is -infinity: 0 x is 0 for numbers alone
        float zero = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (full || uint32_t(i) < at.count) zero = fmaf(f[i], 0.0f, zero);
        const bool whole = __all_sync(0xffffffffu, zero == 0.0f && bias.plain && !bias.masks);
        if (!whole) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) numbers = numbers && f[i] < INFINITY;
            numbers = __all_sync(0xffffffffu, numbers);
        }
        if (!p.sigmoid) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) most = fmaxf(most, f[i]);
            most = route_top(most);
            if (!numbers) {
                bool nan = most == INFINITY;
#pragma unroll
                for (int i = 0; i < VPT; ++i) nan = nan || f[i] != f[i];
                bad = __any_sync(0xffffffffu, nan);
            }
            if (!p.by_logit || !p.renorm) {
                float c[VPT];
                const float from = most == -INFINITY ? 0.0f : most;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    c[i] = act::ex2((f[i] - from) * act::kLog2e);
                    sum += c[i];
                }
                sum = warp_sum(sum);
                const float over = act::rcp(sum);
                tol = (132.0f * over + 4.0f * bias.widest) * 0x1p-24f + (over + bias.widest) * float(Key::kMask + 1u) * 0x1p-23f;
                if (!p.by_logit) {
                    float b[VPT];
                    route_load_bias<VPT>(p, at, full, b);
#pragma unroll
                    for (int i = 0; i < VPT; ++i)  // (-infinity stays what it is)
                        f[i] = whole || f[i] != -INFINITY ? fmaf(c[i], over, b[i]) : f[i];
                }
            }
            if (bad) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (f[i] != -INFINITY) f[i] = __uint_as_float(0x7FC00000u);
            }
        } else if (!p.by_logit) {
            float b[VPT];
            route_load_bias<VPT>(p, at, full, b);
#pragma unroll
            for (int i = 0; i < VPT; ++i) f[i] = whole || f[i] != -INFINITY ? act::sigmoid(f[i]) + b[i] : f[i];
        }
        if (whole) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) key[i] = full || uint32_t(i) < at.count ? Key::finite(f[i], i) : 0u;
        } else {
            if (bias.masks) {  // (a score that is NaN would hide it)
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (uint32_t(i) < at.count && p.bias[at.first + i] == -INFINITY) f[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) key[i] = Key::any(f[i], i);
        }
    }
    r->most = most;
    r->sum = sum;
    r->bad = bad;
    route_sort<VPT>(key);
    bool again = false;  // with too many experts, or no numbers, the whole row goes in 64 bits
    if (p.groups > 1u) {
        uint32_t one = key[0], two = VPT > 1 ? key[VPT > 1 ? 1 : 0] : 0u;
        for (uint32_t d = at.lanes / 2u; d > 0u; d >>= 1) {
            const uint32_t o1 = __shfl_xor_sync(0xffffffffu, one, d);
            if (sums) two = max(min(one, o1), max(two, __shfl_xor_sync(0xffffffffu, two, d)));
            one = max(one, o1);
        }
        uint32_t score = one >> Key::kBits;
        if (sums && one != 0u) {
            const bool nan = score == 1u || (two >> Key::kBits) == 1u;
            score = nan ? 1u : route_key(Key::value(one) + (two != 0u ? Key::value(two) : 0.0f));
        }
        // a group's lanes compare it with every lanes-th of the others
        auto rank_of = [&](auto mine) {
            uint32_t rank = 0;
            for (uint32_t i = 0; i < p.groups; i += at.lanes) {
                const uint32_t g = i + (lane & (at.lanes - 1u));
                const auto o = __shfl_sync(0xffffffffu, mine, g << p.spread);
                rank += (g < p.groups && (o > mine || (o == mine && g < at.group))) ? 1u : 0u;
            }
            for (uint32_t d = at.lanes / 2u; d > 0u; d >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, d);
            return rank;
        };
        bool kept = rank_of(score) < p.top_groups;
        if (p.top_groups < p.groups && !exact_keys) {
            const uint32_t worst = __reduce_min_sync(0xffffffffu, kept ? score : 0xffffffffu);
            const uint32_t best = __reduce_max_sync(0xffffffffu, kept ? 0u : score);
            // (NaN and what cannot be chosen is no close call)
            bool close;
            if (p.by_logit) close = worst == best;
            else if (sums) close = !(route_value(worst) - route_value(best) > 2.0f * tol);
            else close = !(Key::value(worst << Key::kBits) - Key::value(best << Key::kBits) > tol);
            if (close && best > 1u) {
                // every group's score from those that may be its largest (two)
                const float least = Key::value(sums && two != 0u ? two : one) - (p.by_logit ? 0.0f : tol);
                int32_t own[3];
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    own[i] = (i < VPT && key[i % VPT] != 0u && Key::value(key[i % VPT]) >= least)
                                 ? int32_t(at.first + (Key::kMask - (key[i % VPT] & Key::kMask)))
                                 : -1;
                if (!numbers) again = true;
                else if (__any_sync(0xffffffffu, own[2] >= 0)) again = !route_even(p, row);
                else kept = route_rank64(p, row, most, sums, own[0], own[1]) < p.top_groups;
            }
        }
        if (!kept) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) key[i] = 0u;
        }
    }
    // The next largest key: the lowest lane that has its value puts it down as choice j and goes on to its own next.
    uint32_t now = key[0];
    uint32_t *next_key = keep + lane;
#pragma unroll
    for (int i = 1; i < VPT; ++i) keep[(i - 1) * 32 + lane] = key[i];
    keep[(VPT - 1) * 32 + lane] = 0u;  // (a lane without keys is never the one)
    const uint32_t below = (1u << lane) - 1u;
    auto take = [&](uint32_t j, uint32_t k) {
        const bool have = (now >> Key::kBits) == k;
        const uint32_t who = __ballot_sync(0xffffffffu, have);
        if (have && (who & below) == 0u) {
            pick[j] = make_uint2(now, at.first + (Key::kMask - (now & Key::kMask)));
            now = *next_key;
            next_key += 32;
        }
    };
    auto near = [&](uint32_t a, uint32_t b) {  // keys without their last bits, a >= b
        if (b <= 1u) return false;
        return p.by_logit ? a == b : !(Key::value(a << Key::kBits) - Key::value(b << Key::kBits) > tol);
    };
    // as many as are wanted, and those that may take the last one's place
    uint32_t rest = __reduce_max_sync(0xffffffffu, now >> Key::kBits), last = 0u, count = 0;
#pragma unroll 1
    while (rest != 0u && count < 32u) {
        if (count >= p.top && (exact_keys || !near(last, rest))) break;
        if (count < p.top) last = rest;
        take(count, rest);
        rest = __reduce_max_sync(0xffffffffu, now >> Key::kBits);
        ++count;
    }
    __syncwarp();
    const uint2 got = pick[lane];
    int32_t id = lane < count ? int32_t(got.y) : -1;
    if (!exact_keys) {
        const uint32_t mine = lane < count ? got.x >> Key::kBits : 0u;
        const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
        bool beside = lane + 1u < count && near(mine, next);
        const bool more = count == 32u && near(last, rest);  // others than those looked at may take the last one's place
        if (more || __any_sync(0xffffffffu, beside)) {
            // equal logits and biases are equal scores, and their order by index is right
            const int32_t after = __shfl_down_sync(0xffffffffu, id, 1);
            if (beside && route_same(p, row, id, after)) beside = false;
            if (more) again = again || !route_even(p, row);
            else if (__any_sync(0xffffffffu, beside) && numbers) id = route_order64(p, row, most, id, count);
            else again = again || __any_sync(0xffffffffu, beside);
        }
        if (again) id = route_exact<VPT>(p, row);
    }
    return lane < p.top ? id : -1;
}

// The choice of one row and its weights, stored.  Returns the id of choice `lane`.
template <int VPT>
__device__ __forceinline__ int32_t route_row(const RouteScoredParams &p, uint32_t row, const RouteLane &at, const RouteBias &bias,
                                             uint32_t *keep, uint2 *pick)
{
    const uint32_t lane = threadIdx.x & 31u;
    RouteRow r;
    const int32_t id = route_choose<VPT>(p, row, at, bias, keep, pick, &r);
    const float l = id >= 0 ? route_logit(p, size_t(row) * p.experts + id) : -INFINITY;
    float w = 0.0f, over = p.sigmoid ? 1.0f : r.sum;
    const float from = p.renorm ? route_top(l) : p.sigmoid ? 0.0f : r.most;
    if (id >= 0) w = p.sigmoid ? route_sigmoid(l, fminf(from, 0.0f)) : r.bad ? __uint_as_float(0x7FC00000u) : act::ex2((l - from) * act::kLog2e);
    if (p.renorm) over = warp_sum(w);
    w *= p.scale * act::rcp(over);
    if (lane < p.top) {
        p.ids[size_t(row) * p.top + lane] = id;
        p.weights[size_t(row) * p.top + lane] = id >= 0 ? w : 0.0f;
    }
    __syncwarp();  // (the picks are read)
    return id;
}

// Many rows: 32 to a block.
template <int VPT>
__global__ void __launch_bounds__(16 * kRouteRows, VPT <= 8 ? 2 : 1) route_scored_kernel(const __grid_constant__ RouteScoredParams p)
{
    constexpr int kThreads = 16 * kRouteRows;
    constexpr uint32_t kWarps = kThreads / 32;
    __shared__ uint32_t s_mask[2][kRouteMaxExperts];  // bit w: the block's row w, kWarps + w
    __shared__ int32_t s_base[kRouteMaxExperts];
    __shared__ int32_t s_scan[32];
    extern __shared__ __align__(8) uint8_t s_lists[];  // for each warp its picks (256 bytes) and keys (128 VPT)
    const uint32_t warp = threadIdx.x >> 5;
    for (uint32_t e = threadIdx.x; e < p.experts; e += kThreads) s_mask[0][e] = s_mask[1][e] = 0u;
    __syncthreads();
    ptx::griddep_wait();

    const RouteLane at(p);
    const uint32_t row0 = blockIdx.x * (2u * kWarps);
    const RouteBias bias(p, at);
    uint2 *pick = reinterpret_cast<uint2 *>(s_lists + warp * kRouteListBytes<VPT>);
    uint32_t *keep = reinterpret_cast<uint32_t *>(pick + 32);
    int32_t id0 = -1, id1 = -1;
#pragma unroll 1
    for (uint32_t q = 0; q < 2u; ++q) {
        const uint32_t row = row0 + warp + q * kWarps;
        if (row >= p.rows) break;  // (a whole warp)
        const int32_t id = route_row<VPT>(p, row, at, bias, keep, pick);
        if (id >= 0) atomicOr(&s_mask[q][id], 1u << warp);
        if (q == 0u) id0 = id;
        else id1 = id;
    }
    const int32_t id[2] = {id0, id1};
    route_rank<kThreads>(p, row0, id, s_mask, s_base, s_scan);
    ptx::griddep_launch_dependents();
}

// Few rows: a cluster of CTAs, each with a row for each of its warps, that read one another's masks and so all know the
// counts.  (64 rows of 256 experts on one SM took 12.4 us, of 1024 72.6.)
constexpr int kRouteFewThreads = 256;
constexpr int kRouteFewPer = kRouteFewThreads / 32;  // rows of a CTA
constexpr int kRouteFewCtas = kRouteFewRows / kRouteFewPer;
static_assert(kRouteFewCtas <= 8, "a portable cluster");

template <int VPT>
__global__ void __launch_bounds__(kRouteFewThreads) route_scored_few_kernel(const __grid_constant__ RouteScoredParams p)
{
    constexpr uint32_t kMost = kRouteMaxExperts / kRouteFewThreads;  // experts of a thread, at most
    __shared__ uint32_t s_mask[kRouteMaxExperts];  // bit w: the CTA's row w
    __shared__ int32_t s_base[kRouteMaxExperts];
    __shared__ int32_t s_scan[kRouteFewPer];
    extern __shared__ __align__(8) uint8_t s_lists[];  // as above
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, cta = blockIdx.x, ctas = gridDim.x;  // (one cluster)
    for (uint32_t e = threadIdx.x; e < p.experts; e += kRouteFewThreads) s_mask[e] = 0u;
    __syncthreads();
    ptx::griddep_wait();

    const uint32_t row = cta * kRouteFewPer + warp;
    int32_t id = -1;
    if (row < p.rows) {
        const RouteLane at(p);
        const RouteBias bias(p, at);
        uint2 *pick = reinterpret_cast<uint2 *>(s_lists + warp * kRouteListBytes<VPT>);
        id = route_row<VPT>(p, row, at, bias, reinterpret_cast<uint32_t *>(pick + 32), pick);
        if (id >= 0) atomicOr(&s_mask[id], 1u << warp);
    }
    if (ctas > 1u) ptx::cluster_sync();
    else __syncthreads();
    // a thread's experts are neighbours: the rows of all CTAs that chose them, and those of the CTAs before this one
    const uint32_t per = (p.experts + kRouteFewThreads - 1u) / kRouteFewThreads, first = threadIdx.x * per;
    int32_t count[kMost], before[kMost], sum = 0;
#pragma unroll
    for (uint32_t i = 0; i < kMost; ++i) {
        count[i] = before[i] = 0;
        if (i >= per || first + i >= p.experts) continue;
        const uint32_t mine = ptx::smem_addr(&s_mask[first + i]);
        for (uint32_t c = 0; c < ctas; ++c) {
            const int32_t n = __popc(c == cta ? s_mask[first + i] : ptx::ld_shared_cluster_u32(ptx::map_to_rank(mine, c)));
            count[i] += n;
            before[i] += c < cta ? n : 0;
        }
        sum += count[i];
    }
    int32_t x = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= uint32_t(d)) x += o;
    }
    if (lane == 31u) s_scan[warp] = x;
    __syncthreads();
    int32_t start = x - sum, total = 0;
#pragma unroll
    for (uint32_t w = 0; w < uint32_t(kRouteFewPer); ++w) {
        if (w < warp) start += s_scan[w];
        total += s_scan[w];
    }
#pragma unroll
    for (uint32_t i = 0; i < kMost; ++i) {
        if (i >= per || first + i >= p.experts) continue;
        s_base[first + i] = start + before[i];
        if (cta == 0u) p.offsets[first + i] = start;
        start += count[i];
    }
    if (cta == 0u && threadIdx.x == 0u) p.offsets[p.experts] = total;
    for (uint32_t i = uint32_t(total) + cta * kRouteFewThreads + threadIdx.x; i < p.rows * p.top; i += ctas * kRouteFewThreads) p.order[i] = -1;
    __syncthreads();
    if (row < p.rows && lane < p.top) {
        const uint32_t flat = row * p.top + lane;
        int32_t at = -1;
        if (id >= 0) {
            at = s_base[id] + __popc(s_mask[id] & ((1u << warp) - 1u));
            p.order[at] = int32_t(flat);
        }
        p.position[flat] = at;
    }
    ptx::griddep_launch_dependents();
    if (ctas > 1u) ptx::cluster_sync();  // (the masks are read)
}

// A row's logits as the gradient's kernel takes them: four neighbours to a lane, or (fours false) `lane`, 32 + lane, ...
template <int VPT>
__device__ __forceinline__ void route_load_grad(const RouteScoredParams &p, size_t row, bool fours, float (&f)[VPT])
{
    if (VPT < 4 || !fours) {
        route_load<VPT>(p.logits, p.dtype, row, p.experts, true, f);
        return;
    }
    const uint32_t lane = threadIdx.x & 31u;
#pragma unroll
    for (int i = 0; i < VPT / 4; ++i) {
        const uint32_t e = 4u * (uint32_t(i) * 32u + lane);
        const bool have = e < p.experts;
        if (p.dtype == 2u) {
            const float4 v = have ? *reinterpret_cast<const float4 *>(static_cast<const float *>(p.logits) + row * p.experts + e)
                                  : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            f[4 * i] = v.x;
            f[4 * i + 1] = v.y;
            f[4 * i + 2] = v.z;
            f[4 * i + 3] = v.w;
        } else {
            const uint32_t none = p.dtype == 1u ? 0xFF80FF80u : 0xFC00FC00u;
            const uint2 v = have ? *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.logits) + row * p.experts + e)
                                 : make_uint2(none, none);
            const float2 a = ragged_unpack(v.x, p.dtype == 1u), b = ragged_unpack(v.y, p.dtype == 1u);
            f[4 * i] = a.x;
            f[4 * i + 1] = a.y;
            f[4 * i + 2] = b.x;
            f[4 * i + 3] = b.y;
        }
    }
}

// Gradient of the logits; ids outside [0, experts) take no part.
//   sigmoid   dl_j = scale s_j (1 - s_j) dw_j, or with renorm, v = s / (sum of the chosen s),
//             scale v_j (1 - s_j) (dw_j - sum_i v_i dw_i)
//   softmax   dl = scale s (dw - sum_i s_i dw_i), with renorm the same of v, for the chosen ones alone
// A warp takes two rows side by side up to 256 experts, and four neighbouring experts to a lane where they come in fours
// (16384 rows, 256 experts: 11.1 us with one row and one expert).
template <int VPT>
__global__ void __launch_bounds__(256) route_scored_grad_kernel(const __grid_constant__ RouteScoredParams p)
{
    constexpr int kRows = VPT <= 8 ? 2 : 1, kQuads = VPT >= 4 ? VPT / 4 : 1;
    __shared__ __align__(16) float s_row[8 * kRows * VPT * 32];
    ptx::griddep_wait();
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const bool all = !p.sigmoid && !p.renorm;  // every expert's logit has a gradient
    const bool fours = VPT >= 4 && p.experts % 4u == 0u && (reinterpret_cast<uintptr_t>(p.dlogits) & 15u) == 0u;
    int32_t id[kRows];
    float dw[kRows], l[kRows];
    uint32_t row[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
        row[q] = (blockIdx.x * 8u + warp) * uint32_t(kRows) + uint32_t(q);
        const bool have = row[q] < p.rows && lane < p.top;
        id[q] = have ? p.ids[size_t(row[q]) * p.top + lane] : -1;
        dw[q] = have ? p.scale * p.dweights[size_t(row[q]) * p.top + lane] : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
        if (uint32_t(id[q]) >= p.experts) id[q] = -1;
        l[q] = id[q] >= 0 ? route_logit(p, size_t(row[q]) * p.experts + id[q]) : -INFINITY;
        if (id[q] < 0) dw[q] = 0.0f;
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
        float *mine = s_row + (warp * kRows + q) * (VPT * 32);
        if (VPT >= 4) {
#pragma unroll
            for (int i = 0; i < kQuads; ++i) reinterpret_cast<float4 *>(mine)[i * 32 + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) mine[i * 32 + lane] = 0.0f;
        }
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
        if (row[q] >= p.rows) break;  // (a whole warp)
        float *mine = s_row + (warp * kRows + q) * (VPT * 32);
        float f[VPT];
        float d = dw[q], inner = 0.0f, over = 0.0f;  // over: 1 / the sum of a row's exponentials
        if (p.sigmoid || p.renorm) {
            float w = 1.0f;  // the score, or with renorm its share
            if (p.renorm) {
                const float top = route_top(l[q]);
                w = id[q] < 0 ? 0.0f : p.sigmoid ? route_sigmoid(l[q], fminf(top, 0.0f)) : act::ex2((l[q] - top) * act::kLog2e);
                w *= act::rcp(warp_sum(w));
                inner = warp_sum(id[q] >= 0 ? w * dw[q] : 0.0f);
            } else if (id[q] >= 0) {
                w = route_sigmoid(l[q], 0.0f);
            }
            d = id[q] < 0 ? 0.0f : w * (d - inner);
            if (p.sigmoid) d *= route_sigmoid(-l[q], 0.0f);  // 1 - s
        } else {
            route_load_grad<VPT>(p, row[q], fours, f);
            float most = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) most = fmaxf(most, f[i]);
            most = route_top(most);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                f[i] = f[i] == -INFINITY ? 0.0f : act::ex2((f[i] - most) * act::kLog2e);
                sum += f[i];
            }
            sum = warp_sum(sum);
            over = sum == 0.0f ? 0.0f : act::rcp(sum);  // (a row with every expert at -infinity has no gradient)
            inner = warp_sum(id[q] >= 0 ? act::ex2((l[q] - most) * act::kLog2e) * over * d : 0.0f);
        }
        // the same expert twice: its gradients add up, in the order of the choices
        const uint32_t peers = __match_any_sync(0xffffffffu, id[q]);
        if (__any_sync(0xffffffffu, id[q] >= 0 && (peers & (peers - 1u)) != 0u)) {
            float together = 0.0f;
            for (uint32_t j = 0; j < p.top; ++j) {
                const float o = __shfl_sync(0xffffffffu, d, j);
                if ((peers >> j) & 1u) together += o;
            }
            d = together;
        }
        __syncwarp();
        if (id[q] >= 0) mine[id[q]] = d;
        __syncwarp();
        float *out = p.dlogits + size_t(row[q]) * p.experts;
        if (fours) {
#pragma unroll
            for (int i = 0; i < kQuads; ++i) {
                const uint32_t e = 4u * (uint32_t(i) * 32u + lane);
                if (e >= p.experts) continue;
                float4 v = reinterpret_cast<const float4 *>(mine)[i * 32 + lane];
                if (all) {
                    v.x = f[(4 * i) % VPT] * over * (v.x - inner);
                    v.y = f[(4 * i + 1) % VPT] * over * (v.y - inner);
                    v.z = f[(4 * i + 2) % VPT] * over * (v.z - inner);
                    v.w = f[(4 * i + 3) % VPT] * over * (v.w - inner);
                }
                *reinterpret_cast<float4 *>(out + e) = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const uint32_t e = uint32_t(i) * 32u + lane;
                if (e >= p.experts) continue;
                const float v = mine[i * 32 + lane];
                out[e] = all ? f[i] * over * (v - inner) : v;
            }
        }
    }
    ptx::griddep_launch_dependents();
}

}  // namespace gemm_f16
