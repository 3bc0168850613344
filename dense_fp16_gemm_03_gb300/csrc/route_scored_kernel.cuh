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
// Bound by issued instructions, as the top-k router.
#pragma once

#include "gemm_ragged.h"
#include "linear_act.cuh"
#include "route_kernel.cuh"

namespace gemm_f16 {

struct RouteScoredParams : RouteParams {
    const float *bias;     // [experts], or null
    uint32_t sigmoid;      // else softmax
    uint32_t groups, top_groups, group_top;
    uint32_t size;         // experts of a group
    uint32_t run;          // experts of a lane
    uint32_t by_logit;     // c has the logits' order
    float scale;
};

// Which experts a lane has: [first, first + count).
struct RouteLane {
    uint32_t lanes, group, first, count;
    __device__ __forceinline__ explicit RouteLane(const RouteScoredParams &p)
    {
        const uint32_t lane = threadIdx.x & 31u;
        lanes = 32u / p.groups;
        group = lane / lanes;
        const uint32_t from = (lane - group * lanes) * p.run;
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
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        f[i] = p.dtype == 1u ? __uint_as_float(raw[i] << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(raw[i])));
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
        double v = p.sigmoid ? 1.0 / (1.0 + exp(-c[i])) : exp(c[i] - double(most)) / sum;
        if (!p.sigmoid && bad) v = NAN;
        if (p.bias) v += double(p.bias[at.first + i]);
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
    return l < 0.0f ? expf(l - from) / (1.0f + expf(l)) : 1.0f / (1.0f + expf(-l));
}

// Whether two experts of a row have the same logit and the same bias, and with them the same c.
__device__ __forceinline__ bool route_same(const RouteScoredParams &p, size_t row, int32_t a, int32_t b)
{
    return route_logit(p, row * p.experts + a) == route_logit(p, row * p.experts + b) && (!p.bias || p.bias[a] == p.bias[b]);
}

template <int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS) route_scored_kernel(const __grid_constant__ RouteScoredParams p)
{
    constexpr uint32_t kWarps = THREADS / 32;
    __shared__ uint32_t s_mask[2][kRouteMaxExperts];  // bit w: the block's row w, kWarps + w
    __shared__ int32_t s_base[kRouteMaxExperts];
    __shared__ int32_t s_scan[32];
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    for (uint32_t e = threadIdx.x; e < p.experts; e += THREADS) s_mask[0][e] = s_mask[1][e] = 0u;
    __syncthreads();
    ptx::griddep_wait();

    const RouteLane at(p);
    const uint32_t row0 = blockIdx.x * (2u * kWarps);
    const bool sums = p.groups > 1u && p.group_top == 2u;
    float bias[VPT], widest = 0.0f;  // the largest of the finite biases' magnitudes
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        bias[i] = (p.bias && uint32_t(i) < at.count) ? p.bias[at.first + i] : 0.0f;
        if (fabsf(bias[i]) < INFINITY) widest = fmaxf(widest, fabsf(bias[i]));
    }
    widest = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(widest)));

    int32_t id[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint32_t row = row0 + warp + uint32_t(q) * kWarps;
        const bool live = row < p.rows;
        id[q] = -1;
        if (!live) continue;  // (a whole warp)
        float f[VPT], c[VPT];
        route_load_run<VPT>(p, row, at, live, f);
        float most = -INFINITY, sum = 0.0f, tol = (16.0f + 4.0f * widest) * 0x1p-24f;
        bool bad = false;  // a softmax of NaN or +infinity: every score is NaN
        if (!p.sigmoid) {
            bool nan = false;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                most = fmaxf(most, f[i]);
                nan = nan || f[i] != f[i];
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
            bad = __any_sync(0xffffffffu, nan) || most == INFINITY;
            if (!p.by_logit || !p.renorm) {
                const float from = most == -INFINITY ? 0.0f : most;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    c[i] = act::ex2((f[i] - from) * act::kLog2e);
                    sum += c[i];
                }
                sum = warp_sum(sum);
                const float over = act::rcp(sum);
                tol = (132.0f * over + 4.0f * widest) * 0x1p-24f;
#pragma unroll
                for (int i = 0; i < VPT; ++i) c[i] *= over;
            }
        } else if (!p.by_logit) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) c[i] = act::sigmoid(f[i]);
        }
        uint32_t key[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const float v = bad ? __uint_as_float(0x7FC00000u) : p.by_logit ? f[i] : c[i] + bias[i];
            key[i] = f[i] == -INFINITY ? 0u : route_key(v);
        }
        bool close = false;
        if (p.groups > 1u) {
            uint32_t one = 0u, two = 0u;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                two = max(two, min(one, key[i]));
                one = max(one, key[i]);
            }
            for (uint32_t d = at.lanes / 2u; d > 0u; d >>= 1) {
                const uint32_t o1 = __shfl_xor_sync(0xffffffffu, one, d);
                if (sums) two = max(min(one, o1), max(two, __shfl_xor_sync(0xffffffffu, two, d)));
                one = max(one, o1);
            }
            uint32_t score = one;
            if (sums && two != 0u) score = route_key(route_value(one) + route_value(two));
            uint32_t rank = 0;
            for (uint32_t g = 0; g < p.groups; ++g) {
                const uint32_t o = __shfl_sync(0xffffffffu, score, g * at.lanes);
                rank += (o > score || (o == score && g < at.group)) ? 1u : 0u;
            }
            const bool kept = rank < p.top_groups;
            if (p.top_groups < p.groups && !p.by_logit) {
                const uint32_t worst = __reduce_min_sync(0xffffffffu, kept ? score : 0xffffffffu);
                const uint32_t best = __reduce_max_sync(0xffffffffu, kept ? 0u : score);
                // (NaN and what cannot be chosen is no close call)
                close = best > 1u && !(route_value(worst) - route_value(best) > 2.0f * tol);
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (!kept) key[i] = 0u;
        }
        // the largest key of the lane, and where it is
        uint32_t best = 0u, spot = 0u;
        auto look = [&]() {
            best = 0u;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (key[i] > best) {
                    best = key[i];
                    spot = uint32_t(i);
                }
        };
        look();
        uint32_t mine = 0u;  // key of choice `lane`
        for (uint32_t j = 0; j < p.top; ++j) {
            const uint32_t k = __reduce_max_sync(0xffffffffu, best);
            if (k == 0u) break;
            const uint32_t e = __reduce_min_sync(0xffffffffu, best == k ? at.first + spot : 0xffffffffu);
            if (lane == j) {
                mine = k;
                id[q] = int32_t(e);
            }
            if (best == k && at.first + spot == e) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (uint32_t(i) == spot) key[i] = 0u;
                look();
            }
        }
        if (!p.by_logit) {
            const uint32_t rest = __reduce_max_sync(0xffffffffu, best);
            uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
            if (lane + 1u == p.top) next = rest;
            bool near = lane < p.top && next > 1u && !(route_value(mine) - route_value(next) > tol);
            if (__any_sync(0xffffffffu, near)) {
                // equal logits and biases are equal scores, and their order by index is right
                const uint32_t other = __reduce_min_sync(0xffffffffu, best == rest ? at.first + spot : 0xffffffffu);
                int32_t after = __shfl_down_sync(0xffffffffu, id[q], 1);
                if (lane + 1u == p.top) after = int32_t(other);
                if (near && mine == next && route_same(p, row, id[q], after)) near = false;
                close = close || __any_sync(0xffffffffu, near);
            }
            if (close) id[q] = route_exact<VPT>(p, row);
        }
        // weights, from the chosen logits
        const float l = id[q] >= 0 ? route_logit(p, size_t(row) * p.experts + id[q]) : -INFINITY;
        float w = 0.0f, over = p.sigmoid ? 1.0f : sum;
        const float from = p.renorm ? route_top(l) : p.sigmoid ? 0.0f : most;
        if (id[q] >= 0) w = p.sigmoid ? route_sigmoid(l, fminf(from, 0.0f)) : bad ? __uint_as_float(0x7FC00000u) : expf(l - from);
        if (p.renorm) over = warp_sum(w);
        w = p.scale * (w / over);
        if (lane < p.top) {
            p.ids[size_t(row) * p.top + lane] = id[q];
            p.weights[size_t(row) * p.top + lane] = id[q] >= 0 ? w : 0.0f;
            if (id[q] >= 0) atomicOr(&s_mask[q][id[q]], 1u << warp);
        }
    }
    route_rank<THREADS>(p, row0, id, s_mask, s_base, s_scan);
    ptx::griddep_launch_dependents();
}

// Gradient of the logits, one warp per row; ids outside [0, experts) take no part.
//   sigmoid   dl_j = scale s_j (1 - s_j) dw_j, or with renorm, v = s / (sum of the chosen s),
//             scale v_j (1 - s_j) (dw_j - sum_i v_i dw_i)
//   softmax   dl = scale s (dw - sum_i s_i dw_i), with renorm the same of v, for the chosen ones alone
template <int VPT>
__global__ void __launch_bounds__(256) route_scored_grad_kernel(const __grid_constant__ RouteScoredParams p)
{
    __shared__ float s_row[8 * VPT * 32];
    ptx::griddep_wait();
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t row = blockIdx.x * 8u + (threadIdx.x >> 5);
    if (row < p.rows) {
        int32_t id = lane < p.top ? p.ids[size_t(row) * p.top + lane] : -1;
        if (uint32_t(id) >= p.experts) id = -1;
        const bool all = !p.sigmoid && !p.renorm;  // every expert's logit has a gradient
        const float dw = id >= 0 ? p.scale * p.dweights[size_t(row) * p.top + lane] : 0.0f;
        const float l = id >= 0 ? route_logit(p, size_t(row) * p.experts + id) : -INFINITY;
        float f[VPT];
        if (all) route_load<VPT>(p.logits, p.dtype, row, p.experts, true, f);
        float *mine = s_row + (threadIdx.x >> 5) * (VPT * 32);
#pragma unroll
        for (int i = 0; i < VPT; ++i) mine[i * 32 + lane] = 0.0f;
        float d = dw, inner = 0.0f, sum = 0.0f;
        if (p.sigmoid || p.renorm) {
            float w = 1.0f;  // the score, or with renorm its share
            if (p.renorm) {
                const float top = route_top(l);
                w = id < 0 ? 0.0f : p.sigmoid ? route_sigmoid(l, fminf(top, 0.0f)) : expf(l - top);
                w /= warp_sum(w);
                inner = warp_sum(id >= 0 ? w * dw : 0.0f);
            } else if (id >= 0) {
                w = route_sigmoid(l, 0.0f);
            }
            d = id < 0 ? 0.0f : w * (dw - inner);
            if (p.sigmoid) d *= l < 0.0f ? 1.0f / (1.0f + expf(l)) : route_sigmoid(-l, 0.0f);  // 1 - s
        } else {
            float most = -INFINITY;
#pragma unroll
            for (int i = 0; i < VPT; ++i) most = fmaxf(most, f[i]);
            most = route_top(most);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                f[i] = f[i] == -INFINITY ? 0.0f : expf(f[i] - most);
                sum += f[i];
            }
            sum = warp_sum(sum);
            inner = warp_sum(id >= 0 ? expf(l - most) / sum * dw : 0.0f);
        }
        // the same expert twice: its gradients add up, in the order of the choices
        const uint32_t peers = __match_any_sync(0xffffffffu, id);
        if (__any_sync(0xffffffffu, id >= 0 && (peers & (peers - 1u)) != 0u)) {
            float together = 0.0f;
            for (uint32_t j = 0; j < p.top; ++j) {
                const float o = __shfl_sync(0xffffffffu, d, j);
                if ((peers >> j) & 1u) together += o;
            }
            d = together;
        }
        __syncwarp();
        if (id >= 0) mine[id] = d;
        __syncwarp();
        float *out = p.dlogits + size_t(row) * p.experts;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t e = uint32_t(i) * 32u + lane;
            if (e >= p.experts) continue;
            const float v = mine[i * 32 + lane];
            // (a row with every expert at -infinity has no gradient)
            out[e] = !all ? v : sum == 0.0f ? 0.0f : f[i] / sum * (v - inner);
        }
    }
    ptx::griddep_launch_dependents();
}

}  // namespace gemm_f16
