// The experts' router: top-k of every row's logits, softmax weights, and the
// rows sorted by expert (offsets, order, position) as the grouped products
// take them; and the gradient of the logits.
//
// One warp per row: the row's logits live in registers (VPT per lane) as keys
// whose unsigned order is the floats' order, so one step of the choice is a
// register maximum, a warp maximum of the key and a warp minimum of the index
// (ties to the lowest).  Which rows of a block chose an expert is two 32-bit
// masks in shared memory, so a choice's rank among the block's rows is a
// population count, independent of the order in which the warps set the bits.
// One block of 64 rows does everything in one launch; more rows go 32 to a
// block, and route_place_kernel turns the ranks into positions with the counts
// of the blocks before, which it sums itself for few blocks (every block sums
// them again: 512 blocks of 128 experts took 18.7 us) and finds summed by
// route_scan_kernel otherwise (3.5 and 5.3 us).
//
// Bound by latency for few rows (64 rows, 64 experts, 8 choices: 5.5 us) and by
// issued instructions for many (16384 rows, 128 experts: 12 us for the choice,
// some 300 instructions a row, where its bytes take 1; 25 us with the placing and
// the gradient).  Loads in a lane's own order before any conversion, keys sorted
// in the lane up to 128 experts, and two rows of a warp side by side brought the
// choice from 19 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace gemm_f16 {

// A block's rows, two for each of its warps (the bits of two masks).  Up to kRouteFewRows rows one block does
// everything; more go 32 to a block, which keeps more warps on an SM.
constexpr int kRouteFewRows = 64;
constexpr int kRouteRows = 32;
constexpr int kRouteThreads = 1024;  // of the block for few rows, and of the kernels that place rows
constexpr int kRouteDirectBlocks = 32;  // up to so many blocks each one sums the counts before it by itself
constexpr int kRouteMaxExperts = 1024;

struct RouteParams {
    const void *logits;
    uint32_t dtype;  // 0 fp16, 1 bf16, 2 fp32
    uint32_t rows, experts, top, renorm, blocks;
    int32_t *ids;
    float *weights;
    int32_t *offsets, *order, *position;
    int32_t *hist;    // [blocks, experts]: a block's rows per expert, then (scanned) those of the blocks before it
    int32_t *totals;  // [experts]
    const float *dweights;
    float *dlogits;
};

// A row's logits, `lane`, 32 + lane, ... (-infinity past the last): all loads before the first conversion.
template <int VPT>
__device__ __forceinline__ void route_load(const void *base, uint32_t dtype, size_t row, uint32_t experts, bool live,
                                           float (&f)[VPT])
{
    const uint32_t lane = threadIdx.x & 31u;
    if (dtype == 2u) {
        const float *p = static_cast<const float *>(base) + row * experts + lane;
#pragma unroll
        for (int i = 0; i < VPT; ++i) f[i] = (live && uint32_t(i) * 32u + lane < experts) ? p[i * 32] : -INFINITY;
        return;
    }
    const uint16_t *p = static_cast<const uint16_t *>(base) + row * experts + lane;
    const uint32_t none = dtype == 1u ? 0xFF80u : 0xFC00u;  // -infinity
    uint32_t raw[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) raw[i] = (live && uint32_t(i) * 32u + lane < experts) ? uint32_t(p[i * 32]) : none;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        f[i] = dtype == 1u ? __uint_as_float(raw[i] << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(raw[i])));
}

// Unsigned order = float order; -0 counts as +0.  0: never chosen (-infinity), 1: NaN.
__device__ __forceinline__ uint32_t route_key(float f)
{
    if (f != f) return 1u;
    const uint32_t u = __float_as_uint(f + 0.0f);
    if (u == 0xFF800000u) return 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float route_value(uint32_t key)
{
    if (key == 1u) return __uint_as_float(0x7FC00000u);
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Exclusive prefix sum over a block of 1024 threads; `s` holds 32 words.  *total gets the whole sum.
__device__ __forceinline__ int32_t route_block_scan(int32_t v, int32_t *s, int32_t *total)
{
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    int32_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= uint32_t(d)) x += o;
    }
    __syncthreads();
    if (lane == 31u) s[warp] = x;
    __syncthreads();
    int32_t w = s[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= uint32_t(d)) w += o;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int32_t before = __shfl_sync(0xffffffffu, w, warp ? warp - 1u : 0u);
    return x - v + (warp ? before : 0);
}

template <int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS) route_topk_kernel(const __grid_constant__ RouteParams p)
{
    constexpr uint32_t kWarps = THREADS / 32;
    __shared__ uint32_t s_mask[2][kRouteMaxExperts];  // bit w: the block's row w, kWarps + w
    __shared__ int32_t s_base[kRouteMaxExperts];
    __shared__ int32_t s_scan[32];
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    for (uint32_t e = threadIdx.x; e < p.experts; e += THREADS) s_mask[0][e] = s_mask[1][e] = 0u;
    __syncthreads();
    ptx::griddep_wait();

    // A warp's two rows go through the choice side by side where their keys fit the registers: a step is a
    // chain of warp reductions, and the other row's fills its gaps.
    constexpr int kRowsPerWarp = 2;
    constexpr int kTogether = VPT <= 8 ? kRowsPerWarp : 1;
    constexpr bool kSort = VPT <= 4;  // (28 exchanges for eight keys are more than they spare)
    int32_t id[kRowsPerWarp];
    const uint32_t row0 = blockIdx.x * (2u * kWarps);
#pragma unroll
    for (int q0 = 0; q0 < kRowsPerWarp; q0 += kTogether) {
        uint32_t key[kTogether][VPT], mine[kTogether];
        float f[kTogether][VPT], top_value[kTogether], sum[kTogether];
        bool live[kTogether];
#pragma unroll
        for (int q = 0; q < kTogether; ++q) {
            const uint32_t row = row0 + warp + uint32_t(q0 + q) * kWarps;
            live[q] = row < p.rows;
            id[q0 + q] = -1;
            mine[q] = 0u;  // key of choice `lane`
            top_value[q] = -INFINITY;
            route_load<VPT>(p.logits, p.dtype, row, p.experts, live[q], f[q]);
        }
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                key[q][i] = route_key(f[q][i]);
                top_value[q] = fmaxf(top_value[q], f[q][i]);
            }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
#pragma unroll
            for (int q = 0; q < kTogether; ++q)
                top_value[q] = fmaxf(top_value[q], __shfl_xor_sync(0xffffffffu, top_value[q], d));
#pragma unroll
        for (int q = 0; q < kTogether; ++q) {
            sum[q] = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (key[q][i]) sum[q] += expf(f[q][i] - top_value[q]);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
#pragma unroll
            for (int q = 0; q < kTogether; ++q) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], d);
        // A lane's keys in falling order, equal ones by rising index: a step then looks at the first alone.
        uint32_t slot[kTogether][kSort ? VPT : 1];
        if constexpr (kSort) {
#pragma unroll
            for (int q = 0; q < kTogether; ++q) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) slot[q][i] = uint32_t(i) * 32u + lane;
#pragma unroll
                for (int end = VPT - 1; end > 0; --end)
#pragma unroll
                    for (int i = 0; i < end; ++i)
                        if (key[q][i + 1] > key[q][i]) {
                            const uint32_t k = key[q][i], a = slot[q][i];
                            key[q][i] = key[q][i + 1];
                            slot[q][i] = slot[q][i + 1];
                            key[q][i + 1] = k;
                            slot[q][i + 1] = a;
                        }
            }
        }
        for (uint32_t j = 0; j < p.top; ++j) {
            uint32_t best[kTogether], at[kTogether], k[kTogether], e[kTogether];
#pragma unroll
            for (int q = 0; q < kTogether; ++q) {
                if constexpr (kSort) {
                    best[q] = key[q][0];
                    at[q] = slot[q][0];
                } else {
                    best[q] = at[q] = 0u;
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        if (key[q][i] > best[q]) {
                            best[q] = key[q][i];
                            at[q] = uint32_t(i) * 32u + lane;
                        }
                }
                k[q] = __reduce_max_sync(0xffffffffu, best[q]);
            }
#pragma unroll
            for (int q = 0; q < kTogether; ++q)
                e[q] = __reduce_min_sync(0xffffffffu, best[q] == k[q] ? at[q] : 0xffffffffu);
#pragma unroll
            for (int q = 0; q < kTogether; ++q) {
                // (k = 0: only experts at -infinity are left, nothing to take)
                if (at[q] == e[q]) {
                    if constexpr (kSort) {
#pragma unroll
                        for (int i = 0; i + 1 < VPT; ++i) {
                            key[q][i] = key[q][i + 1];
                            slot[q][i] = slot[q][i + 1];
                        }
                        key[q][VPT - 1] = 0u;
                    } else {
#pragma unroll
                        for (int i = 0; i < VPT; ++i)
                            if (uint32_t(i) == (e[q] >> 5)) key[q][i] = 0u;
                    }
                }
                if (lane == j && k[q] != 0u) {
                    mine[q] = k[q];
                    id[q0 + q] = int32_t(e[q]);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < kTogether; ++q) {
            const uint32_t row = row0 + warp + uint32_t(q0 + q) * kWarps;
            float w = mine[q] ? expf(route_value(mine[q]) - top_value[q]) : 0.0f;
            const float chosen = warp_sum(w);
            // (a NaN anywhere in the row shows in every weight, chosen or not)
            if (p.renorm && sum[q] == sum[q]) sum[q] = chosen;
            w = mine[q] ? w / sum[q] : 0.0f;
            if (live[q] && lane < p.top) {
                p.ids[size_t(row) * p.top + lane] = id[q0 + q];
                p.weights[size_t(row) * p.top + lane] = w;
                if (id[q0 + q] >= 0) atomicOr(&s_mask[q0 + q][id[q0 + q]], 1u << warp);
            }
        }
    }
    __syncthreads();
    const uint32_t t = threadIdx.x;
    if (THREADS < kRouteThreads || p.blocks > 1u) {
        for (uint32_t e = t; e < p.experts; e += THREADS)
            p.hist[size_t(blockIdx.x) * p.experts + e] = __popc(s_mask[0][e]) + __popc(s_mask[1][e]);
    } else {
        const int32_t count = t < p.experts ? __popc(s_mask[0][t]) + __popc(s_mask[1][t]) : 0;
        int32_t total;
        const int32_t before = route_block_scan(count, s_scan, &total);
        if (t < p.experts) {
            s_base[t] = before;
            p.offsets[t] = before;
        }
        if (t == 0) p.offsets[p.experts] = total;
        for (uint32_t i = uint32_t(total) + t; i < p.rows * p.top; i += THREADS) p.order[i] = -1;
        __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < kRowsPerWarp; ++q) {
        const uint32_t row = row0 + warp + uint32_t(q) * kWarps;
        if (row >= p.rows || lane >= p.top) continue;
        const size_t flat = size_t(row) * p.top + lane;
        int32_t at = -1;
        if (id[q] >= 0) {
            // the block's rows before this one that chose the same expert (rows of this warp: r = warp, 32 + warp)
            at = __popc(s_mask[q][id[q]] & ((1u << warp) - 1u)) + (q ? __popc(s_mask[0][id[q]]) : 0);
            if (p.blocks == 1u) {
                at += s_base[id[q]];
                p.order[at] = int32_t(flat);
            }
        }
        p.position[flat] = at;  // more blocks: the rank in this block, completed by route_place_kernel
    }
    ptx::griddep_launch_dependents();
}

// Counts of 32 experts a block, over all blocks of route_topk_kernel: hist becomes the exclusive prefix over
// the blocks, totals the sum.  32 x 32 threads: threadIdx.y takes a run of blocks.
__global__ void __launch_bounds__(1024) route_scan_kernel(const __grid_constant__ RouteParams p)
{
    __shared__ int32_t s_sum[32][33];
    ptx::griddep_wait();
    const uint32_t lane = threadIdx.x & 31u, part = threadIdx.x >> 5;
    const uint32_t e = blockIdx.x * 32u + lane;
    const uint32_t each = (p.blocks + 31u) / 32u;
    const uint32_t lo = min(part * each, p.blocks), hi = min(lo + each, p.blocks);
    int32_t sum = 0;
    if (e < p.experts)
        for (uint32_t b = lo; b < hi; ++b) sum += p.hist[size_t(b) * p.experts + e];
    s_sum[part][lane] = sum;
    __syncthreads();
    int32_t x = s_sum[lane][part];  // this warp scans the parts of expert `part` of the block
    const int32_t v = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= uint32_t(d)) x += o;
    }
    s_sum[lane][part] = x - v;
    if (lane == 31u && blockIdx.x * 32u + part < p.experts) p.totals[blockIdx.x * 32u + part] = x;
    __syncthreads();
    int32_t before = s_sum[part][lane];
    if (e < p.experts)
        for (uint32_t b = lo; b < hi; ++b) {
            int32_t *at = p.hist + size_t(b) * p.experts + e;
            const int32_t c = *at;
            *at = before;
            before += c;
        }
    ptx::griddep_launch_dependents();
}

// Positions of one block's choices from their ranks, the blocks' prefixes and the experts' totals.
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const __grid_constant__ RouteParams p)
{
    __shared__ int32_t s_base[kRouteMaxExperts];
    __shared__ int32_t s_scan[32];
    __shared__ int2 s_part[kRouteThreads];
    ptx::griddep_wait();
    const uint32_t t = threadIdx.x;
    int32_t count = 0, prefix = 0;  // of expert t: all its rows, and those of the blocks before this one
    if (p.blocks <= kRouteDirectBlocks) {
        // `lanes` threads to an expert, each sums every lanes-th block; then one adds them up
        uint32_t lanes = kRouteThreads / p.experts;
        lanes = lanes > 32u ? 32u : lanes;
        const uint32_t e = t % p.experts, part = t / p.experts;
        int32_t a = 0, b = 0;
        if (part < lanes) {
#pragma unroll 8
            for (uint32_t i = part; i < p.blocks; i += lanes) {
                const int32_t c = p.hist[size_t(i) * p.experts + e];
                a += c;
                b += i < blockIdx.x ? c : 0;
            }
        }
        s_part[t] = make_int2(a, b);
        __syncthreads();
        if (t < p.experts)
            for (uint32_t i = 0; i < lanes; ++i) {
                const int2 c = s_part[i * p.experts + t];
                count += c.x;
                prefix += c.y;
            }
    } else if (t < p.experts) {
        count = p.totals[t];
        prefix = p.hist[size_t(blockIdx.x) * p.experts + t];
    }
    int32_t total;
    const int32_t before = route_block_scan(count, s_scan, &total);
    if (t < p.experts) {
        s_base[t] = before + prefix;
        if (blockIdx.x == 0) p.offsets[t] = before;
    }
    if (blockIdx.x == 0 && t == 0) p.offsets[p.experts] = total;
    __syncthreads();
    const size_t begin = size_t(blockIdx.x) * kRouteRows * p.top;
    const size_t all = size_t(p.rows) * p.top;
    const size_t end = min(begin + size_t(kRouteRows) * p.top, all);
    for (size_t i = begin + t; i < end; i += kRouteThreads) {
        const int32_t e = p.ids[i];
        if (e >= 0) {
            const int32_t at = s_base[e] + p.position[i];
            p.position[i] = at;
            p.order[at] = int32_t(i);
        }
        if (i >= size_t(total)) p.order[i] = -1;
    }
    ptx::griddep_launch_dependents();
}

// Gradient of the logits, one warp per row.
template <int VPT>
__global__ void __launch_bounds__(256) route_grad_kernel(const __grid_constant__ RouteParams p)
{
    __shared__ float s_row[8 * VPT * 32];
    ptx::griddep_wait();
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t row = blockIdx.x * 8u + (threadIdx.x >> 5);
    if (row < p.rows) {
        const size_t at = size_t(row) * p.top + lane;
        const int32_t id = lane < p.top ? p.ids[at] : -1;
        const float w = id >= 0 ? p.weights[at] : 0.0f;
        const float dw = id >= 0 ? p.dweights[at] : 0.0f;
        const float inner = warp_sum(id >= 0 ? w * dw : 0.0f);
        float f[VPT], d[VPT];
        float top_value = -INFINITY, sum = 0.0f;
        if (!p.renorm) route_load<VPT>(p.logits, p.dtype, row, p.experts, true, f);
        // the chosen experts' values, put in their places through shared memory
        float *mine = s_row + (threadIdx.x >> 5) * (VPT * 32);
#pragma unroll
        for (int i = 0; i < VPT; ++i) mine[i * 32 + lane] = 0.0f;
        __syncwarp();
        if (id >= 0 && id < int32_t(p.experts)) mine[id] = p.renorm ? w * (dw - inner) : dw;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < VPT; ++i) d[i] = mine[i * 32 + lane];
        if (!p.renorm) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) top_value = fmaxf(top_value, f[i]);
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) top_value = fmaxf(top_value, __shfl_xor_sync(0xffffffffu, top_value, s));
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                f[i] = (f[i] == -INFINITY) ? 0.0f : expf(f[i] - top_value);
                sum += f[i];
            }
            sum = warp_sum(sum);
            // a row with every expert at -infinity has no weights and no gradient
#pragma unroll
            for (int i = 0; i < VPT; ++i) d[i] = sum == 0.0f ? 0.0f : f[i] / sum * (d[i] - inner);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t e = uint32_t(i) * 32u + lane;
            if (e < p.experts) p.dlogits[size_t(row) * p.experts + e] = d[i];
        }
    }
    ptx::griddep_launch_dependents();
}

}  // namespace gemm_f16
