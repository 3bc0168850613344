// The experts' router: top-k of every row's logits, softmax weights, and the
// rows sorted by expert (offsets, order, position) as the grouped products
// take them; and the gradient of the logits.
//
// One warp per row: the row's logits live in registers (VPT per lane) as keys
// whose unsigned order is the floats' order, so one step of the choice is a
// register maximum, a warp maximum of the key and a warp minimum of the index
// (ties to the lowest).  One block takes 64 rows; which rows of the block chose
// an expert is a 64-bit mask in shared memory, so a choice's rank among the
// block's rows is a population count, independent of the order in which the
// warps set the bits.  One block serves up to 64 rows in one launch; for more,
// the blocks' counts are scanned over the blocks (route_scan_kernel) and each
// block turns its ranks into positions (route_place_kernel).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace gemm_f16 {

constexpr int kRouteRows = 64;       // rows of a block: the bits of a mask
constexpr int kRouteThreads = 1024;
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

__device__ __forceinline__ float route_load(const void *base, uint32_t dtype, size_t i)
{
    if (dtype == 2u) return static_cast<const float *>(base)[i];
    if (dtype == 1u) return __bfloat162float(static_cast<const __nv_bfloat16 *>(base)[i]);
    return __half2float(static_cast<const __half *>(base)[i]);
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

template <int VPT>
__global__ void __launch_bounds__(kRouteThreads) route_topk_kernel(const __grid_constant__ RouteParams p)
{
    __shared__ unsigned long long s_mask[kRouteMaxExperts];
    __shared__ int32_t s_base[kRouteMaxExperts];
    __shared__ int32_t s_scan[32];
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    for (uint32_t e = threadIdx.x; e < p.experts; e += kRouteThreads) s_mask[e] = 0ull;
    __syncthreads();
    ptx::griddep_wait();

    constexpr int kRowsPerWarp = kRouteRows / (kRouteThreads / 32);
    int32_t id[kRowsPerWarp];
    const uint32_t row0 = blockIdx.x * kRouteRows;
#pragma unroll
    for (int q = 0; q < kRowsPerWarp; ++q) {
        const uint32_t r = warp + uint32_t(q) * (kRouteThreads / 32), row = row0 + r;
        id[q] = -1;
        if (row >= p.rows) continue;
        uint32_t key[VPT];
        float top_value = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t e = uint32_t(i) * 32u + lane;
            const float f = e < p.experts ? route_load(p.logits, p.dtype, size_t(row) * p.experts + e) : -INFINITY;
            key[i] = route_key(f);
            top_value = fmaxf(top_value, f);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top_value = fmaxf(top_value, __shfl_xor_sync(0xffffffffu, top_value, d));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (key[i]) sum += expf(route_value(key[i]) - top_value);
        sum = warp_sum(sum);
        uint32_t mine = 0u;  // key of choice `lane`
        for (uint32_t j = 0; j < p.top; ++j) {
            uint32_t best = 0u, at = 0u;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = uint32_t(i);
                }
            const uint32_t k = __reduce_max_sync(0xffffffffu, best);
            if (k == 0u) break;  // only experts at -infinity are left
            const uint32_t e = __reduce_min_sync(0xffffffffu, best == k ? at * 32u + lane : 0xffffffffu);
            if ((e & 31u) == lane) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (uint32_t(i) == (e >> 5)) key[i] = 0u;
            }
            if (lane == j) {
                mine = k;
                id[q] = int32_t(e);
            }
        }
        float w = mine ? expf(route_value(mine) - top_value) : 0.0f;
        const float chosen = warp_sum(w);
        // (a NaN anywhere in the row shows in every weight, chosen or not)
        if (p.renorm && sum == sum) sum = chosen;
        w = mine ? w / sum : 0.0f;
        if (lane < p.top) {
            p.ids[size_t(row) * p.top + lane] = id[q];
            p.weights[size_t(row) * p.top + lane] = w;
            if (id[q] >= 0) atomicOr(&s_mask[id[q]], 1ull << r);
        }
    }
    __syncthreads();
    const uint32_t t = threadIdx.x;
    const int32_t count = t < p.experts ? __popcll(s_mask[t]) : 0;
    if (p.blocks > 1u) {
        if (t < p.experts) p.hist[size_t(blockIdx.x) * p.experts + t] = count;
    } else {
        int32_t total;
        const int32_t before = route_block_scan(count, s_scan, &total);
        if (t < p.experts) {
            s_base[t] = before;
            p.offsets[t] = before;
        }
        if (t == 0) p.offsets[p.experts] = total;
        for (uint32_t i = uint32_t(total) + t; i < p.rows * p.top; i += kRouteThreads) p.order[i] = -1;
        __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < kRowsPerWarp; ++q) {
        const uint32_t r = warp + uint32_t(q) * (kRouteThreads / 32), row = row0 + r;
        if (row >= p.rows || lane >= p.top) continue;
        const size_t flat = size_t(row) * p.top + lane;
        int32_t at = -1;
        if (id[q] >= 0) {
            at = __popcll(s_mask[id[q]] & ((1ull << r) - 1ull));
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
    ptx::griddep_wait();
    const uint32_t t = threadIdx.x;
    int32_t total;
    const int32_t before = route_block_scan(t < p.experts ? p.totals[t] : 0, s_scan, &total);
    if (t < p.experts) {
        s_base[t] = before + p.hist[size_t(blockIdx.x) * p.experts + t];
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
#pragma unroll
        for (int i = 0; i < VPT; ++i) d[i] = 0.0f;
        for (uint32_t j = 0; j < p.top; ++j) {
            const int32_t e = __shfl_sync(0xffffffffu, id, j);
            const float v = __shfl_sync(0xffffffffu, p.renorm ? w * (dw - inner) : dw, j);
            if (e >= 0 && (uint32_t(e) & 31u) == lane) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (uint32_t(i) == (uint32_t(e) >> 5)) d[i] = v;
            }
        }
        if (!p.renorm) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const uint32_t e = uint32_t(i) * 32u + lane;
                f[i] = e < p.experts ? route_load(p.logits, p.dtype, size_t(row) * p.experts + e) : -INFINITY;
                top_value = fmaxf(top_value, f[i]);
            }
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
