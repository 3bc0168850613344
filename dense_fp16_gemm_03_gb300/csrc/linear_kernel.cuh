// The kernels beside the linear products (whose own is gemm_ragged_kernel with
// an epilogue): the gradient through an activation where no product comes
// before, and the sum of the bias gradient's parts.
//
// A bias gradient is a sum over a group's rows.  Each tile of the product, or
// block of linear_grad_kernel, adds up its own rows and writes one line of partial
// sums; linear_sum_kernel adds a group's lines in a fixed order, so results repeat
// bit for bit, and no atomics or cleared buffers are needed.
#pragma once

#include "ragged_kernel.cuh"

namespace gemm_f16 {

constexpr int kLinearThreads = 256;
constexpr int kLinearGradBlocks = 4;  // of linear_grad_kernel on an SM

// Row offsets as ragged_table has them (clamped, running maximum; null: one group of all rows), and the number of pieces
// of `per` rows before each group.  Run by the whole block.
__device__ __forceinline__ void linear_table(const int32_t *offsets, uint32_t groups, uint32_t rows, uint32_t per, int32_t *row,
                                             uint32_t *piece)
{
    for (uint32_t i = threadIdx.x; i <= groups; i += kLinearThreads)
        row[i] = offsets ? max(0, min(offsets[i], int32_t(rows))) : (i ? int32_t(rows) : 0);
    __syncthreads();
    if (threadIdx.x < 32u) {
        const uint32_t lane = threadIdx.x, n = groups + 1u;
        const uint32_t c = (n + 31u) / 32u, b = min(lane * c, n), e = min(b + c, n);
        int32_t top = 0;
        for (uint32_t i = b; i < e; ++i) top = max(top, row[i]);
        int32_t before = top;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= uint32_t(d)) before = max(before, o);
        }
        before = __shfl_up_sync(0xffffffffu, before, 1);
        if (lane == 0) before = 0;
        for (uint32_t i = b; i < e; ++i) {
            before = max(before, row[i]);
            row[i] = before;
        }
        __syncwarp();
        uint32_t sum = 0;
        for (uint32_t i = b; i < min(e, groups); ++i) sum += (uint32_t(row[i + 1] - row[i]) + per - 1u) / per;
        uint32_t first = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, first, d);
            if (lane >= uint32_t(d)) first += o;
        }
        first -= sum;
        for (uint32_t i = b; i < e; ++i) {
            piece[i] = first;
            if (i < groups) first += (uint32_t(row[i + 1] - row[i]) + per - 1u) / per;
        }
    }
    __syncthreads();
}

// dbias[g] from the lines of partial sums of group g: 32 columns a block, eight threads a column.
struct LinearSumParams {
    const float *sums;       // [lines, cols]
    const int32_t *offsets;  // or null
    float *dbias;            // [groups, cols]
    uint32_t groups, rows;
    uint32_t per;            // rows of a line's piece
    uint32_t cols;
};

__global__ void __launch_bounds__(kLinearThreads) linear_sum_kernel(const __grid_constant__ LinearSumParams p)
{
    __shared__ int32_t s_row[kRagMaxGroups + 1];
    __shared__ uint32_t s_piece[kRagMaxGroups + 1];
    __shared__ float s_sum[kLinearThreads / 32][33];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    linear_table(p.offsets, p.groups, p.rows, p.per, s_row, s_piece);
    const uint32_t g = blockIdx.y, lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t col = blockIdx.x * 32u + lane;
    const uint32_t first = s_piece[g], end = s_piece[g + 1u];
    float sum = 0.0f;
    if (col < p.cols) {
#pragma unroll 4
        for (uint32_t i = first + warp; i < end; i += kLinearThreads / 32) sum += p.sums[size_t(i) * p.cols + col];
    }
    s_sum[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && col < p.cols) {
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < kLinearThreads / 32; ++i) all += s_sum[i][lane];
        p.dbias[size_t(g) * p.cols + col] = all;
    }
}

// dz = dy f'(z) and the sums of its columns: a block takes a piece of `per` rows of a group and a strip of columns, a thread
// eight columns (16 bytes) of every so many rows.  A strip is 256, 128 or 64 columns, as they fill the matrix's width
// best (40000 rows of 264 columns in strips of 256: 23 us).  Bound by HBM for many rows: 16384 x 4096 through gelu with its
// bias gradient 70 us, 5.75 TB/s; few rows by the latency of the two launches (777 x 1000 in eight groups 7.2 us).
struct LinearGradParams {
    const void *dy, *z;      // z: null without activation
    void *dz;                // or null
    float *sums;             // [pieces, cols] (one piece: dbias itself), or null
    const int32_t *offsets;  // or null
    uint32_t groups, rows, cols, per;
    uint32_t lanes;          // 2^lanes threads to a row of a strip
    uint32_t strips;
    uint32_t act, bf16;
};

template <int ACT>
__device__ __forceinline__ void linear_grad_rows(const LinearGradParams &p, uint32_t begin, uint32_t end, uint32_t col, act::Two (&sum)[4])
{
    const bool bf16 = p.bf16 != 0u;
    const uint32_t step = kLinearThreads >> p.lanes;
    constexpr int kAhead = 4;
    const size_t pitch = size_t(p.cols) * 2u;
    const char *dy = static_cast<const char *>(p.dy) + size_t(col) * 2u;
    const char *z = static_cast<const char *>(p.z) + size_t(col) * 2u;
    char *dz = static_cast<char *>(p.dz) + size_t(col) * 2u;
    for (uint32_t r = begin + (threadIdx.x >> p.lanes); r < end; r += step * kAhead) {
        uint4 d[kAhead], v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const uint32_t row = r + uint32_t(i) * step;
            const bool there = row < end;
            d[i] = there ? *reinterpret_cast<const uint4 *>(dy + row * pitch) : make_uint4(0u, 0u, 0u, 0u);
            v[i] = (ACT != GEMM_ACT_NONE && there) ? *reinterpret_cast<const uint4 *>(z + row * pitch) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const uint32_t row = r + uint32_t(i) * step;
            if (row >= end) break;
            const uint32_t a[4] = {d[i].x, d[i].y, d[i].z, d[i].w}, b[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 g = ragged_unpack(a[j], bf16), at = ragged_unpack(b[j], bf16);
                const act::Two f = act::apply_grad<ACT>(act::two(g.x, g.y), act::two(at.x, at.y));
                sum[j] = sum[j] + f;
                const float2 out = act::apart(f);
                w[j] = ragged_pack(out.x, out.y, bf16);
            }
            if (p.dz) *reinterpret_cast<uint4 *>(dz + row * pitch) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

__global__ void __launch_bounds__(kLinearThreads, kLinearGradBlocks) linear_grad_kernel(const __grid_constant__ LinearGradParams p)
{
    __shared__ int32_t s_row[kRagMaxGroups + 1];
    __shared__ uint32_t s_piece[kRagMaxGroups + 1];
    __shared__ __align__(8) float s_sum[8 * kLinearThreads];  // a line of a strip's columns for each of its rows' threads
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    linear_table(p.offsets, p.groups, p.rows, p.per, s_row, s_piece);
    const uint32_t width = 8u << p.lanes;  // columns of a strip
    const uint32_t piece = blockIdx.x / p.strips, strip = blockIdx.x - piece * p.strips;
    const uint32_t at = (threadIdx.x * 8u) & (width - 1u), col = strip * width + at;
    if (p.dz) {  // rows of no group
        const uint64_t quads = p.cols / 8u, first = uint64_t(blockIdx.x) * kLinearThreads + threadIdx.x;
        const uint64_t stride = uint64_t(gridDim.x) * kLinearThreads;
        const uint32_t head = uint32_t(s_row[0]), end = uint32_t(s_row[p.groups]);
        uint4 *out = static_cast<uint4 *>(p.dz);
        for (uint64_t i = first; i < head * quads; i += stride) out[i] = make_uint4(0u, 0u, 0u, 0u);
        for (uint64_t i = end * quads + first; i < p.rows * quads; i += stride) out[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (piece >= s_piece[p.groups]) return;
    uint32_t g = 0, hi = p.groups;  // the group with s_piece[g] <= piece < s_piece[g + 1]
    while (hi - g > 1u) {
        const uint32_t mid = (g + hi) >> 1;
        if (s_piece[mid] <= piece) g = mid;
        else hi = mid;
    }
    const uint32_t begin = uint32_t(s_row[g]) + (piece - s_piece[g]) * p.per;
    const uint32_t end = min(begin + p.per, uint32_t(s_row[g + 1u]));
    act::Two sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = act::two(0.0f);
    if (col < p.cols)
        act::with_kind(p.act, [&](auto kind) { linear_grad_rows<decltype(kind)::value>(p, begin, end, col, sum); });
    if (p.sums == nullptr) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<float2 *>(&s_sum[threadIdx.x * 8u + 2u * uint32_t(j)]) = act::apart(sum[j]);
    __syncthreads();
    const uint32_t mine = strip * width + threadIdx.x;
    if (threadIdx.x < width && mine < p.cols) {
        float all = 0.0f;
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < 8u * kLinearThreads; i += width) all += s_sum[i];
        p.sums[size_t(piece) * p.cols + mine] = all;
    }
}

}  // namespace gemm_f16
