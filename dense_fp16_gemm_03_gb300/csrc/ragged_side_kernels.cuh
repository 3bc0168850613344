// The small kernels around the ragged products: tensor maps that end with a
// group's rows and the sum of a weight gradient's parts, and the adapters row by
// row and their lists.
#pragma once

#include "ragged_kernel.cuh"

namespace gemm_f16 {

// kTN: every group's tensor maps with the rows ending at the group's end, so that TMA fills the rest of its last K block
// with zeros (32 uneven groups of 16384 rows in all, 4096 x 4096: 442 us with the helper zeroing each tile's last
// block, 358 so).  One block per group, one warp per map; some 3 us in front of the product.
struct RaggedMapsParams {
    CUtensorMap maps[4];
    const int32_t *offsets;
    uint32_t groups, rows;
    uint32_t have;      // bit i: maps[i] is one
    CUtensorMap *out;   // [groups][4]
};

__global__ void __launch_bounds__(128) ragged_maps_kernel(const __grid_constant__ RaggedMapsParams p)
{
    __shared__ __align__(128) CUtensorMap s_map[4];
    ptx::griddep_wait();
    const uint32_t lane = threadIdx.x & 31u, i = threadIdx.x >> 5, g = blockIdx.x;
    // the group's end as ragged_table has it: the largest of the clamped offsets up to it
    int32_t end = 0;
    for (uint32_t k = lane; k <= g + 1u; k += 32u) end = max(end, min(p.offsets[k], int32_t(p.rows)));
    end = __reduce_max_sync(0xffffffffu, end);
    if ((p.have >> i) & 1u) {
        reinterpret_cast<uint32_t *>(&s_map[i])[lane] = reinterpret_cast<const uint32_t *>(&p.maps[i])[lane];
        __syncwarp();
        if (lane == 0) ptx::tensormap_set_dim1(ptx::smem_addr(&s_map[i]), uint32_t(max(end, 1)));
        __syncwarp();
        ptx::tensormap_publish(p.out + 4u * g + i, ptx::smem_addr(&s_map[i]));
    }
    ptx::griddep_launch_dependents();
}

// kTN with few tiles: the rows of a group are cut into parts of `part_rows` (a multiple of a K block), each part's sum
// goes to a matrix of its own in fp32, and this kernel adds a group's parts, in order, and rounds once.  Bound by L2 for
// large matrices, else by its launch.  One block row per group.  (10560 rows in one group, 64 x 248: 63.6 us whole, 15.6
// in parts; 27407 rows in 3 groups, 640 x 104: 89.3 and 18.7; 9426 in 2, 144 x 3328: 32.6 and 25.3.)
constexpr uint32_t kRagPartGroups = 128;

struct RaggedPartsParams {
    const float4 *parts;  // [parts][n * k / 4]
    const int32_t *offsets;
    void *out;            // [groups, n, k]
    uint32_t groups, rows, part_rows;
    uint32_t quads;       // n * k / 4
    uint32_t out32, bf16;
};

__global__ void __launch_bounds__(256) ragged_parts_kernel(const __grid_constant__ RaggedPartsParams p)
{
    __shared__ int32_t s_row[kRagPartGroups + 1];
    __shared__ uint32_t s_parts[kRagPartGroups];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint32_t i = threadIdx.x, g = blockIdx.y;
    if (i <= p.groups) s_row[i] = max(0, min(p.offsets[i], int32_t(p.rows)));
    __syncthreads();
    if (i < p.groups) {  // as ragged_table has them
        int32_t begin = 0;
        for (uint32_t j = 0; j <= i; ++j) begin = max(begin, s_row[j]);
        s_parts[i] = uint32_t((max(begin, s_row[i + 1]) - begin + int32_t(p.part_rows) - 1) / int32_t(p.part_rows));
    }
    __syncthreads();
    uint32_t first = 0;
    for (uint32_t j = 0; j < g; ++j) first += s_parts[j];
    const uint32_t count = s_parts[g];
    const uint32_t q = blockIdx.x * 256u + i;
    if (q >= p.quads) return;
    const float4 *from = p.parts + size_t(first) * p.quads + q;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (uint32_t j = 0; j < count; ++j) {
        const float4 v = from[size_t(j) * p.quads];
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
    }
    const size_t at = size_t(g) * p.quads + q;
    if (p.out32)
        static_cast<float4 *>(p.out)[at] = sum;
    else
        static_cast<uint2 *>(p.out)[at] = make_uint2(ragged_pack(sum.x, sum.y, p.bf16 != 0u), ragged_pack(sum.z, sum.w, p.bf16 != 0u));
}

// Adapters without the tensor cores: with an adapter to nearly every row, all of the work is reading a and b once, and
// each row sees its own adapter only.  u = scale x a^T and delta = u b^T stay in fp32.  They run beside the projection,
// which starts at once and waits for delta in its epilogue.  16 rows with 16 adapters of rank 16, 8192 x 4096, take 22 us,
// as without adapters 20; 64 with 64 take 30 (as K blocks of the projection 36): there the two kernels, 7 us each on an
// idle GPU, end after the projection's loads.
//
// For a few rows of a low rank a cluster of eight CTAs takes a row through both steps and trades u through distributed
// shared memory: one launch fewer, 2 to 4 us of the host's time, and the GPU's with it, then by the two kernels: 16 rows,
// rank 16, 8192 x 4096, 21.7 us and 23.6; 32 rows 23.1 and 24.7; 1 row, 4096 x 4096, 14.4 and 13.9.  But 64 rows take 32.6
// and 29.0, and rank 64 (16 rows, 11008 x 4096) 35.8 and 33.3: a row's work on eight SMs only.
struct LoraFewParams {
    const void *x, *a, *b;
    const int32_t *ids;
    const float *scale;
    float *u;       // [rows, rank]
    float *delta;   // [rows, n]
    uint32_t rows, n, k, rank, adapters, bf16;
};

// Four of a row's u's (before the scale) by WARPS warps that share k: each lane multiplies 8 elements at a time.  The sums
// of a single warp are in all lanes; of four, thread t returns number t mod 4, and s_sum is the block's.
template <int WARPS>
__device__ __forceinline__ float lora_dot4(const LoraFewParams &p, uint32_t row, int32_t id, uint32_t r0, float (*s_sum)[4])
{
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const bool bf16 = p.bf16 != 0u;
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.x) + size_t(row) * p.k * 2u);
    const char *a = static_cast<const char *>(p.a) + (size_t(id) * p.rank + r0) * p.k * 2u;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (uint32_t i = WARPS == 1 ? lane : threadIdx.x; i < p.k / 8u; i += 32u * WARPS) {
        const uint4 xv = x[i];
        uint4 av[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) av[r] = reinterpret_cast<const uint4 *>(a + size_t(r) * p.k * 2u)[i];
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 xf = ragged_unpack(xw[j], bf16);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t aw = j == 0 ? av[r].x : j == 1 ? av[r].y : j == 2 ? av[r].z : av[r].w;
                const float2 af = ragged_unpack(aw, bf16);
                sum[r] = fmaf(xf.x, af.x, sum[r]);
                sum[r] = fmaf(xf.y, af.y, sum[r]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], d);
    const uint32_t r = threadIdx.x & 3u;
    if constexpr (WARPS == 1) {
        return r == 0u ? sum[0] : r == 1u ? sum[1] : r == 2u ? sum[2] : sum[3];
    } else {
        __syncthreads();  // the four before have been read
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) s_sum[warp][i] = sum[i];
        __syncthreads();
        return (s_sum[0][r] + s_sum[1][r]) + (s_sum[2][r] + s_sum[3][r]);
    }
}

// 128 columns of a row's delta by one warp.  LANES lanes share a row of b, 16 bytes each, with their part of u in
// registers; eight rows' loads are in flight.  (One lane to a row of b read a line per lane and load.)
template <int LANES>
__device__ __forceinline__ void lora_columns(const LoraFewParams &p, uint32_t row, int32_t id, uint32_t col0, const float (&u)[8])
{
    const uint32_t lane = threadIdx.x & 31u, part = lane % LANES;
    const bool bf16 = p.bf16 != 0u, live = 8u * part < p.rank;
    constexpr uint32_t kRows = 32 / LANES;  // rows of b a warp reads at a time
    constexpr uint32_t kFlight = 8;         // and such reads in flight
    const char *b = static_cast<const char *>(p.b) + size_t(id) * p.n * p.rank * 2u + 16u * part;
#pragma unroll 1
    for (uint32_t i0 = 0; i0 < 128u; i0 += kFlight * kRows) {
        uint4 v[kFlight];
#pragma unroll
        for (int i = 0; i < int(kFlight); ++i) {
            const uint32_t col = col0 + i0 + uint32_t(i) * kRows + lane / LANES;
            v[i] = (live && col < p.n && i0 + uint32_t(i) * kRows < 128u)
                       ? *reinterpret_cast<const uint4 *>(b + size_t(col) * p.rank * 2u)
                       : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < int(kFlight); ++i) {
            if (i0 + uint32_t(i) * kRows >= 128u) continue;
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = ragged_unpack(w[j], bf16);
                sum = fmaf(f.x, u[2 * j], sum);
                sum = fmaf(f.y, u[2 * j + 1], sum);
            }
#pragma unroll
            for (int d = LANES / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const uint32_t col = col0 + i0 + uint32_t(i) * kRows + lane / LANES;
            if (part == 0u && col < p.n) p.delta[size_t(row) * p.n + col] = sum;
        }
    }
}

// An item is a row and four of its u's: a block's (WARPS = 4), or, where there are more of them than the GPU has blocks at
// a time, a warp's.  (Here and below items are counted in 32 bits: rows that have more go by the tensor cores.)
template <int WARPS>
__global__ void __launch_bounds__(128) lora_shrink_kernel(const __grid_constant__ LoraFewParams p)
{
    __shared__ float s_sum[4][4];
    ptx::griddep_wait();
    // (after the wait: what the next kernels read from before this one is complete as well)
    ptx::griddep_launch_dependents();
    constexpr uint32_t kItems = 4 / WARPS;  // of a block at a time
    const uint32_t parts = p.rank / 4u;
    for (uint32_t item = blockIdx.x * kItems + (WARPS == 1 ? threadIdx.x >> 5 : 0u); item < p.rows * parts; item += gridDim.x * kItems) {
        const uint32_t row = item / parts, r0 = (item - row * parts) * 4u;
        const int32_t id = p.ids[row];
        if (uint32_t(id) >= p.adapters) continue;
        const float v = lora_dot4<WARPS>(p, row, id, r0, s_sum) * (p.scale ? p.scale[id] : 1.0f);
        const uint32_t t = WARPS == 1 ? threadIdx.x & 31u : threadIdx.x;
        if (t < 4u) p.u[size_t(row) * p.rank + r0 + t] = v;
    }
}

// An item, a warp's, is a row and 128 of its columns.
template <int LANES>
__global__ void __launch_bounds__(128) lora_expand_kernel(const __grid_constant__ LoraFewParams p)
{
    // The product behind this kernel reads nothing of the kernel before this one; that one has waited for all before it.
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const uint32_t part = (threadIdx.x & 31u) % LANES, parts = (p.n + 127u) / 128u;
    for (uint32_t item = blockIdx.x * 4u + (threadIdx.x >> 5); item < p.rows * parts; item += gridDim.x * 4u) {
        const uint32_t row = item / parts;
        const int32_t id = p.ids[row];
        if (uint32_t(id) >= p.adapters) continue;
        float u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = 8u * part < p.rank ? p.u[size_t(row) * p.rank + 8u * part + j] : 0.0f;
        lora_columns<LANES>(p, row, id, (item - row * parts) * 128u, u);
    }
}

// Both steps of one row by a cluster.
constexpr uint32_t kLoraCluster = 8;

template <int LANES>
__global__ void __launch_bounds__(128) lora_rows_kernel(const __grid_constant__ LoraFewParams p)
{
    __shared__ float s_sum[4][4];
    __shared__ float s_u[32];
    ptx::cluster_sync();  // every CTA of the cluster runs: its shared memory may be written
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();  // (after the wait, as above)
    const uint32_t part = (threadIdx.x & 31u) % LANES, rank = ptx::cluster_ctarank(), row = blockIdx.x / kLoraCluster;
    const int32_t id = p.ids[row];
    if (uint32_t(id) >= p.adapters) return;  // (the same for the whole cluster)
    for (uint32_t r0 = 4u * rank; r0 < p.rank; r0 += 4u * kLoraCluster) {
        const float v = lora_dot4<4>(p, row, id, r0, s_sum) * (p.scale ? p.scale[id] : 1.0f);
        if (threadIdx.x < 4u * kLoraCluster)  // four values to every CTA
            ptx::st_shared_cluster_u32(ptx::map_to_rank(ptx::smem_addr(&s_u[r0 + (threadIdx.x & 3u)]), threadIdx.x >> 2),
                                       __float_as_uint(v));
    }
    __syncwarp();
    ptx::cluster_sync();
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = 8u * part < p.rank ? s_u[8u * part + j] : 0.0f;
    for (uint32_t item = rank * 4u + (threadIdx.x >> 5); item < (p.n + 127u) / 128u; item += 4u * kLoraCluster)
        lora_columns<LANES>(p, row, id, item * 128u, u);
}

// Lists for the tensor cores' form: the adapters present in each tile of `per` rows (per <= 256), in order of first
// appearance.  Rows with an id outside [0, adapters) have none.  Two cuttings of the same rows at once: `tiles` blocks for
// the first, the rest for the second.  Bound by latency, some 4 us.
struct LoraListParams {
    const int32_t *ids;
    uint32_t rows, adapters, tiles;
    uint32_t per[2];
    int32_t *counts[2], *list[2];
};

__global__ void __launch_bounds__(256) lora_list_kernel(const __grid_constant__ LoraListParams p)
{
    __shared__ __align__(16) int32_t s_id[256];
    __shared__ uint32_t s_warp[8];
    ptx::griddep_wait();
    const uint32_t cut = blockIdx.x < p.tiles ? 0u : 1u, tile = blockIdx.x - cut * p.tiles, per = p.per[cut];
    const uint32_t t = threadIdx.x, row = tile * per + t;
    int32_t id = (p.adapters != 0u && t < per && row < p.rows) ? p.ids[row] : -1;
    if (uint32_t(id) >= p.adapters) id = -1;
    s_id[t] = id;
    __syncthreads();
    // the first row with its id: every earlier one differs (four at a time, the same words for the whole warp)
    bool first = id >= 0;
    for (uint32_t i = 0; i < (t | 31u) + 1u; i += 4u) {
        const int4 v = *reinterpret_cast<const int4 *>(s_id + i);
        first &= !((v.x == id && i < t) || (v.y == id && i + 1u < t) || (v.z == id && i + 2u < t) || (v.w == id && i + 3u < t));
    }
    const uint32_t vote = __ballot_sync(0xffffffffu, first);
    if ((t & 31u) == 0) s_warp[t >> 5] = __popc(vote);
    __syncthreads();
    uint32_t at = __popc(vote & ((1u << (t & 31u)) - 1u)), total = 0;
    for (uint32_t w = 0; w < 8u; ++w) {
        if (w < (t >> 5)) at += s_warp[w];
        total += s_warp[w];
    }
    if (first) p.list[cut][size_t(tile) * per + at] = id;
    if (t == 0) p.counts[cut][tile] = int32_t(total);
    ptx::griddep_launch_dependents();
}

}  // namespace gemm_f16
