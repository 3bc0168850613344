// Inline-PTX wrappers and tensor-core descriptors that the ragged products
// use beside ptx.cuh: three-dimensional TMA copies, and descriptors whose
// operand types, majors and N are chosen at run time.  Written from the PTX
// ISA description of each instruction.
#pragma once

#include "ptx.cuh"

namespace gemm_f16 {
namespace ptx {

// 3-D tiled load global -> this CTA's shared memory, completing on the
// barrier `bar` (this CTA).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, uint32_t bar, int32_t x, int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Same, for a CTA pair: the completion barrier may live in either CTA of the
// pair (`bar` is a shared::cluster address).
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void *tmap, uint32_t bar, int32_t x, int32_t y,
                                                 int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// 4-D tiled loads, as the 3-D ones.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, uint32_t bar, int32_t x, int32_t y, int32_t z,
                                            int32_t w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const void *tmap, uint32_t bar, int32_t x, int32_t y,
                                                 int32_t z, int32_t w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// 3-D tiled store shared -> global (elements outside the tensor are skipped).
__device__ __forceinline__ void tma_store_3d(const void *tmap, uint32_t src, int32_t x, int32_t y, int32_t z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// Tensor maps edited on the device: set the extent of dimension 1 of the map in shared memory at `smem`; a whole
// warp copies it to 128-byte aligned global memory, visible to TMA after the acquire below by the thread that uses it.
__device__ __forceinline__ void tensormap_set_dim1(uint32_t smem, uint32_t extent)
{
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(smem), "r"(extent) : "memory");
}

__device__ __forceinline__ void tensormap_publish(void *global, uint32_t smem)
{
    asm volatile(
        "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
            reinterpret_cast<uint64_t>(global)),
        "r"(smem)
        : "memory");
}

__device__ __forceinline__ void tensormap_acquire(const void *global)
{
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(global)) : "memory");
}

// A release by several arrivals: the fence makes all earlier writes visible in the cluster, the arrivals behind it wait
// for nothing more.
__device__ __forceinline__ void fence_cluster()
{
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar_cluster)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// True in one lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0u;
}

__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint64_t exch_gpu_u64(uint64_t *p, uint64_t v)
{
    uint64_t old;
    asm volatile("atom.acq_rel.gpu.global.exch.b64 %0, [%1], %2;" : "=l"(old) : "l"(p), "l"(v) : "memory");
    return old;
}

__device__ __forceinline__ uint32_t ld_relaxed_gpu_u32(const uint32_t *p)
{
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void st_global_v2(void *p, uint32_t a, uint32_t b)
{
    asm volatile("st.global.v2.b32 [%0], {%1, %2};" ::"l"(p), "r"(a), "r"(b) : "memory");
}

}  // namespace ptx

// tcgen05 shared-memory matrix descriptor of a tile that TMA wrote with
// 128-byte swizzling (rows of 128 bytes, atoms of 8 rows = 1024 bytes).
// K-major: atoms stacked along M/N at a stride byte offset of 1024, leading
// byte offset unused.  MN-major: 64-element-wide columns of 64 K rows, the
// leading byte offset (8 KB) steps between columns, the stride byte offset
// (1 KB) between groups of 8 K rows.  Fields: start address >> 4 (bits 0-13),
// leading >> 4 (16-29), stride >> 4 (32-45), version 1 (46-48), swizzle mode 2
// (61-63); tiles are 1024-byte aligned.
__device__ __forceinline__ uint64_t ragged_desc(uint32_t addr, bool mn_major)
{
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(mn_major ? (8192u >> 4) : 1u) << 16) |
           (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// tcgen05 instruction descriptor, kind::f16, D fp32 (bits 4-5 = 1), without
// N: A and B both fp16 (bits 7-9, 10-12 = 0) or both bf16 (= 1), A and B
// K-major or MN-major (bits 15, 16), M >> 4 in bits 24-28.  ragged_idesc_n adds
// N >> 3 in bits 17-22.
__device__ __forceinline__ uint32_t ragged_idesc(uint32_t m, bool bf16, bool a_mn, bool b_mn)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? (1u << 15) : 0u) | (b_mn ? (1u << 16) : 0u) |
           ((m >> 4) << 24);
}

__device__ __forceinline__ uint32_t ragged_idesc_n(uint32_t n)
{
    return (n >> 3) << 17;
}

}  // namespace gemm_f16
