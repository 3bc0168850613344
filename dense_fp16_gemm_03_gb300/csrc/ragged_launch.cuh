// Host side that the ragged products' translation units share: kernel variants
// and what a device holds of them, tensor maps, checks of arguments, launches,
// and the choice between few-row and many-row tiles.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <initializer_list>
#include <mutex>
#include <string.h>

#include "device_state.h"
#include "gemm_ragged.h"
#include "ragged_kernel.cuh"

namespace gemm_f16 {
namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kSizeLimit = int64_t(1) << 31;
constexpr int64_t kIterLimit = (int64_t(1) << 32) - 1;  // K-block iterations of a split launch are counted in 32 bits

int64_t cdiv(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

int64_t round_up(int64_t a, int64_t b)
{
    return cdiv(a, b) * b;
}

// ------------------------------------------------------------ variants

// One compiled kernel: the CTA pair of each mode for many rows, the single CTA with a 64-row N side
// for few.
struct RaggedVariant {
    int mode, cg, qcap, qbox, smem, threads;
    const void *fn;
};

// (the last arguments, if any, follow the ring's stages in the kernel's template)
#define RAGGED_VARIANT(MODE, CG, QCAP, ...)                                                      \
    RaggedVariant                                                                                \
    {                                                                                            \
        MODE, CG, QCAP, RaggedCfg<MODE, CG, QCAP, __VA_ARGS__>::kQBox,                           \
            RaggedCfg<MODE, CG, QCAP, __VA_ARGS__>::kSmemBytes,                                  \
            RaggedCfg<MODE, CG, QCAP, __VA_ARGS__>::kThreads,                                    \
            reinterpret_cast<const void *>(&gemm_ragged_kernel<MODE, CG, QCAP, __VA_ARGS__>)     \
    }

template <int COUNT>
struct RaggedDeviceOf {
    bool ready = false;
    unsigned long long ctx_id = 0;
    int slots[COUNT] = {};  // co-resident CTAs (single) or pairs of each variant
    int num_sms = 0;
    uint32_t *error_word = nullptr;
};

// A kernel and its dynamic shared memory.
struct KernelSmem {
    const void *fn;
    int bytes;
};

// State of the current device for a table of variants, `beside` small kernels that run in front of them, and `large` ones that
// need more shared memory than a launch has unasked, made once per context.
template <int COUNT>
gemm_status_t ragged_device_of(const RaggedVariant (&variants)[COUNT], const void *const *beside, int num_beside,
                               const KernelSmem *large, int num_large, RaggedDeviceOf<COUNT> **out)
{
    DeviceState state;
    gemm_status_t st = current_device_state(&state);
    if (st != GEMM_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    static std::mutex mutex;
    static RaggedDeviceOf<COUNT> devices[kMaxDevices];
    std::lock_guard<std::mutex> lock(mutex);
    RaggedDeviceOf<COUNT> &d = devices[dev];
    if (!d.ready || d.ctx_id != state.ctx_id) {
        RaggedDeviceOf<COUNT> made;
        made.ctx_id = state.ctx_id;
        made.num_sms = state.num_sms;
        made.error_word = state.error_word;
        for (int v = 0; v < COUNT; ++v) {
            const RaggedVariant &var = variants[v];
            if (cudaFuncSetAttribute(var.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, var.smem) != cudaSuccess) {
                cudaGetLastError();
                return GEMM_ERR_CUDA;
            }
            made.slots[v] = state.num_sms / var.cg;
            if (var.cg > 1) {
                cudaLaunchConfig_t cfg;
                memset(&cfg, 0, sizeof(cfg));
                cfg.gridDim = dim3(unsigned(made.slots[v] * var.cg), 1, 1);
                cfg.blockDim = dim3(unsigned(var.threads), 1, 1);
                cfg.dynamicSmemBytes = size_t(var.smem);
                cudaLaunchAttribute attr;
                attr.id = cudaLaunchAttributeClusterDimension;
                attr.val.clusterDim.x = unsigned(var.cg);
                attr.val.clusterDim.y = 1;
                attr.val.clusterDim.z = 1;
                cfg.attrs = &attr;
                cfg.numAttrs = 1;
                int clusters = 0;
                if (cudaOccupancyMaxActiveClusters(&clusters, var.fn, &cfg) == cudaSuccess && clusters > 0)
                    made.slots[v] = clusters;
                else
                    cudaGetLastError();
            }
        }
        for (int i = 0; i < num_large; ++i) {
            if (cudaFuncSetAttribute(large[i].fn, cudaFuncAttributeMaxDynamicSharedMemorySize, large[i].bytes) != cudaSuccess) {
                cudaGetLastError();
                return GEMM_ERR_CUDA;
            }
        }
        // The small kernels in front of a product run with the SM's memory split as the product wants it: an SM does not
        // change the split under a running block, and the product's CTA would wait for the block to end.
        for (int i = 0; i < num_beside; ++i) {
            if (cudaFuncSetAttribute(beside[i], cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
                cudaSuccess) {
                cudaGetLastError();
                return GEMM_ERR_CUDA;
            }
        }
        made.ready = true;
        d = made;
    }
    *out = &d;
    return GEMM_OK;
}

// --------------------------------------------------------- tensor maps

PFN_cuTensorMapEncodeTiled_v12000 g_ragged_encode = nullptr;

gemm_status_t ragged_encoder(PFN_cuTensorMapEncodeTiled_v12000 *fn)
{
    static std::once_flag once;
    std::call_once(once, []() {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_ragged_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
        else
            cudaGetLastError();
    });
    *fn = g_ragged_encode;
    return g_ragged_encode ? GEMM_OK : GEMM_ERR_CUDA;
}

// `count` row-major matrices of rows x cols, boxes of box_cols x box_rows in 128-byte-swizzled shared memory,
// zeros outside a matrix.
gemm_status_t encode_stack(CUtensorMap *map, const void *ptr, gemm_dtype_t dtype, int64_t count, int64_t rows, int64_t cols,
                           int box_cols, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    gemm_status_t st = ragged_encoder(&enc);
    if (st != GEMM_OK) return st;
    const uint64_t size = dtype == GEMM_DTYPE_F32 ? 4u : 2u;
    cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(count)};
    cuuint64_t strides[2] = {cuuint64_t(cols) * size, cuuint64_t(cols) * cuuint64_t(rows) * size};
    cuuint32_t box[3] = {cuuint32_t(box_cols), cuuint32_t(box_rows), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapDataType type = dtype == GEMM_DTYPE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == GEMM_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUresult r = enc(map, type, 3, const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    // (a matrix stride of 2^40 bytes or more cannot be described)
    return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_UNSUPPORTED_SHAPE;
}

// `count` row-major matrices of rows x (64 groups + rest) columns, as (64 columns, row, group, matrix): boxes of two
// groups x 64 rows.
gemm_status_t encode_pairs(CUtensorMap *map, const void *ptr, gemm_dtype_t dtype, int64_t count, int64_t rows, int64_t cols,
                           uint32_t *groups)
{
    *groups = uint32_t(cols / 64);
    if (cols < 128) {
        *groups = 0;
        return GEMM_OK;
    }
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    gemm_status_t st = ragged_encoder(&enc);
    if (st != GEMM_OK) return st;
    cuuint64_t dims[4] = {64, cuuint64_t(rows), cuuint64_t(cols / 64), cuuint64_t(count)};
    cuuint64_t strides[3] = {cuuint64_t(cols) * 2u, 128, cuuint64_t(cols) * cuuint64_t(rows) * 2u};
    cuuint32_t box[4] = {64, 64, 2, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type =
        dtype == GEMM_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUresult r = enc(map, type, 4, const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_UNSUPPORTED_SHAPE;
}

// The N-side operand [rows, cols] in boxes of `box` rows, half and a quarter of them.
gemm_status_t encode_rows(CUtensorMap (&maps)[3], const void *ptr, gemm_dtype_t dtype, int64_t rows, int64_t cols, int box)
{
    for (int i = 0; i < 3; ++i) {
        gemm_status_t st = encode_stack(&maps[i], ptr, dtype, 1, rows, cols, kRagBlockK, box >> i);
        if (st != GEMM_OK) return st;
    }
    return GEMM_OK;
}

// ---------------------------------------------------------- validation

gemm_status_t check_pointer(const void *p, bool used, uintptr_t align = 16)
{
    if (!used) return GEMM_OK;
    if (p == nullptr) return GEMM_ERR_INVALID_ARG;
    return (reinterpret_cast<uintptr_t>(p) & (align - 1u)) ? GEMM_ERR_ALIGNMENT : GEMM_OK;
}

gemm_status_t check_sizes(std::initializer_list<int64_t> any, std::initializer_list<int64_t> by8)
{
    for (int64_t v : any)
        if (v < 0) return GEMM_ERR_INVALID_ARG;
    for (int64_t v : by8)
        if (v < 0) return GEMM_ERR_INVALID_ARG;
    for (int64_t v : any)
        if (v >= kSizeLimit) return GEMM_ERR_UNSUPPORTED_SHAPE;
    for (int64_t v : by8)
        if (v >= kSizeLimit || v % 8 != 0) return GEMM_ERR_UNSUPPORTED_SHAPE;
    return GEMM_OK;
}

bool operand_type(gemm_dtype_t t)
{
    return t == GEMM_DTYPE_F16 || t == GEMM_DTYPE_BF16;
}

// ------------------------------------------------------------- launches

gemm_status_t launch(const void *fn, dim3 grid, unsigned threads, int smem, int cluster, void **args, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (cluster > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = unsigned(cluster);
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // set-up overlaps the previous kernel's tail
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    cfg.attrs = attr;
    cfg.numAttrs = unsigned(na);
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

long long wait_limit_for(int64_t k_blocks)
{
    return 2000000000LL + k_blocks * 65536LL;
}

// Bytes of split work for one variant: a partial tile and a flag per CTA.
size_t split_bytes(const RaggedVariant &var, int slots)
{
    const size_t ctas = size_t(slots) * size_t(var.cg);
    return ctas * 128u * size_t(var.qcap) * 4u + ctas * 8u;
}

void use_split(RaggedParams *p, const RaggedVariant &var, int slots, void *ws)
{
    const size_t ctas = size_t(slots) * size_t(var.cg);
    p->sk = 1;
    p->partials = static_cast<float *>(ws);
    p->flags = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + ctas * 128u * size_t(var.qcap) * 4u);
    p->stamp = next_launch_stamp();
}

// `p`: the kernel's parameters, `base` the part of them that every variant has.
gemm_status_t launch_variant(const RaggedVariant &var, int slots, uint32_t *error_word, RaggedParams &base, void *p, int64_t most_units,
                             cudaStream_t stream)
{
    int64_t workers = slots;
    if (most_units < workers) workers = most_units < 1 ? 1 : most_units;
    base.error_word = error_word;
    base.by[0] = make_fastdiv(uint32_t(kRagBand) * base.tiles_p);
    for (int d = 1; d <= kRagBand; ++d) base.by[d] = make_fastdiv(uint32_t(d));
    void *args[1] = {p};
    return launch(var.fn, dim3(unsigned(workers * var.cg), 1, 1), unsigned(var.threads), var.smem, var.cg, args, stream);
}

// Tiles of a forward or data-gradient launch, at most (a group's last tile may be a part of one).
int64_t most_tiles(const RaggedVariant &var, int64_t groups, int64_t rows, int64_t pdim)
{
    return cdiv(pdim, 128 * var.cg) * (rows / var.qcap + (groups < rows ? groups : rows));
}

constexpr int64_t kWideSplitBlocks = 16;  // K blocks below which splitting pairs' tiles never pays

// A forward or data-gradient launch: single CTAs with a 64-row N side, or CTA pairs with up to 256 rows, and whether
// tiles are split over K (every worker then takes the same number of K blocks; the partial sums cost a join).
struct RaggedChoice {
    bool wide;
    bool split;
};

// Whichever of the four an estimate of the time has ahead for groups of equal size: the bytes at HBM's rate or whole
// waves of tiles, split ones an even share, and each way's fixed time.  The constants (us) are fitted to 600 launches of
// random sizes (1 to 64 groups, 1 to 30000 rows, n and k 128 to 6144; all four measured): on 549 others the choice is 1.5%
// slower than the fastest on average, 20% when single CTAs always split and ran up to 64 rows a group
// (16 rows in 36 groups, 1264 x 368: 6.6 us unsplit, 9.8 split; 12 rows in 2 groups, 728 x 4808: 18.8 and 10.7; 409 rows in
// 50 groups, data gradient, 2968 x 5656: 419 split single CTAs, 253 pairs).  Splitting many tiles loses more than the join:
// workers that are at different depths of K share no weights' pages, nor, with pairs, the rows in L2.
// `beside` (us): other work that the main loops run beside and their ends wait for.
// `f`, `w`: the two variants, and the slots that the device has for each.
RaggedChoice ragged_choice(const RaggedVariant &f, int few_slots, const RaggedVariant &w, int wide_slots, int64_t groups, int64_t rows,
                           int64_t pdim, int64_t kdim, bool may_split, double beside)
{
    const int64_t live = groups < rows ? groups : rows;
    if (live == 0) return {false, false};
    const double each = double(rows) / double(live), blocks = double(cdiv(kdim, kRagBlockK));
    const double bytes = 2.0 * (double(live) * double(pdim) * double(kdim) + double(rows) * double(pdim + kdim)) / 6.6e6;
    const double part = each < w.qcap ? each / w.qcap : 1.0;  // of a pair's N side
    const int64_t few_tiles = live * cdiv(int64_t(each), f.qcap) * cdiv(pdim, 128);
    const int64_t wide_tiles = live * cdiv(int64_t(each), w.qcap) * cdiv(pdim, 256);
    const double few_share = double(few_tiles) / few_slots, wide_share = double(wide_tiles) / wide_slots;
    const double few_block = 0.195 + 0.093 * (few_share < 1.0 ? few_share : 1.0);  // a CTA alone, and with its share of L2's rate
    const double wide_block = 0.226 + 0.08 * part;
    const double least = bytes > beside ? bytes : beside;
    RaggedChoice best = {false, false};
    double time = 1e30;
    auto offer = [&](bool wide, bool split, double fixed, double loops) {
        const double t = fixed + (loops > least ? loops : least);
        if (t < time) {
            time = t;
            best = {wide, split};
        }
    };
    offer(false, false, 3.6, double(cdiv(few_tiles, few_slots)) * (blocks * few_block + 0.4));
    offer(true, false, 3.8, double(cdiv(wide_tiles, wide_slots)) * (blocks * wide_block + 0.8 + 1.76 * part));
    if (may_split) {
        offer(false, true, 7.7, few_share * blocks * 0.288 + 0.4);
        if (rows > f.qcap && wide_share < 1.0 && blocks >= kWideSplitBlocks)
            offer(true, true, 8.5 + 9.6 * part, wide_share * blocks * wide_block);
    }
    return best;
}

}  // namespace
}  // namespace gemm_f16
