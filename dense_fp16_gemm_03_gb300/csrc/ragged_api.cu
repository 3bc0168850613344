// C ABI of the ragged products and the router (declared in include/gemm_ragged.h):
// argument validation, the choice of kernel variant, workspace layout, tensor
// maps and launches.  The kernels are in ragged_kernel.cuh and route_kernel.cuh.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>
#include <math.h>
#include <string.h>

#include "device_state.h"
#include "gemm_ragged.h"
#include "ragged_kernel.cuh"
#include "route_kernel.cuh"

using namespace gemm_f16;

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

#define RAGGED_VARIANT(MODE, CG, QCAP, ST)                                                               \
    RaggedVariant                                                                                        \
    {                                                                                                    \
        MODE, CG, QCAP, RaggedCfg<MODE, CG, QCAP, ST>::kQBox, RaggedCfg<MODE, CG, QCAP, ST>::kSmemBytes, \
            RaggedCfg<MODE, CG, QCAP, ST>::kThreads,                                                     \
            reinterpret_cast<const void *>(&gemm_ragged_kernel<MODE, CG, QCAP, ST>)                      \
    }

enum RaggedVariantId { kVNtWide, kVNtFew, kVNnWide, kVNnFew, kVTn, kVLoraU, kVLoraY };
const RaggedVariant kRagged[] = {
    RAGGED_VARIANT(kNT, 2, 256, 6), RAGGED_VARIANT(kNT, 1, 64, 8),
    RAGGED_VARIANT(kNN, 2, 256, 6), RAGGED_VARIANT(kNN, 1, 64, 8),
    RAGGED_VARIANT(kTN, 2, 256, 6),
    RAGGED_VARIANT(kLoraU, 1, 64, 8),
    RAGGED_VARIANT(kLoraY, 2, 256, 6),
};
constexpr int kNumRagged = int(sizeof(kRagged) / sizeof(kRagged[0]));

// The instances of the adapters' kernels whose lanes hold a rank's 16-byte pieces.
const void *lora_rows_instance(int64_t rank)
{
    return rank <= 8    ? reinterpret_cast<const void *>(&lora_rows_kernel<1>)
           : rank <= 16 ? reinterpret_cast<const void *>(&lora_rows_kernel<2>)
                        : reinterpret_cast<const void *>(&lora_rows_kernel<4>);
}

const void *lora_expand_instance(int64_t rank)
{
    return rank <= 8    ? reinterpret_cast<const void *>(&lora_expand_kernel<1>)
           : rank <= 16 ? reinterpret_cast<const void *>(&lora_expand_kernel<2>)
           : rank <= 32 ? reinterpret_cast<const void *>(&lora_expand_kernel<4>)
           : rank <= 64 ? reinterpret_cast<const void *>(&lora_expand_kernel<8>)
                        : reinterpret_cast<const void *>(&lora_expand_kernel<16>);
}

const void *const kBeside[] = {
    lora_rows_instance(8),    lora_rows_instance(16),   lora_rows_instance(32),
    lora_expand_instance(8),  lora_expand_instance(16), lora_expand_instance(32),
    lora_expand_instance(64), lora_expand_instance(128), reinterpret_cast<const void *>(&lora_shrink_kernel<1>),
    reinterpret_cast<const void *>(&lora_shrink_kernel<4>), reinterpret_cast<const void *>(&lora_list_kernel), reinterpret_cast<const void *>(&ragged_maps_kernel),
};

struct RaggedDevice {
    bool ready = false;
    unsigned long long ctx_id = 0;
    int slots[kNumRagged] = {};  // co-resident CTAs (single) or pairs of each variant
    int num_sms = 0;
    uint32_t *error_word = nullptr;
};

std::mutex g_ragged_mutex;
RaggedDevice g_ragged_devices[kMaxDevices];

// State of the current device for these kernels, made once per context.
gemm_status_t ragged_device(RaggedDevice **out)
{
    DeviceState state;
    gemm_status_t st = current_device_state(&state);
    if (st != GEMM_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    std::lock_guard<std::mutex> lock(g_ragged_mutex);
    RaggedDevice &d = g_ragged_devices[dev];
    if (!d.ready || d.ctx_id != state.ctx_id) {
        RaggedDevice made;
        made.ctx_id = state.ctx_id;
        made.num_sms = state.num_sms;
        made.error_word = state.error_word;
        for (int v = 0; v < kNumRagged; ++v) {
            const RaggedVariant &var = kRagged[v];
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
        // The small kernels in front of a product run with the SM's memory split as the product wants it: an SM does not
        // change the split under a running block, and the product's CTA would wait for the block to end.
        for (const void *fn : kBeside) {
            if (cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
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

// Bytes of the weight gradient's tensor maps, four per group.
size_t maps_bytes(int64_t groups)
{
    return size_t(groups) * 4u * sizeof(CUtensorMap);
}

void use_split(RaggedParams *p, const RaggedVariant &var, int slots, void *ws)
{
    const size_t ctas = size_t(slots) * size_t(var.cg);
    p->sk = 1;
    p->partials = static_cast<float *>(ws);
    p->flags = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + ctas * 128u * size_t(var.qcap) * 4u);
    p->stamp = next_launch_stamp();
}

gemm_status_t launch_ragged(int variant, const RaggedDevice *dev, RaggedParams &p, int64_t most_units, cudaStream_t stream)
{
    const RaggedVariant &var = kRagged[variant];
    int64_t workers = dev->slots[variant];
    if (most_units < workers) workers = most_units < 1 ? 1 : most_units;
    p.error_word = dev->error_word;
    p.by[0] = make_fastdiv(uint32_t(kRagBand) * p.tiles_p);
    for (int d = 1; d <= kRagBand; ++d) p.by[d] = make_fastdiv(uint32_t(d));
    void *args[1] = {&p};
    return launch(var.fn, dim3(unsigned(workers * var.cg), 1, 1), unsigned(var.threads), var.smem, var.cg, args, stream);
}

// ------------------------------------------------------ grouped products

constexpr int64_t kMinPartRows = 256;      // rows of a part of a weight gradient's group, at least
constexpr int64_t kWideSplitBlocks = 16;  // K blocks below which splitting pairs' tiles never pays

// A forward or data-gradient launch: single CTAs with a 64-row N side, or CTA pairs with up to 256 rows, and whether
// tiles are split over K (every worker then takes the same number of K blocks; the partial sums cost a join).
struct RaggedChoice {
    int variant;
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
RaggedChoice grouped_choice(int mode, int64_t groups, int64_t rows, int64_t pdim, int64_t kdim, bool may_split, double beside,
                            const RaggedDevice *dev)
{
    const int few_v = mode == kNT ? kVNtFew : kVNnFew, wide_v = mode == kNT ? kVNtWide : kVNnWide;
    const RaggedVariant &f = kRagged[few_v], &w = kRagged[wide_v];
    const int64_t live = groups < rows ? groups : rows;
    if (live == 0) return {few_v, false};
    const double each = double(rows) / double(live), blocks = double(cdiv(kdim, kRagBlockK));
    const double bytes = 2.0 * (double(live) * double(pdim) * double(kdim) + double(rows) * double(pdim + kdim)) / 6.6e6;
    const double part = each < w.qcap ? each / w.qcap : 1.0;  // of a pair's N side
    const int64_t few_tiles = live * cdiv(int64_t(each), f.qcap) * cdiv(pdim, 128);
    const int64_t wide_tiles = live * cdiv(int64_t(each), w.qcap) * cdiv(pdim, 256);
    const double few_share = double(few_tiles) / dev->slots[few_v], wide_share = double(wide_tiles) / dev->slots[wide_v];
    const double few_block = 0.195 + 0.093 * (few_share < 1.0 ? few_share : 1.0);  // a CTA alone, and with its share of L2's rate
    const double wide_block = 0.226 + 0.08 * part;
    const double least = bytes > beside ? bytes : beside;
    RaggedChoice best = {few_v, false};
    double time = 1e30;
    auto offer = [&](int variant, bool split, double fixed, double loops) {
        const double t = fixed + (loops > least ? loops : least);
        if (t < time) {
            time = t;
            best = {variant, split};
        }
    };
    offer(few_v, false, 3.6, double(cdiv(few_tiles, dev->slots[few_v])) * (blocks * few_block + 0.4));
    offer(wide_v, false, 3.8, double(cdiv(wide_tiles, dev->slots[wide_v])) * (blocks * wide_block + 0.8 + 1.76 * part));
    if (may_split) {
        offer(few_v, true, 7.7, few_share * blocks * 0.288 + 0.4);
        if (rows > f.qcap && wide_share < 1.0 && blocks >= kWideSplitBlocks)
            offer(wide_v, true, 8.5 + 9.6 * part, wide_share * blocks * wide_block);
    }
    return best;
}

// Rows of the parts that a weight-gradient launch cuts its groups into, 0 for whole groups.  Tiles of few groups leave pairs
// idle while each goes through all rows of its group, 0.35 us a K block; parts fill the pairs and cost the sum of their
// matrices, written and read through L2 at some 4.5 TB/s, and a launch.
int64_t grouped_part_rows(int64_t groups, int64_t rows, int64_t n, int64_t k, const RaggedDevice *dev)
{
    const RaggedVariant &v = kRagged[kVTn];
    const int64_t each = cdiv(n, 128 * v.cg) * cdiv(k, v.qcap), slots = dev->slots[kVTn];  // tiles of a matrix
    if (groups * each > slots || groups > int64_t(kRagPartGroups) || rows <= kMinPartRows) return 0;
    const double live = double(groups < rows ? groups : rows), loops = 0.35 * double(rows) / kRagBlockK;
    const double matrix = double(n) * double(k) * 8.0 / 4.5e6;  // us
    double parts = double(slots / each) - 0.5 * live;  // (a group's last part is a half, on average)
    const double best = sqrt(loops / matrix);
    if (best < parts) parts = best;
    if (parts <= live) return 0;
    int64_t part = round_up(int64_t(double(rows) / parts) + 1, kRagBlockK);
    if (part < kMinPartRows) part = kMinPartRows;
    const double split = loops * double(part) / double(rows) + 3.0 + (double(rows) / double(part) + 0.5 * live) * matrix;
    return split < loops / live ? part : 0;
}

// Bytes of the parts' matrices, of `parts` parts.
size_t part_bytes(int64_t parts, int64_t n, int64_t k)
{
    return size_t(parts) * size_t(n) * size_t(k) * 4u;
}

// What any number of rows up to this one may need for parts.
size_t part_room(int64_t groups, int64_t rows, int64_t n, int64_t k, const RaggedDevice *dev)
{
    const RaggedVariant &v = kRagged[kVTn];
    const int64_t each = cdiv(n, 128 * v.cg) * cdiv(k, v.qcap), slots = dev->slots[kVTn];
    if (groups * each > slots || each == 0 || groups > int64_t(kRagPartGroups) || rows <= kMinPartRows) return 0;
    return part_bytes(slots / each + groups, n, k);
}

// Tiles of a forward or data-gradient launch, at most (a group's last tile may be a part of one).
int64_t most_tiles(const RaggedVariant &var, int64_t groups, int64_t rows, int64_t pdim)
{
    return cdiv(pdim, 128 * var.cg) * (rows / var.qcap + (groups < rows ? groups : rows));
}

// Bytes of split work that any number of rows up to this one may need.
size_t split_room(int64_t rows, int64_t kdim, const RaggedDevice *dev)
{
    const size_t few = split_bytes(kRagged[kVNtFew], dev->slots[kVNtFew]);
    const size_t wide = split_bytes(kRagged[kVNtWide], dev->slots[kVNtWide]);
    return rows > kRagged[kVNtFew].qcap && cdiv(kdim, kRagBlockK) >= kWideSplitBlocks && wide > few ? wide : few;
}

gemm_status_t grouped(int mode, gemm_dtype_t dtype, gemm_dtype_t out_type, int64_t groups, int64_t rows, int64_t n, int64_t k,
                      const int32_t *offsets, const void *first, const void *second, void *out, void *ws, size_t ws_bytes,
                      uint32_t skip_fill, long long wait_limit, cudaStream_t stream)
{
    gemm_status_t st = check_sizes({groups, rows}, {n, k});
    if (st != GEMM_OK) return st;
    if (!operand_type(dtype) || (out_type != dtype && !(mode == kTN && out_type == GEMM_DTYPE_F32)))
        return GEMM_ERR_INVALID_ARG;
    if (groups > GEMM_GROUPED_MAX_GROUPS) return GEMM_ERR_UNSUPPORTED_SHAPE;
    const int64_t pdim = mode == kNN ? k : n;           // M side of the instruction
    const int64_t kdim = mode == kNT ? k : mode == kNN ? n : rows;  // contraction
    const int64_t out_rows = mode == kTN ? groups * n : rows;
    const int64_t out_cols = mode == kNT ? n : k;
    const size_t out_bytes = size_t(out_rows) * size_t(out_cols) * (out_type == GEMM_DTYPE_F32 ? 4u : 2u);
    const bool sum = kdim > 0 && groups > 0;  // anything to add up
    st = check_pointer(out, out_bytes > 0);
    if (st == GEMM_OK) st = check_pointer(first, out_bytes > 0 && sum);
    if (st == GEMM_OK) st = check_pointer(second, out_bytes > 0 && sum);
    if (st == GEMM_OK) st = check_pointer(offsets, out_bytes > 0 && sum, 4);
    if (st != GEMM_OK) return st;
    if (out_bytes == 0) return GEMM_OK;
    RaggedDevice *dev = nullptr;
    st = ragged_device(&dev);
    if (st != GEMM_OK) return st;
    RaggedChoice choice = {kVTn, false};
    if (mode != kTN) choice = grouped_choice(mode, groups, rows, pdim, kdim, ws != nullptr, 0.0, dev);
    const int variant = choice.variant;
    const RaggedVariant &var = kRagged[variant];
    const int64_t part_rows = mode == kTN && ws && skip_fill == ~0u ? grouped_part_rows(groups, rows, n, k, dev) : 0;
    const int64_t parts = part_rows ? rows / part_rows + (groups < rows ? groups : rows) : 0;
    const size_t need = part_rows       ? part_bytes(parts, n, k)
                        : mode == kTN   ? maps_bytes(groups)
                        : choice.split  ? split_bytes(var, dev->slots[variant])
                                        : 0;
    if (ws != nullptr || ws_bytes != 0) {
        if (ws == nullptr || ws_bytes < need) return GEMM_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(ws) & 255u) return GEMM_ERR_ALIGNMENT;
    }
    if (!sum) {
        if (cudaMemsetAsync(out, 0, out_bytes, stream) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
        return GEMM_OK;
    }
    RaggedParams p;
    memset(&p, 0, sizeof(p));
    p.offsets = offsets;
    p.groups = uint32_t(groups);
    p.rows = uint32_t(rows);
    p.pdim = uint32_t(pdim);
    p.qdim = uint32_t(mode == kTN ? k : 0);
    p.kdim = uint32_t(kdim);
    p.k_blocks = uint32_t(cdiv(kdim, kRagBlockK));
    p.tiles_p = uint32_t(cdiv(pdim, 128 * var.cg));
    p.tiles_q = uint32_t(mode == kTN ? cdiv(k, var.qcap) : 0);
    p.bf16 = dtype == GEMM_DTYPE_BF16;
    p.out32 = out_type == GEMM_DTYPE_F32;
    p.out = out;
    p.skip_fill = skip_fill;
    p.wait_limit = wait_limit ? wait_limit : wait_limit_for(p.k_blocks);
    int64_t most;  // tiles, at most
    if (mode == kTN) most = int64_t(p.tiles_p) * p.tiles_q * (part_rows ? parts : groups);  // (groups without rows are zeroed)
    else most = most_tiles(var, groups, rows, pdim);
    if (most >= kSizeLimit) return GEMM_ERR_UNSUPPORTED_SHAPE;
    if (mode == kTN) {
        st = encode_stack(&p.tm_p, first, dtype, 1, rows, n, 64, 64);
        if (st == GEMM_OK) st = encode_stack(&p.tm_q[0], second, dtype, 1, rows, k, 64, 64);
        if (st == GEMM_OK) st = encode_pairs(&p.tm_p2, first, dtype, 1, rows, n, &p.p_groups);
        if (st == GEMM_OK) st = encode_pairs(&p.tm_q2, second, dtype, 1, rows, k, &p.q_groups);
        if (part_rows) {
            p.part_rows = uint32_t(part_rows);
            p.whole_groups = uint32_t(groups);
            p.groups = uint32_t(parts);
            p.out32 = 1;
            p.out = ws;
            if (st == GEMM_OK) st = encode_stack(&p.tm_x, ws, GEMM_DTYPE_F32, parts, n, k, 32, 32);
        } else if (st == GEMM_OK) {
            st = encode_stack(&p.tm_x, out, out_type, groups, n, k, p.out32 ? 32 : 64, 32);
        }
    } else {
        st = encode_stack(&p.tm_p, second, dtype, groups, n, k, 64, mode == kNT ? 128 : 64);
        if (st == GEMM_OK && mode == kNN) st = encode_pairs(&p.tm_p2, second, dtype, groups, n, k, &p.p_groups);
        if (st == GEMM_OK) st = encode_rows(p.tm_q, first, dtype, rows, kdim, var.qbox);
        if (choice.split && most * p.k_blocks < kIterLimit) {
            use_split(&p, var, dev->slots[variant], ws);
            most *= p.k_blocks;
        }
    }
    if (st != GEMM_OK) return st;
    // (one or two tiles a worker: the kernel that writes the maps would take longer than the helper it spares)
    const int64_t live = groups < rows ? groups : rows;
    if (ws && mode == kTN && !part_rows && int64_t(p.tiles_p) * p.tiles_q * live > 2 * dev->slots[variant]) {
        RaggedMapsParams mp;
        memset(&mp, 0, sizeof(mp));
        mp.maps[0] = p.tm_p;
        mp.maps[1] = p.tm_q[0];
        mp.maps[2] = p.tm_p2;
        mp.maps[3] = p.tm_q2;
        mp.have = 3u | (p.p_groups ? 4u : 0u) | (p.q_groups ? 8u : 0u);
        mp.offsets = offsets;
        mp.groups = uint32_t(groups);
        mp.rows = uint32_t(rows);
        mp.out = static_cast<CUtensorMap *>(ws);
        p.maps = mp.out;
        void *args[1] = {&mp};
        st = launch(reinterpret_cast<const void *>(&ragged_maps_kernel), dim3(unsigned(groups), 1, 1), 128, 0, 1, args, stream);
        if (st != GEMM_OK) return st;
    }
    st = launch_ragged(variant, dev, p, most, stream);
    if (st != GEMM_OK || !part_rows) return st;
    RaggedPartsParams add;
    add.parts = static_cast<const float4 *>(ws);
    add.offsets = offsets;
    add.out = out;
    add.groups = uint32_t(groups);
    add.rows = uint32_t(rows);
    add.part_rows = uint32_t(part_rows);
    add.quads = uint32_t(n * k / 4);
    add.out32 = out_type == GEMM_DTYPE_F32;
    add.bf16 = p.bf16;
    void *args[1] = {&add};
    return launch(reinterpret_cast<const void *>(&ragged_parts_kernel), dim3(unsigned(cdiv(add.quads, 256)), unsigned(groups), 1), 256, 0,
                  1, args, stream);
}

// ------------------------------------------------------------- adapters

constexpr int64_t kLoraURows = 64;  // rows of a tile of the product that computes u
// Rows and rank up to which one kernel takes both of the adapters' steps beside the projection (measured at the kernel).
constexpr int64_t kLoraRowsRows = 32, kLoraRowsRank = 32;

// Time (us) of the adapters row by row, without tensor cores: every row's a and b, from L2 mostly, at about 5 TB/s.
double lora_alone(int64_t rows, int64_t n, int64_t k, int64_t rank)
{
    return 2.0 * double(rows) * double(rank) * double(n + k) / 5e6;
}

// Rows whose items the adapters' two kernels can count: an item is four of a row's u's or 128 of its columns, and the 32-bit
// number of the last one, a stride of the grid further (sixteen blocks of four items an SM at most), does not wrap.
int64_t lora_beside_rows(int64_t n, int64_t rank)
{
    const int64_t each = rank / 4 > cdiv(n, 128) ? rank / 4 : cdiv(n, 128);
    return ((int64_t(1) << 32) - (int64_t(1) << 20)) / (each < 1 ? 1 : each);
}

// Whether the adapters run row by row beside the projection.  On the tensor cores each row tile takes K blocks for every
// adapter in it, 1.6 us of a worker's time for 64 of the rank, after some 15 us of launches that depend on one another.  How
// many adapters a tile of up to 256 rows has is in ids on the device: one where rows come in prompts, all where each row is
// a request of its own.  (adapters)^0.7 stands between: over 400 launches of random sizes (65 to 16000 rows, n 128 to 8192, k
// 128 to 4096, 1 to 256 adapters of rank 8 to 128, all even over their logarithms but the rank) it costs 21% over the faster
// way on average where each row is a request, at most 4.8 times, and 4.7% where rows come in up to 128 runs, at most 3.1
// times; all adapters cost 3.4% and 45%, at most 2.0 and 15.7 times, their square root 36% and 3.3%, at most 5.4 and 2.1.
// `pairs`: co-resident CTA pairs of the tensor cores' way.
bool lora_beside(int pairs, int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters)
{
    if (rows > lora_beside_rows(n, rank)) return false;
    if (rows <= kRagged[kVNtFew].qcap) return true;
    const RaggedVariant &y = kRagged[kVLoraY];
    const double waves = double(cdiv(n, 128 * y.cg)) * double(cdiv(rows, y.qcap)) / pairs;
    const double blocks = pow(double(adapters < y.qcap ? adapters : y.qcap), 0.7) * double(cdiv(rank, kRagBlockK));
    return lora_alone(rows, n, k, rank) < 15.0 + (waves < 1.0 ? 1.0 : waves) * blocks * 1.6;
}

// How the work and the workspace are laid out.  Beside: u and delta in fp32.  Otherwise: counts and lists
// of the adapters per row tile (of y's product and of u's), and u; rows beyond what the kernels' table holds go in passes.
struct LoraPlan {
    bool beside;
    int variant_y;
    bool split_y;          // beside: whether the projection's tiles are split
    int64_t per, tiles;    // y's row tiles, of one pass
    int64_t tiles_u;
    int64_t pass_rows;
    size_t counts, list, counts_u, list_u, u, delta, split, total;  // offsets
};

LoraPlan lora_layout(const RaggedDevice *dev, int64_t rows, int64_t n, int64_t k, int64_t rank, bool beside)
{
    LoraPlan l;
    memset(&l, 0, sizeof(l));
    l.beside = beside;
    // (4 us more: their launches.  Loops that end before the adapters do anyhow are not worth a join: 320 launches of
    // random sizes are 1.6% off the fastest of the four ways this way, 3.5% without)
    const RaggedChoice y_beside = grouped_choice(kNT, 1, rows, n, k, true, 4.0 + lora_alone(rows, n, k, rank), dev);
    l.variant_y = l.beside ? y_beside.variant : kVLoraY;
    l.split_y = l.beside && y_beside.split;
    const RaggedVariant &y = kRagged[l.variant_y];
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += size_t(round_up(int64_t(bytes), 256));
        return was;
    };
    if (l.beside) {
        l.pass_rows = rows;
        l.u = take(size_t(rows) * size_t(rank) * 4u);
        l.delta = take(size_t(rows) * size_t(n) * 4u);
        l.split = take(split_room(rows, k, dev));
        l.total = at;
        return l;
    }
    l.pass_rows = int64_t(kRagMaxGroups) * kLoraURows;
    if (rows < l.pass_rows) l.pass_rows = rows;
    l.tiles = cdiv(l.pass_rows, y.qcap);
    l.per = round_up(cdiv(l.pass_rows, l.tiles), 16 * y.cg);
    l.tiles_u = cdiv(l.pass_rows, kLoraURows);
    l.counts = take(size_t(l.tiles) * 4u);
    l.list = take(size_t(l.tiles) * size_t(l.per) * 4u);
    l.counts_u = take(size_t(l.tiles_u) * 4u);
    l.list_u = take(size_t(l.tiles_u) * size_t(kLoraURows) * 4u);
    l.u = take(size_t(l.pass_rows) * size_t(rank) * 4u);  // in two parts of the operands' type
    size_t split = split_bytes(kRagged[kVLoraU], dev->slots[kVLoraU]);
    const size_t split_y = l.tiles == 1 ? split_bytes(y, dev->slots[l.variant_y]) : 0;
    if (split_y > split) split = split_y;
    l.split = take(split);
    l.total = at;
    return l;
}

LoraPlan lora_plan(const RaggedDevice *dev, int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters)
{
    return lora_layout(dev, rows, n, k, rank, lora_beside(dev->slots[kVLoraY], rows, n, k, rank, adapters));
}

// Bytes that serve any number of rows up to this one: the layout of the most rows that run beside the projection, that of
// all rows on the tensor cores, and that of the one row tile that is split.
size_t lora_bytes(const RaggedDevice *dev, int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters)
{
    size_t most = lora_plan(dev, rows, n, k, rank, adapters).total;
    const int64_t tile = kRagged[kVLoraY].qcap;
    if (rows > kRagged[kVNtFew].qcap) {
        const size_t one = lora_layout(dev, rows < tile ? rows : tile, n, k, rank, false).total;
        if (one > most) most = one;
    }
    // the limit of lora_beside is the same for all rows of a tile: the largest such row number of each tile, from the top
    const int64_t countable = lora_beside_rows(n, rank);
    for (int64_t top = rows < countable ? rows : countable; top > 0; top = (top - 1) / tile * tile) {
        const int64_t low = (top - 1) / tile * tile;
        int64_t lo = low, hi = top;  // beside holds up to lo (or nowhere in this tile), not from hi + 1 on
        while (lo < hi) {
            const int64_t mid = lo + (hi - lo + 1) / 2;
            if (lora_beside(dev->slots[kVLoraY], mid, n, k, rank, adapters)) lo = mid;
            else hi = mid - 1;
        }
        if (lo > low) {
            const size_t beside = lora_layout(dev, lo, n, k, rank, true).total;
            if (beside > most) most = beside;
            break;
        }
    }
    return most;
}

// `skip_fill`: of the product that writes y.
gemm_status_t lora(gemm_dtype_t dtype, int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters, const void *x,
                   const void *w, const void *a, const void *b, const int32_t *ids, const float *scale, void *y,
                   void *workspace, size_t ws_bytes, uint32_t skip_fill, long long wait_limit, cudaStream_t s)
{
    gemm_status_t st = check_sizes({rows, adapters}, {n, k, rank});
    if (st != GEMM_OK) return st;
    if (!operand_type(dtype)) return GEMM_ERR_INVALID_ARG;
    if (rank > GEMM_LORA_MAX_RANK) return GEMM_ERR_UNSUPPORTED_SHAPE;
    const bool any = rows > 0 && n > 0;
    const bool adapted = any && k > 0 && adapters > 0 && rank > 0;
    st = check_pointer(y, any);
    if (st == GEMM_OK) st = check_pointer(x, any && k > 0);
    if (st == GEMM_OK) st = check_pointer(w, any && k > 0);
    if (st == GEMM_OK) st = check_pointer(a, adapted);
    if (st == GEMM_OK) st = check_pointer(b, adapted);
    if (st == GEMM_OK) st = check_pointer(ids, adapted, 4);
    if (st == GEMM_OK && scale) st = check_pointer(scale, adapted, 4);
    if (st != GEMM_OK) return st;
    if (!any) return GEMM_OK;
    RaggedDevice *dev = nullptr;
    st = ragged_device(&dev);
    if (st != GEMM_OK) return st;
    const LoraPlan l = lora_plan(dev, rows, n, k, rank, adapters);
    if (workspace == nullptr || ws_bytes < l.total) return GEMM_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GEMM_ERR_ALIGNMENT;
    if (k == 0) {
        if (cudaMemsetAsync(y, 0, size_t(rows) * size_t(n) * 2u, s) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
        return GEMM_OK;
    }
    char *ws = static_cast<char *>(workspace);
    if (l.beside) {
        RaggedParams p;
        memset(&p, 0, sizeof(p));
        p.groups = 1;
        p.rows = uint32_t(rows);
        p.pdim = uint32_t(n);
        p.kdim = uint32_t(k);
        p.k_blocks = uint32_t(cdiv(k, kRagBlockK));
        const RaggedVariant &vy = kRagged[l.variant_y];
        p.tiles_p = uint32_t(cdiv(n, 128 * vy.cg));
        p.bf16 = dtype == GEMM_DTYPE_BF16;
        p.out = y;
        p.skip_fill = skip_fill;
        p.wait_limit = wait_limit ? wait_limit : wait_limit_for(p.k_blocks);
        st = encode_stack(&p.tm_p, w, dtype, 1, n, k, kRagBlockK, 128);
        if (st == GEMM_OK) st = encode_rows(p.tm_q, x, dtype, rows, k, vy.qbox);
        if (st != GEMM_OK) return st;
        if (adapted) {
            LoraFewParams f;
            f.x = x;
            f.a = a;
            f.b = b;
            f.ids = ids;
            f.scale = scale;
            f.u = reinterpret_cast<float *>(ws + l.u);
            f.delta = reinterpret_cast<float *>(ws + l.delta);
            f.rows = uint32_t(rows);
            f.n = uint32_t(n);
            f.k = uint32_t(k);
            f.rank = uint32_t(rank);
            f.adapters = uint32_t(adapters);
            f.bf16 = p.bf16;
            void *args[1] = {&f};
            const int64_t room = dev->num_sms;
            if (rows <= kLoraRowsRows && rank <= kLoraRowsRank) {
                st = launch(lora_rows_instance(rank), dim3(unsigned(rows * kLoraCluster), 1, 1), 128, 0, kLoraCluster,
                            args, s);
                if (st != GEMM_OK) return st;
            } else {
                // Few blocks on an SM where the product takes every SM's first CTA (64 rows with 64 adapters of rank 16,
                // 8192 x 4096: four and two 28.6 us, eight and four 30.5, one and two 33.5) or is the longer part, more where
                // its CTAs leave room (2749 rows, 17 adapters of rank 32, 160 x 216: 28.8 us, sixteen and eight 20.2; 139
                // rows, 3544 x 448: 16.9 and 13.7).  Warps for items where eight blocks an SM would not hold them (913 rows,
                // 208 x 304, rank 48: 33.2 us by blocks, 23.0 by warps; but 1024 items of 8192 x 4096 44.4 and 53.0).
                const bool roomy = !l.split_y && vy.cg == 1;
                const int64_t shrink = rows * (rank / 4), expand = cdiv(rows * cdiv(n, 128), 4);
                const bool warps = shrink > 8 * room;
                const int64_t most_shrink = (roomy ? 16 : 4) * room, most_expand = (roomy ? 8 : 2) * room;
                const int64_t blocks = warps ? cdiv(shrink, 4) : shrink;
                st = launch(warps ? reinterpret_cast<const void *>(&lora_shrink_kernel<1>)
                                  : reinterpret_cast<const void *>(&lora_shrink_kernel<4>),
                            dim3(unsigned(blocks < most_shrink ? blocks : most_shrink), 1, 1), 128, 0, 1, args, s);
                if (st != GEMM_OK) return st;
                st = launch(lora_expand_instance(rank), dim3(unsigned(expand < most_expand ? expand : most_expand), 1, 1), 128,
                            0, 1, args, s);
                if (st != GEMM_OK) return st;
            }
            p.delta = f.delta;
            p.ids = ids;
            p.adapters = f.adapters;
        }
        int64_t most = most_tiles(vy, 1, rows, n);
        if (most >= kSizeLimit) return GEMM_ERR_UNSUPPORTED_SHAPE;
        if (l.split_y && most * p.k_blocks < kIterLimit) {
            use_split(&p, vy, dev->slots[l.variant_y], ws + l.split);
            most *= p.k_blocks;
        }
        return launch_ragged(l.variant_y, dev, p, most, s);
    }
    const RaggedVariant &vu = kRagged[kVLoraU], &vy = kRagged[l.variant_y];

    RaggedParams u, p;
    memset(&u, 0, sizeof(u));
    u.kdim = uint32_t(k);
    u.k_blocks = uint32_t(cdiv(k, kRagBlockK));
    u.bf16 = dtype == GEMM_DTYPE_BF16;
    u.scale = scale;
    u.adapters = adapted ? uint32_t(adapters) : 0u;
    u.rank = uint32_t(rank);
    u.rank_blocks = uint32_t(cdiv(rank, kRagRank));
    u.skip_fill = ~0u;
    u.wait_limit = wait_limit ? wait_limit : wait_limit_for(cdiv(k, kRagBlockK) + 4096);
    p = u;
    p.skip_fill = skip_fill;
    // y = x w^T + u b^T
    p.pdim = uint32_t(n);
    p.tiles_p = uint32_t(cdiv(n, 128 * vy.cg));
    p.per = uint32_t(l.per);
    p.u = ws + l.u;
    st = encode_stack(&p.tm_p, w, dtype, 1, n, k, kRagBlockK, 128);
    if (st == GEMM_OK && adapted) st = encode_stack(&p.tm_x, b, dtype, adapters, n, rank, kRagBlockK, 128);
    if (!adapted) p.tm_x = p.tm_p;  // (never loaded from)
    // u = scale x a^T for many rows: one tile per row tile and adapter in it
    if (adapted) {
        u.pdim = uint32_t(rank);
        u.tiles_p = 1;
        u.per = uint32_t(kLoraURows);
        u.out = ws + l.u;
        if (st == GEMM_OK) st = encode_stack(&u.tm_p, a, dtype, adapters, rank, k, kRagBlockK, 128);
    }
    if (st != GEMM_OK) return st;
    if (int64_t(p.tiles_p) * l.tiles >= kSizeLimit) return GEMM_ERR_UNSUPPORTED_SHAPE;

    for (int64_t r0 = 0; r0 < rows; r0 += l.pass_rows) {
        const int64_t r = rows - r0 < l.pass_rows ? rows - r0 : l.pass_rows;
        const int64_t tiles = cdiv(r, l.per);
        const char *xr = static_cast<const char *>(x) + size_t(r0) * size_t(k) * 2u;
        const int32_t *idr = adapted ? ids + r0 : nullptr;
        p.groups = uint32_t(tiles);
        p.tiles_q = uint32_t(tiles);
        p.rows = uint32_t(r);
        p.ids = idr;
        p.out = static_cast<char *>(y) + size_t(r0) * size_t(n) * 2u;
        st = encode_rows(p.tm_q, xr, dtype, r, k, vy.qbox);
        if (st != GEMM_OK) return st;
        {
            const int64_t tiles_u = adapted ? cdiv(r, kLoraURows) : 0;
            LoraListParams lp;
            lp.ids = idr;
            lp.rows = uint32_t(r);
            lp.adapters = u.adapters;
            lp.tiles = uint32_t(tiles);
            lp.per[0] = uint32_t(l.per);
            lp.per[1] = uint32_t(kLoraURows);
            lp.counts[0] = reinterpret_cast<int32_t *>(ws + l.counts);
            lp.counts[1] = reinterpret_cast<int32_t *>(ws + l.counts_u);
            lp.list[0] = reinterpret_cast<int32_t *>(ws + l.list);
            lp.list[1] = reinterpret_cast<int32_t *>(ws + l.list_u);
            void *args[1] = {&lp};
            st = launch(reinterpret_cast<const void *>(&lora_list_kernel), dim3(unsigned(tiles + tiles_u), 1, 1), 256, 0, 1, args, s);
            if (st != GEMM_OK) return st;
            p.counts = reinterpret_cast<int32_t *>(ws + l.counts);
            p.list = reinterpret_cast<int32_t *>(ws + l.list);
            if (adapted) {
                u.counts = reinterpret_cast<int32_t *>(ws + l.counts_u);
                u.list = reinterpret_cast<int32_t *>(ws + l.list_u);
                u.groups = uint32_t(tiles_u);
                u.rows = uint32_t(r);
                u.ids = idr;
                st = encode_rows(u.tm_q, xr, dtype, r, k, vu.qbox);
                if (st != GEMM_OK) return st;
                u.sk = 0;
                if (r * int64_t(u.k_blocks) < kIterLimit) use_split(&u, vu, dev->slots[kVLoraU], ws + l.split);
                st = launch_ragged(kVLoraU, dev, u, r * int64_t(u.k_blocks), s);
                if (st != GEMM_OK) return st;
            }
        }
        int64_t most = int64_t(p.tiles_p) * tiles;
        p.sk = 0;
        if (l.tiles == 1 && most * (p.k_blocks + l.per * p.rank_blocks) < kIterLimit) {
            use_split(&p, vy, dev->slots[l.variant_y], ws + l.split);
            most *= p.k_blocks;
        }
        st = launch_ragged(l.variant_y, dev, p, most, s);
        if (st != GEMM_OK) return st;
    }
    return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t gemm_grouped_workspace_size(int64_t groups, int64_t rows, int64_t n, int64_t k, size_t *bytes)
{
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_sizes({groups, rows}, {n, k});
    if (st != GEMM_OK) return st;
    if (groups > GEMM_GROUPED_MAX_GROUPS) return GEMM_ERR_UNSUPPORTED_SHAPE;
    RaggedDevice *dev = nullptr;
    st = ragged_device(&dev);
    if (st != GEMM_OK) return st;
    // what any number of rows up to this one may need, so that a buffer for the most rows serves them all
    *bytes = maps_bytes(groups);
    for (size_t room : {split_room(rows, n > k ? n : k, dev), part_room(groups, rows, n, k, dev)})
        if (room > *bytes) *bytes = room;
    return GEMM_OK;
}

gemm_status_t gemm_grouped_nt(gemm_dtype_t dtype, int64_t groups, int64_t rows, int64_t n, int64_t k, const int32_t *offsets,
                              const void *x, const void *w, void *y, void *workspace, size_t ws_bytes, gemm_stream_t stream)
{
    return grouped(kNT, dtype, dtype, groups, rows, n, k, offsets, x, w, y, workspace, ws_bytes, ~0u, 0,
                   reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_grouped_nn(gemm_dtype_t dtype, int64_t groups, int64_t rows, int64_t n, int64_t k, const int32_t *offsets,
                              const void *dy, const void *w, void *dx, void *workspace, size_t ws_bytes, gemm_stream_t stream)
{
    return grouped(kNN, dtype, dtype, groups, rows, n, k, offsets, dy, w, dx, workspace, ws_bytes, ~0u, 0,
                   reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_grouped_tn(gemm_dtype_t dtype, gemm_dtype_t out, int64_t groups, int64_t rows, int64_t n, int64_t k,
                              const int32_t *offsets, const void *dy, const void *x, void *dw, void *workspace, size_t ws_bytes,
                              gemm_stream_t stream)
{
    return grouped(kTN, dtype, out, groups, rows, n, k, offsets, dy, x, dw, workspace, ws_bytes, ~0u, 0,
                   reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_grouped_stall_test(int32_t mode, gemm_dtype_t dtype, int64_t groups, int64_t rows, int64_t n, int64_t k,
                                      const int32_t *offsets, const void *first, const void *second, void *out, void *workspace,
                                      size_t ws_bytes, uint32_t skip_fill, long long wait_limit_cycles, gemm_stream_t stream)
{
    if (mode < kNT || mode > kTN || wait_limit_cycles <= 0) return GEMM_ERR_INVALID_ARG;
    return grouped(mode, dtype, dtype, groups, rows, n, k, offsets, first, second, out, workspace, ws_bytes, skip_fill,
                   wait_limit_cycles, reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_lora_workspace_size(int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters, size_t *bytes)
{
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_sizes({rows, adapters}, {n, k, rank});
    if (st != GEMM_OK) return st;
    if (rank > GEMM_LORA_MAX_RANK) return GEMM_ERR_UNSUPPORTED_SHAPE;
    RaggedDevice *dev = nullptr;
    st = ragged_device(&dev);
    if (st != GEMM_OK) return st;
    *bytes = rows ? lora_bytes(dev, rows, n, k, rank, adapters) : 0;
    return GEMM_OK;
}

gemm_status_t gemm_lora_way(int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters, int32_t num_sms, int32_t *way)
{
    if (!way || num_sms < 0 || num_sms == 1) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_sizes({rows, adapters}, {n, k, rank});
    if (st != GEMM_OK) return st;
    if (rank > GEMM_LORA_MAX_RANK) return GEMM_ERR_UNSUPPORTED_SHAPE;
    int pairs = num_sms / 2;
    if (num_sms == 0) {
        RaggedDevice *dev = nullptr;
        st = ragged_device(&dev);
        if (st != GEMM_OK) return st;
        pairs = dev->slots[kVLoraY];
    }
    *way = lora_beside(pairs, rows, n, k, rank, adapters) ? GEMM_LORA_BESIDE : GEMM_LORA_TENSOR_CORES;
    return GEMM_OK;
}

gemm_status_t gemm_lora_nt(gemm_dtype_t dtype, int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters,
                           const void *x, const void *w, const void *a, const void *b, const int32_t *ids, const float *scale,
                           void *y, void *workspace, size_t ws_bytes, gemm_stream_t stream)
{
    return lora(dtype, rows, n, k, rank, adapters, x, w, a, b, ids, scale, y, workspace, ws_bytes, ~0u, 0,
                reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_lora_stall_test(gemm_dtype_t dtype, int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters,
                                   const void *x, const void *w, const void *a, const void *b, const int32_t *ids,
                                   const float *scale, void *y, void *workspace, size_t ws_bytes, uint32_t skip_fill,
                                   long long wait_limit_cycles, gemm_stream_t stream)
{
    if (wait_limit_cycles <= 0) return GEMM_ERR_INVALID_ARG;
    return lora(dtype, rows, n, k, rank, adapters, x, w, a, b, ids, scale, y, workspace, ws_bytes, skip_fill, wait_limit_cycles,
                reinterpret_cast<cudaStream_t>(stream));
}

// --------------------------------------------------------------- router

static gemm_status_t check_route(gemm_dtype_t dtype, int64_t rows, int64_t experts, int64_t top)
{
    gemm_status_t st = check_sizes({rows, experts, top}, {});
    if (st != GEMM_OK) return st;
    if (dtype != GEMM_DTYPE_F16 && dtype != GEMM_DTYPE_BF16 && dtype != GEMM_DTYPE_F32) return GEMM_ERR_INVALID_ARG;
    if (experts < 1 || top < 1 || top > experts) return GEMM_ERR_INVALID_ARG;
    if (experts > GEMM_ROUTE_MAX_EXPERTS || top > GEMM_ROUTE_MAX_TOP || rows * top >= kSizeLimit)
        return GEMM_ERR_UNSUPPORTED_SHAPE;
    return GEMM_OK;
}

static int64_t route_blocks(int64_t rows)
{
    return rows <= kRouteFewRows ? 1 : cdiv(rows, kRouteRows);
}

gemm_status_t gemm_route_workspace_size(int64_t rows, int64_t experts, int64_t top, size_t *bytes)
{
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_route(GEMM_DTYPE_F32, rows, experts, top);
    if (st != GEMM_OK) return st;
    const int64_t blocks = route_blocks(rows);
    *bytes = blocks > 1 ? size_t(blocks + 1) * size_t(experts) * 4u : 0;
    return GEMM_OK;
}

// The instance of a kernel whose lanes hold enough values for `experts`.
#define ROUTE_INSTANCE(F, experts)                                                                                       \
    ((experts) <= 32    ? F(1)                                                                                           \
     : (experts) <= 64  ? F(2)                                                                                           \
     : (experts) <= 128 ? F(4)                                                                                           \
     : (experts) <= 256 ? F(8)                                                                                           \
     : (experts) <= 512 ? F(16)                                                                                          \
                        : F(32))
#define ROUTE_TOPK_FEW(V) reinterpret_cast<const void *>(&route_topk_kernel<V, kRouteThreads>)
#define ROUTE_TOPK(V) reinterpret_cast<const void *>(&route_topk_kernel<V, 16 * kRouteRows>)
#define ROUTE_GRAD(V) reinterpret_cast<const void *>(&route_grad_kernel<V>)

gemm_status_t gemm_route_topk(gemm_dtype_t dtype, int64_t rows, int64_t experts, int64_t top, int32_t renorm, const void *logits,
                              int32_t *ids, float *weights, int32_t *offsets, int32_t *order, int32_t *position, void *workspace,
                              size_t ws_bytes, gemm_stream_t stream)
{
    gemm_status_t st = check_route(dtype, rows, experts, top);
    if (st != GEMM_OK) return st;
    const bool any = rows > 0;
    st = check_pointer(logits, any);
    if (st == GEMM_OK) st = check_pointer(offsets, true, 4);
    for (const void *ptr : {static_cast<const void *>(ids), static_cast<const void *>(weights), static_cast<const void *>(order),
                            static_cast<const void *>(position)})
        if (st == GEMM_OK) st = check_pointer(ptr, any, 4);
    if (st != GEMM_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    DeviceState state;
    st = current_device_state(&state);
    if (st != GEMM_OK) return st;
    if (!any) {
        if (cudaMemsetAsync(offsets, 0, size_t(experts + 1) * 4u, s) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
        return GEMM_OK;
    }
    const int64_t blocks = route_blocks(rows);
    if (blocks > 1) {
        if (workspace == nullptr || ws_bytes < size_t(blocks + 1) * size_t(experts) * 4u) return GEMM_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GEMM_ERR_ALIGNMENT;
    }
    RouteParams p;
    memset(&p, 0, sizeof(p));
    p.logits = logits;
    p.dtype = uint32_t(dtype);
    p.rows = uint32_t(rows);
    p.experts = uint32_t(experts);
    p.top = uint32_t(top);
    p.renorm = renorm != 0;
    p.blocks = uint32_t(blocks);
    p.ids = ids;
    p.weights = weights;
    p.offsets = offsets;
    p.order = order;
    p.position = position;
    p.hist = static_cast<int32_t *>(workspace);
    p.totals = p.hist ? p.hist + size_t(blocks) * size_t(experts) : nullptr;
    void *args[1] = {&p};
    if (blocks == 1) return launch(ROUTE_INSTANCE(ROUTE_TOPK_FEW, experts), dim3(1, 1, 1), kRouteThreads, 0, 1, args, s);
    st = launch(ROUTE_INSTANCE(ROUTE_TOPK, experts), dim3(unsigned(blocks), 1, 1), 16 * kRouteRows, 0, 1, args, s);
    if (st != GEMM_OK) return st;
    if (blocks > kRouteDirectBlocks)
        st = launch(reinterpret_cast<const void *>(&route_scan_kernel), dim3(unsigned(cdiv(experts, 32)), 1, 1), 1024, 0, 1, args, s);
    if (st != GEMM_OK) return st;
    return launch(reinterpret_cast<const void *>(&route_place_kernel), dim3(unsigned(blocks), 1, 1), kRouteThreads, 0, 1, args, s);
}

gemm_status_t gemm_route_topk_grad(gemm_dtype_t dtype, int64_t rows, int64_t experts, int64_t top, int32_t renorm,
                                   const void *logits, const int32_t *ids, const float *weights, const float *dweights,
                                   float *dlogits, gemm_stream_t stream)
{
    gemm_status_t st = check_route(dtype, rows, experts, top);
    if (st != GEMM_OK) return st;
    const bool any = rows > 0;
    st = check_pointer(logits, any);
    for (const void *ptr : {static_cast<const void *>(ids), static_cast<const void *>(weights),
                            static_cast<const void *>(dweights), static_cast<const void *>(dlogits)})
        if (st == GEMM_OK) st = check_pointer(ptr, any, 4);
    if (st != GEMM_OK || !any) return st;
    DeviceState state;
    st = current_device_state(&state);
    if (st != GEMM_OK) return st;
    RouteParams p;
    memset(&p, 0, sizeof(p));
    p.logits = logits;
    p.dtype = uint32_t(dtype);
    p.rows = uint32_t(rows);
    p.experts = uint32_t(experts);
    p.top = uint32_t(top);
    p.renorm = renorm != 0;
    p.ids = const_cast<int32_t *>(ids);
    p.weights = const_cast<float *>(weights);
    p.dweights = dweights;
    p.dlogits = dlogits;
    void *args[1] = {&p};
    return launch(ROUTE_INSTANCE(ROUTE_GRAD, experts), dim3(unsigned(cdiv(rows, 8)), 1, 1), 256, 0, 1, args,
                  reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
