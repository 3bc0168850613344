// C ABI of the products with an epilogue and of their gradients (declared in
// include/gemm_linear.h): argument validation, the choice of kernel variant,
// workspace layout, tensor maps and launches.  The kernels are in
// ragged_kernel.cuh (the product), linear_act.cuh and linear_kernel.cuh.
#include <math.h>

#include "linear_kernel.cuh"
#include "ragged_launch.cuh"

using namespace gemm_f16;

namespace {

enum LinearVariantId { kVNtWide, kVNtFew, kVNnWide, kVNnFew, kVSumWide, kVSumFew };
const RaggedVariant kLinear[] = {
    RAGGED_VARIANT(kNT, 2, 256, 6, true),       RAGGED_VARIANT(kNT, 1, 64, 8, true),
    RAGGED_VARIANT(kNN, 2, 256, 6, true),       RAGGED_VARIANT(kNN, 1, 64, 8, true),
    RAGGED_VARIANT(kNN, 2, 256, 6, true, true), RAGGED_VARIANT(kNN, 1, 64, 8, true, true),
};
using LinearDevice = RaggedDeviceOf<int(sizeof(kLinear) / sizeof(kLinear[0]))>;

gemm_status_t linear_device(LinearDevice **out)
{
    return ragged_device_of(kLinear, nullptr, 0, nullptr, 0, out);
}

// What splitting the last wave costs, us: 3000 rows, 5000 x 4096 86.1 -> 78.4, 2500 rows, 4096 x 8192 120.7 -> 98.4, but 4096 rows,
// 4096 x 1024 33.9 -> 44.0 and 8192 rows, 2048 x 512 29.6 -> 39.2.
constexpr double kSplitLastGain = 13.0;

int64_t live_groups(int64_t groups, int64_t rows)
{
    return groups < rows ? groups : rows;
}

// Bytes of the partial sums of a bias gradient: a line for each piece of `per` rows.
size_t sums_bytes(int64_t per, int64_t groups, int64_t rows, int64_t cols)
{
    return size_t(round_up((rows / per + live_groups(groups, rows)) * cols * 4, 256));
}

// How linear_grad_kernel cuts a matrix of so many columns: threads to a row of a strip (their logarithm), and strips.
struct GradStrips {
    int lanes;
    int64_t count;
};

GradStrips grad_strips(int64_t cols)
{
    const int64_t quads = cols / 8;
    GradStrips best = {5, cdiv(quads, 32)};
    double use = 0.0;
    for (int lanes = 5; lanes >= 3; --lanes) {
        const int64_t count = cdiv(quads, int64_t(1) << lanes);
        const double u = double(quads) / double(count << lanes);
        if (u > use + 0.1) {  // (wide strips read longer pieces of a row)
            use = u;
            best = {lanes, count};
        }
    }
    return best;
}

// Rows of a piece of linear_grad_kernel, in whole rounds of its threads: as many pieces as the SMs hold twice (once, three or
// four times: 16384 x 4096 68.3, 69.2, 68.9 and 70.2 us, 8192 x 8192 71.6, 66.6, 66.2 and 65.9, 65536 x 1024 69.6, 70.3, 73.1
// and 74.6), or small ones.
constexpr int64_t kGradRows = 32;

int64_t grad_pieces(int64_t cols, int num_sms)  // of one group, at most
{
    const int64_t most = 2 * kLinearGradBlocks * int64_t(num_sms) / grad_strips(cols).count;
    return most < 1 ? 1 : most;
}

int64_t grad_rows(int64_t rows, int64_t cols, int num_sms)
{
    return round_up(cdiv(rows, grad_pieces(cols, num_sms)), kGradRows);
}

// What any number of rows up to this one may need for the partial sums of linear_grad_kernel.
size_t grad_room(int64_t groups, int64_t rows, int64_t cols, int num_sms)
{
    if (cols == 0) return 0;
    const int64_t pieces = grad_pieces(cols, num_sms), small = cdiv(rows, kGradRows);
    return size_t(round_up(((pieces < small ? pieces : small) + live_groups(groups, rows)) * cols * 4, 256));
}

gemm_status_t check_linear(gemm_dtype_t dtype, gemm_act_t act, int64_t groups, int64_t rows, int64_t n, int64_t k,
                           const int32_t *offsets)
{
    gemm_status_t st = check_sizes({groups, rows}, {n, k});
    if (st != GEMM_OK) return st;
    if (!operand_type(dtype) || act < GEMM_ACT_NONE || act > GEMM_ACT_SILU) return GEMM_ERR_INVALID_ARG;
    if (groups < 1 || (groups > 1 && rows > 0 && offsets == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (groups > GEMM_GROUPED_MAX_GROUPS) return GEMM_ERR_UNSUPPORTED_SHAPE;
    return check_pointer(offsets, offsets != nullptr, 4);
}

// Whether the tiles of pairs that fill no wave are split over K, so that all pairs end together: for groups of equal size, by
// what the last wave leaves idle against a join.
bool split_last_wave(const RaggedVariant &v, int slots, int64_t groups, int64_t rows, int64_t pdim, int64_t kdim)
{
    const int64_t live = live_groups(groups, rows), each = rows / live;
    const double share = double(live * cdiv(each, v.qcap) * cdiv(pdim, 128 * v.cg)) / slots;
    if (share < 1.0) return false;
    const double part = each < v.qcap ? double(each) / v.qcap : 1.0;
    const double tile = double(cdiv(kdim, kRagBlockK)) * (0.226 + 0.08 * part) + 0.8 + 1.76 * part;
    return (ceil(share) - share) * tile > kSplitLastGain;
}

// How a product runs, and what it needs of a workspace: partial sums of a bias gradient, then those of split tiles.
struct LinearPlan {
    int variant;
    bool split, split_last;  // over K: all tiles, or those of the last wave
    bool whole;              // the sums of one tile are dbias
    size_t sums, need;
};

LinearPlan linear_plan(const LinearDevice &dev, int mode, bool grouped, bool bias_grad, int64_t groups, int64_t rows, int64_t pdim,
                       int64_t kdim, bool workspace)
{
    const int few = mode == kNT ? kVNtFew : bias_grad ? kVSumFew : kVNnFew, wide = mode == kNT ? kVNtWide : bias_grad ? kVSumWide : kVNnWide;
    const RaggedChoice choice =
        ragged_choice(kLinear[few], dev.slots[few], kLinear[wide], dev.slots[wide], groups, rows, pdim, kdim, workspace, 0.0);
    LinearPlan p;
    p.variant = choice.wide ? wide : few;
    const RaggedVariant &var = kLinear[p.variant];
    p.split = choice.split;
    p.split_last = choice.wide && !choice.split && workspace && split_last_wave(var, dev.slots[p.variant], groups, rows, pdim, kdim);
    p.whole = !grouped && rows <= var.qcap;
    p.sums = bias_grad && !p.whole ? sums_bytes(var.qcap, groups, rows, pdim) : 0;
    p.need = p.sums + (p.split || p.split_last ? split_bytes(var, dev.slots[p.variant]) : 0);
    return p;
}

// What the products of these sizes, or of fewer rows, may need.  Up to a single CTA's rows pairs split tiles for wide layers
// alone, where their last wave is (28672 x 8192, 64 rows 79.5 us and 86.3 unsplit; 22016 x 4096, one row 32.5 and 41.0), and the
// space for that, four times the single CTAs', is asked for there only.
size_t linear_room(const LinearDevice &dev, int64_t groups, int64_t rows, int64_t n, int64_t k)
{
    const int64_t one = kLinear[kVNtFew].qcap;
    size_t split = split_bytes(kLinear[kVNtFew], dev.slots[kVNtFew]), room = 0;
    if (rows > one)
        for (int v : {kVNtWide, kVNnWide, kVSumWide}) {
            const size_t wide = split_bytes(kLinear[v], dev.slots[v]);
            if (wide > split) split = wide;
        }
    for (int64_t r = 1; r <= rows && r <= one; ++r)
        for (int way = 0; way < 3; ++way) {
            const LinearPlan p = linear_plan(dev, way == 0 ? kNT : kNN, true, way == 2, groups, r, way == 0 ? n : k, way == 0 ? k : n, true);
            if (p.need > room) room = p.need;
        }
    const size_t most = sums_bytes(one, groups, rows, k) + split;  // (the pairs' sums have fewer lines)
    return most > room ? most : room;
}

// The chains of a contraction with column sums.  A whole tile's first one runs while the epilogue has the other accumulator for the
// end of the tile before, so it is long, and the others make up for its error (16384 rows, 4096 x 4096, beside one chain: chains
// of 13 blocks +10%, a first one of 18 +6.6%, of 22 +4% but an error of 9.9e-7; 20 and the others 9 +5.7%, 8.5e-7).
void ragged_chains(uint32_t blocks, uint32_t *first, uint32_t *chain)
{
    const uint32_t most = 20, others = 9;
    const uint32_t two = uint32_t(cdiv(2 * int64_t(blocks), cdiv(blocks, kRagChain) + 1));
    *first = blocks <= uint32_t(kRagChain) ? blocks : two < most ? two : most;
    const uint32_t rest = blocks - *first;
    *chain = rest == 0 ? others : uint32_t(cdiv(rest, cdiv(rest, others)));
}

// A bias gradient of no rows.
gemm_status_t zero_bias(float *dbias, int64_t count, cudaStream_t stream)
{
    if (dbias == nullptr || count == 0) return GEMM_OK;
    LinearDevice *dev = nullptr;
    gemm_status_t st = linear_device(&dev);
    if (st != GEMM_OK) return st;
    if (cudaMemsetAsync(dbias, 0, size_t(count) * 4u, stream) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

gemm_status_t launch_sum(const float *sums, const int32_t *offsets, float *dbias, int64_t groups, int64_t rows, int64_t cols,
                         int64_t per, cudaStream_t stream)
{
    LinearSumParams p;
    p.sums = sums;
    p.offsets = offsets;
    p.dbias = dbias;
    p.groups = uint32_t(groups);
    p.rows = uint32_t(rows);
    p.per = uint32_t(per);
    p.cols = uint32_t(cols);
    void *args[1] = {&p};
    return launch(reinterpret_cast<const void *>(&linear_sum_kernel), dim3(unsigned(cdiv(cols, 32)), unsigned(groups), 1),
                  kLinearThreads, 0, 1, args, stream);
}

// mode kNT: first = x, in = residual, out = y; mode kNN: first = dy, in = z, out = dx.
gemm_status_t linear(int mode, gemm_dtype_t dtype, gemm_act_t act, int64_t groups, int64_t rows, int64_t n, int64_t k,
                     const int32_t *offsets, const void *first, const void *w, const void *bias, const void *in, void *kept,
                     void *out, float *dbias, void *ws, size_t ws_bytes, uint32_t skip_fill, long long wait_limit,
                     cudaStream_t stream)
{
    gemm_status_t st = check_linear(dtype, act, groups, rows, n, k, offsets);
    if (st != GEMM_OK) return st;
    const int64_t pdim = mode == kNT ? n : k, kdim = mode == kNT ? k : n;
    const bool any = rows > 0 && pdim > 0;
    if (mode == kNN && act == GEMM_ACT_NONE) in = nullptr;
    if (any && kdim == 0) return GEMM_ERR_UNSUPPORTED_SHAPE;
    st = check_pointer(out, any);
    if (st == GEMM_OK) st = check_pointer(first, any);
    if (st == GEMM_OK) st = check_pointer(w, any);
    if (st == GEMM_OK) st = check_pointer(in, any && (in != nullptr || (mode == kNN && act != GEMM_ACT_NONE)));
    if (st == GEMM_OK) st = check_pointer(bias, any && bias != nullptr);
    if (st == GEMM_OK) st = check_pointer(kept, any && kept != nullptr);
    if (st == GEMM_OK) st = check_pointer(dbias, pdim > 0 && dbias != nullptr);
    if (st != GEMM_OK) return st;
    if (!any) return zero_bias(dbias, groups * pdim, stream);
    LinearDevice *dev = nullptr;
    st = linear_device(&dev);
    if (st != GEMM_OK) return st;
    const LinearPlan plan = linear_plan(*dev, mode, offsets != nullptr, dbias != nullptr, groups, rows, pdim, kdim, ws != nullptr);
    const int variant = plan.variant;
    const RaggedVariant &var = kLinear[variant];
    if (ws != nullptr || ws_bytes != 0 || plan.sums > 0) {
        if (ws == nullptr || ws_bytes < plan.need) return GEMM_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(ws) & 255u) return GEMM_ERR_ALIGNMENT;
    }
    LinearParams p;
    memset(&p, 0, sizeof(p));
    p.offsets = offsets;
    p.groups = uint32_t(groups);
    p.rows = uint32_t(rows);
    p.pdim = uint32_t(pdim);
    p.kdim = uint32_t(kdim);
    p.k_blocks = uint32_t(cdiv(kdim, kRagBlockK));
    p.tiles_p = uint32_t(cdiv(pdim, 128 * var.cg));
    p.bf16 = dtype == GEMM_DTYPE_BF16;
    p.out = out;
    p.skip_fill = skip_fill;
    p.wait_limit = wait_limit ? wait_limit : wait_limit_for(p.k_blocks);
    p.bias = bias;
    p.in = in;
    p.kept = kept;
    p.sums = dbias == nullptr ? nullptr : plan.whole ? dbias : static_cast<float *>(ws);
    p.act = uint32_t(act);
    ragged_chains(p.k_blocks, &p.first, &p.chain);
    int64_t most = most_tiles(var, groups, rows, pdim);
    if (most >= kSizeLimit) return GEMM_ERR_UNSUPPORTED_SHAPE;
    st = encode_stack(&p.tm_p, w, dtype, groups, n, k, 64, mode == kNT ? 128 : 64);
    if (st == GEMM_OK && mode == kNN) st = encode_pairs(&p.tm_p2, w, dtype, groups, n, k, &p.p_groups);
    if (st == GEMM_OK) st = encode_rows(p.tm_q, first, dtype, rows, kdim, var.qbox);
    if (st != GEMM_OK) return st;
    if ((plan.split || plan.split_last) && most * p.k_blocks < kIterLimit) {
        use_split(&p, var, dev->slots[variant], static_cast<char *>(ws) + plan.sums);
        if (plan.split_last) p.sk = 2;
        most *= p.k_blocks;
    }
    st = launch_variant(var, dev->slots[variant], dev->error_word, p, &p, most, stream);
    if (st != GEMM_OK || plan.sums == 0) return st;
    return launch_sum(p.sums, offsets, dbias, groups, rows, pdim, var.qcap, stream);
}

}  // namespace

extern "C" {

gemm_status_t gemm_linear_workspace_size(int64_t groups, int64_t rows, int64_t n, int64_t k, size_t *bytes)
{
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_sizes({groups, rows}, {n, k});
    if (st != GEMM_OK) return st;
    if (groups < 1) return GEMM_ERR_INVALID_ARG;
    if (groups > GEMM_GROUPED_MAX_GROUPS) return GEMM_ERR_UNSUPPORTED_SHAPE;
    LinearDevice *dev = nullptr;
    st = linear_device(&dev);
    if (st != GEMM_OK) return st;
    *bytes = 0;
    if (rows == 0) return GEMM_OK;
    if (n > 0 && k > 0) *bytes = linear_room(*dev, groups, rows, n, k);
    const size_t grad = grad_room(groups, rows, n, dev->num_sms);
    if (grad > *bytes) *bytes = grad;
    return GEMM_OK;
}

gemm_status_t gemm_linear_nt(gemm_dtype_t dtype, gemm_act_t act, int64_t groups, int64_t rows, int64_t n, int64_t k,
                             const int32_t *offsets, const void *x, const void *w, const void *bias, const void *residual, void *z,
                             void *y, void *workspace, size_t ws_bytes, gemm_stream_t stream)
{
    return linear(kNT, dtype, act, groups, rows, n, k, offsets, x, w, bias, residual, z, y, nullptr, workspace, ws_bytes, ~0u, 0,
                  reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_linear_nn(gemm_dtype_t dtype, gemm_act_t act, int64_t groups, int64_t rows, int64_t n, int64_t k,
                             const int32_t *offsets, const void *dy, const void *w, const void *z, void *dx, float *dbias,
                             void *workspace, size_t ws_bytes, gemm_stream_t stream)
{
    return linear(kNN, dtype, act, groups, rows, n, k, offsets, dy, w, nullptr, z, nullptr, dx, dbias, workspace, ws_bytes, ~0u, 0,
                  reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_linear_grad(gemm_dtype_t dtype, gemm_act_t act, int64_t groups, int64_t rows, int64_t n, const int32_t *offsets,
                               const void *dy, const void *z, void *dz, float *dbias, void *workspace, size_t ws_bytes,
                               gemm_stream_t stream)
{
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    gemm_status_t st = check_linear(dtype, act, groups, rows, n, 0, offsets);
    if (st != GEMM_OK) return st;
    const bool any = rows > 0 && n > 0;
    st = check_pointer(dy, any);
    if (st == GEMM_OK) st = check_pointer(z, any && act != GEMM_ACT_NONE);
    if (st == GEMM_OK) st = check_pointer(dz, any && (dz != nullptr || act != GEMM_ACT_NONE));
    if (st == GEMM_OK) st = check_pointer(dbias, n > 0 && dbias != nullptr);
    if (st != GEMM_OK) return st;
    if (!any) return zero_bias(dbias, groups * n, s);
    if (dz == nullptr && dbias == nullptr) return GEMM_OK;
    LinearDevice *dev = nullptr;
    st = linear_device(&dev);
    if (st != GEMM_OK) return st;
    const int64_t per = grad_rows(rows, n, dev->num_sms), strips = grad_strips(n).count;
    const bool whole = offsets == nullptr && rows <= per;  // the sums of one piece are dbias
    const size_t need = dbias && !whole ? sums_bytes(per, groups, rows, n) : 0;
    if (workspace != nullptr || ws_bytes != 0 || need > 0) {
        if (workspace == nullptr || ws_bytes < need) return GEMM_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GEMM_ERR_ALIGNMENT;
    }
    const int64_t blocks = (rows / per + live_groups(groups, rows)) * strips;  // at most: a group's last piece may be a part of one
    if (blocks >= kSizeLimit) return GEMM_ERR_UNSUPPORTED_SHAPE;
    LinearGradParams p;
    p.dy = dy;
    p.z = act == GEMM_ACT_NONE ? nullptr : z;
    p.dz = dz;
    p.sums = dbias == nullptr ? nullptr : whole ? dbias : static_cast<float *>(workspace);
    p.offsets = offsets;
    p.groups = uint32_t(groups);
    p.rows = uint32_t(rows);
    p.cols = uint32_t(n);
    p.per = uint32_t(per);
    p.lanes = uint32_t(grad_strips(n).lanes);
    p.strips = uint32_t(strips);
    p.act = uint32_t(act);
    p.bf16 = dtype == GEMM_DTYPE_BF16;
    void *args[1] = {&p};
    st = launch(reinterpret_cast<const void *>(&linear_grad_kernel), dim3(unsigned(blocks), 1, 1), kLinearThreads, 0, 1, args, s);
    if (st != GEMM_OK || need == 0) return st;
    return launch_sum(p.sums, offsets, dbias, groups, rows, n, per, s);
}

gemm_status_t gemm_linear_stall_test(int32_t mode, gemm_dtype_t dtype, gemm_act_t act, int64_t groups, int64_t rows, int64_t n,
                                     int64_t k, const int32_t *offsets, const void *first, const void *w, const void *extra,
                                     void *out, float *dbias, void *workspace, size_t ws_bytes, uint32_t skip_fill,
                                     long long wait_limit_cycles, gemm_stream_t stream)
{
    if ((mode != kNT && mode != kNN) || wait_limit_cycles <= 0) return GEMM_ERR_INVALID_ARG;
    return linear(mode, dtype, act, groups, rows, n, k, offsets, first, w, nullptr, extra, nullptr, out, mode == kNN ? dbias : nullptr,
                  workspace, ws_bytes, skip_fill, wait_limit_cycles, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
