/*
 * gemm_ragged.h -- C ABI of the products whose second matrix depends on the
 * row, beside the dense product of gemm_f16.h (same library, same status
 * codes, same rules for streams, ownership and errors):
 *
 *   gemm_grouped_nt / _nn / _tn   products grouped by expert, ragged sizes: the
 *                                 forward product and its two gradients
 *   gemm_lora_nt                  a shared projection with a low-rank adapter of
 *                                 each row's own beside it
 *   gemm_route_topk / _grad       the router that makes the groups: top-k of the
 *                                 experts' logits, its weights, the rows sorted by
 *                                 expert, and the logits' gradient
 *
 * Operands are fp16 or bf16 (all matrices of a call the same), accumulation is
 * fp32, results are rounded once to the operands' type (round to nearest even).
 * Every matrix is row-major and densely packed.  Pointers are device pointers
 * of the current device, 16-byte aligned (GEMM_ERR_ALIGNMENT) and non-null where
 * their size is > 0 (GEMM_ERR_INVALID_ARG); n, k and rank are multiples of 8,
 * every size is < 2^31 (GEMM_ERR_UNSUPPORTED_SHAPE).  Launches are asynchronous
 * on `stream`; outputs are fully overwritten; an output that overlaps an input
 * is undefined.  The library allocates nothing and keeps nothing from one call
 * for the next.  Results repeat bit for bit on the same inputs and workspace
 * size.  Calls may be captured in a CUDA graph after a first call on the device.
 *
 * Workspaces are the caller's, 256-byte aligned, of any contents; calls that
 * share one must not overlap on the GPU.  One left over from an aborted launch
 * (GEMM_ERR_TIMEOUT) serves again, replays of that launch from a graph included.  A pipeline wait that runs past its limit is
 * reported by gemm_f16_take_device_error as for the dense product.
 */
#ifndef GEMM_RAGGED_H_
#define GEMM_RAGGED_H_

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gemm_dtype {
    GEMM_DTYPE_F16 = 0,
    GEMM_DTYPE_BF16 = 1,
    GEMM_DTYPE_F32 = 2 /* outputs of gemm_grouped_tn, logits of the router */
} gemm_dtype_t;

/* Largest number of groups of one call, and of an adapter's rank. */
#define GEMM_GROUPED_MAX_GROUPS 1024
#define GEMM_LORA_MAX_RANK 128
/* Largest number of experts and of choices per row of the router. */
#define GEMM_ROUTE_MAX_EXPERTS 1024
#define GEMM_ROUTE_MAX_TOP 32

/*
 * Grouped products.  Rows are sorted by group: group g has the rows
 * [offsets[g], offsets[g + 1]) (offsets: groups + 1 int32 on the device, read
 * by the kernel; no host copy is needed).  With g(t) the group of row t:
 *
 *   gemm_grouped_nt   y[t, :]  = x[t, :] . w[g(t)]^T     x [rows, k], w [groups, n, k], y [rows, n]
 *   gemm_grouped_nn   dx[t, :] = dy[t, :] . w[g(t)]      dy [rows, n], w [groups, n, k], dx [rows, k]
 *   gemm_grouped_tn   dw[g]    = dy_g^T . x_g            dy [rows, n], x [rows, k], dw [groups, n, k]
 *
 * Groups may be empty (their dw is zero).  Rows of no group (before offsets[0],
 * from offsets[groups] on) have y and dx zero and take no part in dw, so a
 * buffer may be larger than the rows it holds.  Offsets are not validated on the
 * host: the kernel clamps them to [0, rows] and takes the running maximum, so
 * wrong ones give wrong results but reach no other memory.
 * gemm_grouped_tn writes dw as `out` (the operands' type or GEMM_DTYPE_F32).
 * rows, n or groups == 0 is a no-op where it leaves no output; an empty
 * contraction writes zeros.  The contents of rows of other groups never reach a
 * result, whatever they hold (infinities, NaN).
 *
 * gemm_grouped_workspace_size: bytes that serve any of the three calls of these
 * sizes, or of fewer rows, on the current device (partial sums of split tiles and
 * of parts of a group's rows, tensor maps of the groups).  A workspace may be NULL/0 all the same: that costs time
 * where there are few rows, and in gemm_grouped_tn; one that is given but too
 * small is GEMM_ERR_WORKSPACE.
 */
gemm_status_t gemm_grouped_workspace_size(int64_t groups, int64_t rows, int64_t n, int64_t k, size_t *bytes);
gemm_status_t gemm_grouped_nt(gemm_dtype_t dtype, int64_t groups, int64_t rows, int64_t n, int64_t k,
                              const int32_t *offsets, const void *x, const void *w, void *y, void *workspace,
                              size_t ws_bytes, gemm_stream_t stream);
gemm_status_t gemm_grouped_nn(gemm_dtype_t dtype, int64_t groups, int64_t rows, int64_t n, int64_t k,
                              const int32_t *offsets, const void *dy, const void *w, void *dx, void *workspace,
                              size_t ws_bytes, gemm_stream_t stream);
gemm_status_t gemm_grouped_tn(gemm_dtype_t dtype, gemm_dtype_t out, int64_t groups, int64_t rows, int64_t n, int64_t k,
                              const int32_t *offsets, const void *dy, const void *x, void *dw, void *workspace,
                              size_t ws_bytes, gemm_stream_t stream);

/*
 * Shared projection with low-rank adapters, i = ids[t]:
 *
 *   y[t, :] = x[t, :] . w^T + scale[i] (x[t, :] . a[i]^T) . b[i]^T
 *
 * x [rows, k], w [n, k], a [adapters, rank, k], b [adapters, n, rank],
 * y [rows, n]; ids: rows int32 in any order, a row whose id is outside
 * [0, adapters) has no adapter; scale: adapters fp32, or NULL for 1.  The inner
 * product scale (x a^T) stays in fp32, or, where many rows go through the tensor
 * cores, is the sum of two values of the operands' type (and infinite beyond the
 * range of fp16, if that is the type); the two products are added in fp32 and
 * rounded once.  What an adapter holds reaches the rows that
 * have it and no others, infinities and NaN included (a product with an infinity
 * of b may come out as NaN).  The workspace is
 * required (GEMM_ERR_WORKSPACE); gemm_lora_workspace_size gives the bytes that
 * serve these sizes, or fewer rows, on the current device.
 */
gemm_status_t gemm_lora_workspace_size(int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters, size_t *bytes);
/* Which way a call of these sizes takes: row by row beside the projection, or as K blocks of it on the tensor cores.  For
 * the current device (num_sms 0), or, without touching one, for a device of num_sms SMs and half as many CTA pairs. */
enum { GEMM_LORA_BESIDE = 0, GEMM_LORA_TENSOR_CORES = 1 };
gemm_status_t gemm_lora_way(int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters, int32_t num_sms, int32_t *way);
gemm_status_t gemm_lora_nt(gemm_dtype_t dtype, int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters,
                           const void *x, const void *w, const void *a, const void *b, const int32_t *ids,
                           const float *scale, void *y, void *workspace, size_t ws_bytes, gemm_stream_t stream);

/*
 * Router: for every row of logits [rows, experts] (fp16, bf16 or fp32) the `top`
 * largest, ties to the lowest index, in falling order.
 *
 *   ids      [rows, top] int32      the experts
 *   weights  [rows, top] fp32       softmax over all experts at ids, divided by their sum if renorm != 0
 *   offsets  [experts + 1] int32    rows of each expert, as the grouped products take them
 *   order    [rows * top] int32     the choices t * top + j sorted by expert, rows of one expert in rising order
 *   position [rows, top] int32      where each choice stands in `order`
 *
 * An expert at -infinity is never chosen: a row with fewer than `top` others
 * has -1 in ids and position and 0 in weights for the rest, and `order` ends in as
 * many -1 as there are such choices (offsets[experts] counts the others).  A row
 * with a NaN or +infinity among its logits has NaN weights; NaN logits are
 * chosen after all others but before -infinity.
 *
 * The workspace (gemm_route_workspace_size: 0 bytes for up to 64 rows) is
 * required where its size is > 0 (GEMM_ERR_WORKSPACE).
 *
 * gemm_route_topk_grad: dlogits [rows, experts] fp32 from the weights' gradient
 * dweights [rows, top] fp32, with logits, ids and weights of the forward call:
 *   renorm:     dl[ids[j]] = w[j] (dw[j] - sum_i w[i] dw[i]), zero elsewhere
 *   otherwise:  dl[e] = p[e] (sum_j [e = ids[j]] dw[j] - sum_j w[j] dw[j])
 */
gemm_status_t gemm_route_workspace_size(int64_t rows, int64_t experts, int64_t top, size_t *bytes); /* or fewer rows */
gemm_status_t gemm_route_topk(gemm_dtype_t dtype, int64_t rows, int64_t experts, int64_t top, int32_t renorm,
                              const void *logits, int32_t *ids, float *weights, int32_t *offsets, int32_t *order,
                              int32_t *position, void *workspace, size_t ws_bytes, gemm_stream_t stream);
gemm_status_t gemm_route_topk_grad(gemm_dtype_t dtype, int64_t rows, int64_t experts, int64_t top, int32_t renorm,
                                   const void *logits, const int32_t *ids, const float *weights, const float *dweights,
                                   float *dlogits, gemm_stream_t stream);

/*
 * Failure-detection hook for tests, as gemm_f16_nt_run_stall_test: `mode` 0, 1, 2
 * runs gemm_grouped_nt, _nn or _tn (first and second the two operands in that
 * order; tn writes the operands' type) with ring fill `skip_fill` of CTA 0 left
 * undone while the device error word is clear, and waits limited to
 * `wait_limit_cycles`: captured in a graph, a first replay is aborted and the
 * next, before the error is taken, runs through.  No fault, trap or hang.
 */
gemm_status_t gemm_grouped_stall_test(int32_t mode, gemm_dtype_t dtype, int64_t groups, int64_t rows, int64_t n, int64_t k,
                                      const int32_t *offsets, const void *first, const void *second, void *out,
                                      void *workspace, size_t ws_bytes, uint32_t skip_fill, long long wait_limit_cycles,
                                      gemm_stream_t stream);
/* The same of gemm_lora_nt: a fill of the product that writes y. */
gemm_status_t gemm_lora_stall_test(gemm_dtype_t dtype, int64_t rows, int64_t n, int64_t k, int64_t rank, int64_t adapters,
                                   const void *x, const void *w, const void *a, const void *b, const int32_t *ids,
                                   const float *scale, void *y, void *workspace, size_t ws_bytes, uint32_t skip_fill,
                                   long long wait_limit_cycles, gemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_RAGGED_H_ */
