/*
 * gemm_linear.h -- C ABI of products with a bias, an activation and a residual in
 * their epilogue, and of their gradients, beside the products of gemm_f16.h and
 * gemm_ragged.h (same library, same status codes, same rules for streams,
 * ownership, alignment, workspaces and errors as gemm_ragged.h):
 *
 *   gemm_linear_nt     z = x w^T + bias;  y = f(z) + residual
 *   gemm_linear_nn     dx = (dy w) * f'(z), z what f was applied to one layer below;
 *                      dbias = sum of dx over the rows: that layer's bias
 *   gemm_linear_grad   dz = dy * f'(z) and dbias, where no product comes before
 *
 * dw is gemm_grouped_tn(dz, x) of gemm_ragged.h, dresidual is dy.
 *
 * Operands are fp16 or bf16, sums are fp32, every result is rounded once, to the
 * operands' type (dbias: fp32).  f is applied to z before z's rounding, f' to the
 * rounded z that the caller kept.
 */
#ifndef GEMM_LINEAR_H_
#define GEMM_LINEAR_H_

#include "gemm_ragged.h"

#ifdef __cplusplus
extern "C" {
#endif

/* f; the derivative of relu and relu2 at 0 is 0, gelu uses the normal distribution function, gelu_tanh
 * 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))), relu2 is relu(z)^2, silu z / (1 + e^-z). */
typedef enum gemm_act {
    GEMM_ACT_NONE = 0,
    GEMM_ACT_RELU = 1,
    GEMM_ACT_RELU2 = 2,
    GEMM_ACT_GELU = 3,
    GEMM_ACT_GELU_TANH = 4,
    GEMM_ACT_SILU = 5
} gemm_act_t;

/*
 * One weight matrix (offsets NULL, groups 1), or one per group of rows, as the
 * grouped products take them: offsets [groups + 1] int32 on the device, group g has
 * the rows [offsets[g], offsets[g + 1]), clamped and made monotone by the kernels.
 * Rows of no group have y, z, dx and dz zero and take no part in dbias; the dbias
 * of a group without rows is zero.
 *
 *   gemm_linear_nt     x [rows, k], w [groups, n, k], bias [groups, n] or NULL,
 *                      residual [rows, n] or NULL, y [rows, n], z [rows, n] or
 *                      NULL (x w^T + bias, for the backward pass)
 *   gemm_linear_nn     dy [rows, n], w [groups, n, k], z [rows, k] (not read for
 *                      GEMM_ACT_NONE), dx [rows, k], dbias [groups, k] fp32 or NULL
 *   gemm_linear_grad   dy [rows, n], z [rows, n] (not read for GEMM_ACT_NONE),
 *                      dz [rows, n], dbias [groups, n] fp32 or NULL
 *
 * y may be the residual itself, dx may be z, dz may be dy or z (in place); other
 * overlaps are undefined.  The sum of the product needs something to add up: the
 * contraction (k of nt, n of nn) must be > 0 (GEMM_ERR_UNSUPPORTED_SHAPE).  dz may
 * be NULL for GEMM_ACT_NONE, where it would be a copy of dy (with rows of no group
 * zero): it is not written then.
 *
 * gemm_linear_workspace_size: bytes that serve any of the three calls of these
 * sizes, or of fewer rows, on the current device (k 0 for gemm_linear_grad alone).
 * A workspace may be NULL/0 all the same where no dbias is asked for (it costs time
 * where there are few rows); dbias needs one (GEMM_ERR_WORKSPACE).
 */
gemm_status_t gemm_linear_workspace_size(int64_t groups, int64_t rows, int64_t n, int64_t k, size_t *bytes);
gemm_status_t gemm_linear_nt(gemm_dtype_t dtype, gemm_act_t act, int64_t groups, int64_t rows, int64_t n, int64_t k,
                             const int32_t *offsets, const void *x, const void *w, const void *bias, const void *residual,
                             void *z, void *y, void *workspace, size_t ws_bytes, gemm_stream_t stream);
gemm_status_t gemm_linear_nn(gemm_dtype_t dtype, gemm_act_t act, int64_t groups, int64_t rows, int64_t n, int64_t k,
                             const int32_t *offsets, const void *dy, const void *w, const void *z, void *dx, float *dbias,
                             void *workspace, size_t ws_bytes, gemm_stream_t stream);
gemm_status_t gemm_linear_grad(gemm_dtype_t dtype, gemm_act_t act, int64_t groups, int64_t rows, int64_t n,
                               const int32_t *offsets, const void *dy, const void *z, void *dz, float *dbias, void *workspace,
                               size_t ws_bytes, gemm_stream_t stream);

/*
 * Failure-detection hook for tests, as gemm_grouped_stall_test: `mode` 0 runs
 * gemm_linear_nt(first = x, w, extra = residual, out = y) without bias and z, `mode` 1
 * gemm_linear_nn(first = dy, w, extra = z, out = dx, dbias).
 */
gemm_status_t gemm_linear_stall_test(int32_t mode, gemm_dtype_t dtype, gemm_act_t act, int64_t groups, int64_t rows, int64_t n,
                                     int64_t k, const int32_t *offsets, const void *first, const void *w, const void *extra,
                                     void *out, float *dbias, void *workspace, size_t ws_bytes, uint32_t skip_fill,
                                     long long wait_limit_cycles, gemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_LINEAR_H_ */
