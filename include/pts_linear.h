/*
 * pts_linear.h -- C ABI of a linear layer in bf16 for MI355X (gfx950): the product
 * with bias, activation and residual, its gradients, and the orthogonalised
 * update of its weight.
 *
 * The calls take plain pointers and sizes, keep no state and allocate nothing:
 * any number may run at once, on any streams, and each may be recorded into a
 * HIP graph (they launch kernels and nothing else). Everything about memory,
 * streams, status codes and gemm_last_error() is as stated in pts_gemm.h: all
 * pointers are device memory of the caller on the current device, every call is
 * asynchronous on `stream`, arguments are checked before anything is launched,
 * and operands that overlap an output or the workspace are not detected.
 * Results are deterministic: no sum's order depends on timing.
 *
 * bf16 operands (x, w, dy, z) start 16-byte aligned and have row strides that are
 * multiples of 8 elements and below 2^22; rows are read in whole 16-byte pieces
 * (up to their width rounded up to 8), what lies past their width does not count.
 * Extents are below 2^31 - 1024. A problem that takes 2^32 threads or more in one
 * launch is GEMM_ERR_UNSUPPORTED.
 *
 * workspace: 16-byte aligned device memory of at least as many bytes as the
 *   function with _workspace in its name says for the sizes (may be NULL where
 *   that is 0; sizes that every call refuses: 0); calls that may overlap need one
 *   each.
 */
#ifndef PTS_LINEAR_H
#define PTS_LINEAR_H

#include "pts_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * relu(z) = max(z, 0) (a NaN stays)
 * gelu(z) = z Phi(z), Phi the normal distribution function
 * gelu_tanh(z) = z / (1 + exp(-2 sqrt(2 / pi) (z + 0.044715 z^3)))
 * silu(z) = z / (1 + exp(-z))
 */
typedef enum {
    PTS_ACTIVATION_NONE = 0,
    PTS_ACTIVATION_RELU = 1,
    PTS_ACTIVATION_GELU = 2,
    PTS_ACTIVATION_GELU_TANH = 3,
    PTS_ACTIVATION_SILU = 4
} pts_activation;

/*
 * z = x w^T + bias;  y = activation(z) + residual
 * x: m x k, w: n x k, bf16. bias: n elements of bf16 or fp32 (dtype_bias), or NULL.
 * y and residual (NULL: none): m x n, both bf16 or both fp32 (dtype_y), any row
 * strides >= n; the residual may be y itself. z_out (NULL: not written): z in
 * bf16, row stride ldz >= n. Products are exact, sums fp32; y and z are each
 * rounded once (y from the unrounded z). k = 0 gives z = bias. Elements outside
 * m x n are not written.
 */
gemm_status pts_linear(const void *x, int64_t ldx, const void *w, int64_t ldw, const void *bias, int32_t dtype_bias,
                       int32_t activation, const void *residual, int64_t ldr, void *y, int64_t ldy, int32_t dtype_y,
                       void *z_out, int64_t ldz, int64_t m, int64_t n, int64_t k, void *workspace,
                       size_t workspace_bytes, void *stream);
int64_t pts_linear_workspace(int64_t m, int64_t n, int64_t k);

/*
 * The gradients of that layer, from dy (m x n, bf16):
 *   dz = dy activation'(z);  dx = dz w;  dw = dz^T x;  dbias = sum over rows of dz
 * (the residual's is dy itself). z: m x n, bf16, as pts_linear wrote it; not looked
 * at (may be NULL) without an activation. activation'(0) of relu is 0.
 * dx: m x k, bf16; dw: n x k, bf16 or fp32 (dtype_dw); dbias: n fp32. A gradient
 * whose pointer is NULL is not computed; w is needed for dx only, x for dw only.
 * The matrix unit takes dz rounded to bf16 (without an activation it is dy, exact);
 * dbias is summed, in fp32, from the unrounded one. m = 0 gives dw = 0, dbias = 0.
 * For dbias alone the workspace of PTS_ACTIVATION_NONE is enough.
 */
gemm_status pts_linear_backward(const void *dy, int64_t ld_dy, const void *z, int64_t ldz, int32_t activation,
                                const void *x, int64_t ldx, const void *w, int64_t ldw, void *dx, int64_t ld_dx,
                                void *dw, int64_t ld_dw, int32_t dtype_dw, float *dbias, int64_t m, int64_t n,
                                int64_t k, void *workspace, size_t workspace_bytes, void *stream);
int64_t pts_linear_backward_workspace(int64_t m, int64_t n, int64_t k, int32_t activation);

/*
 * Newton-Schulz steps towards the orthogonal factor of each of a stack of
 * matrices x (rows x cols, bf16 or fp32):
 *   X = x / (|x|_F + eps)
 *   `steps` times: X = a X + b (X X^T) X + c (X X^T)^2 X
 * that is p(s) = a s + b s^3 + c s^5 of its singular values. out: bf16, rounded
 * from fp32. Up to 64 rows or columns X and its products are fp32 (its Gram
 * matrices fp64). Beyond, the products' operands are fp16 and their sums fp32; X,
 * between the steps, is fp16 and eight bits more.
 *
 * x: row stride ldx >= cols, matrix i at i * x_stride; out likewise (element
 * aligned; its matrices must not overlap). cols and the smaller of rows and cols
 * are at most 2^22 - 64, count 65535. 1 <= steps <= 64, eps > 0. The coefficients
 * must keep the singular values, which start within [0, 1], in fp16's reach:
 * GEMM_ERR_INVALID_VALUE if |p|, with the roundings of the steps before it, can
 * come above 8 or |b s^2 + c s^4| above 128 on the way. A matrix with an infinity
 * or a NaN comes out NaN; a matrix of zeros stays zero.
 */
gemm_status pts_orthogonalize(const void *x, int32_t dtype_x, int64_t ldx, int64_t x_stride, int64_t count,
                              int64_t rows, int64_t cols, int32_t steps, float a, float b, float c, double eps,
                              void *out, int64_t ld_out, int64_t out_stride, void *workspace, size_t workspace_bytes,
                              void *stream);
int64_t pts_orthogonalize_workspace(int64_t count, int64_t rows, int64_t cols, int32_t steps);

#ifdef __cplusplus
}
#endif

#endif /* PTS_LINEAR_H */
