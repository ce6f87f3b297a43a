/*
 * pts_experts.h -- C ABI of the routed-experts operators in 8-bit floating point
 * for MI355X (gfx950): quantisation to e4m3 with block scales, the dense and the
 * per-expert product of such matrices, the router, and the combination of the
 * experts' outputs.
 *
 * The calls take plain pointers and sizes, keep no state and allocate nothing:
 * any number may run at once, on any streams, and each may be recorded into a
 * HIP graph (they launch kernels and nothing else). Everything about memory,
 * streams, status codes and gemm_last_error() is as stated in pts_gemm.h: all
 * pointers are device memory of the caller on the current device, every call is
 * asynchronous on `stream`, arguments are checked before anything is launched,
 * and operands that overlap an output are not detected. A problem that takes 2^32
 * threads or more in one launch (from 2^26 tokens in the router, 2^27 rows or 2^36
 * elements in the quantiser, 2^28 columns in a product on) may be
 * GEMM_ERR_UNSUPPORTED.
 *
 * e4m3 is the OCP 8-bit format (largest finite value 448, no infinities).
 * "fp32 scale per block" means: the value of element (i, k) is
 * code[i][k] * scale[block of (i, k)]; a block is 128 consecutive k of one row,
 * or 128 rows by 128 k. The last block of a row (or column of blocks) may be
 * shorter.
 */
#ifndef PTS_EXPERTS_H
#define PTS_EXPERTS_H

#include "pts_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PTS_FP8_BLOCK 128
#define PTS_MOE_MAX_EXPERTS 1024
#define PTS_MOE_MAX_TOP 32
#define PTS_MOE_MAX_GROUPS 64

typedef enum { PTS_SCORE_SOFTMAX = 0, PTS_SCORE_SIGMOID = 1 } pts_score;

/*
 * Quantise x (m x k, bf16 or fp32) to e4m3.
 *   scale = max(max |x| over the block / 448, 2^-126)   (fp32 division)
 *   q     = x / scale (fp32 division), rounded to nearest, ties to even
 * A block with an infinity or a NaN gets a NaN scale and NaN codes.
 *
 * layout_x: GEMM_ROW_MAJOR (x[i * ldx + k], ldx >= the row's length) or
 *   GEMM_COL_MAJOR (x[k * ldx + i], ldx >= m).
 * block_m: 1 or 128 rows per block (always 128 k).
 * swiglu: non-zero quantises g / (1 + exp(-g)) * u instead, where row i of x
 *   holds g in its first k and u in its next k elements (so 2 k per row);
 *   row-major, block_m = 1 only. The product is formed in fp32, to 7 * 2^-24 of
 *   its value (for g below -87 also to 2^-149 |g u|, exp's least step), and not
 *   rounded in between.
 * q: m rows of k codes, row stride ldq >= k, a multiple of 16, q 16-byte
 *   aligned; the bytes from k up to the next multiple of 16 are written as 0.
 * scale: element (row or row block i, k block b) at i * scale_stride_m +
 *   b * scale_stride_k (strides >= 1; elements must be distinct).
 */
gemm_status pts_quantize_fp8(const void *x, int32_t dtype_x, int32_t layout_x, int64_t m, int64_t k, int64_t ldx,
                             int32_t block_m, int32_t swiglu, void *q, int64_t ldq, float *scale,
                             int64_t scale_stride_m, int64_t scale_stride_k, void *stream);

/*
 * D = A . B for e4m3 A (m x k) and B (k x n, given as its transpose: column j of
 * B is row j of b), D fp32 or bf16 (dtype_d), m x n, row-major:
 *   D[i][j] = sum over k blocks, ascending, of
 *             (a_scale[i] b_scale[j]) * (sum of the block's products)
 * The sums over k blocks are fp32, one accumulator per element (for few rows: one
 * per eighth of the blocks, added in a fixed order), so results are
 * deterministic. Inside a block, for fp32 output the products are exact and summed
 * in fp32. For bf16 output the matrix unit sums the 8-bit products in groups of 8
 * consecutive k, and what lies 14 binary places below a group's largest product is
 * dropped (2^-13 of that product each at most, 1.4e-5 of a result on normal data,
 * against the 2^-8 of its one rounding to nearest, ties to even).
 *
 * a, b: 16-byte aligned, lda and ldb multiples of 16 and >= k; rows are read in
 *   whole 16-byte pieces (up to k rounded up to 16), bytes past k do not count.
 * a_scale: element (i, kb) at i * a_scale_stride_m + kb * a_scale_stride_k.
 * b_scale: element (j / b_block_n, kb) at (j / b_block_n) * b_scale_stride_n +
 *   kb * b_scale_stride_k, b_block_n = 1 or 128. (The weights' gradient has both
 *   operands scaled per row: b_block_n = 1.)
 * ldd >= n; elements outside m x n are not written. k = 0 gives zeros.
 * m, n < 2^31 - 1024. Strides for which a tile's offsets would not fit in 32
 *   bits (lda or ldb of 2^23 and more) are GEMM_ERR_UNSUPPORTED.
 */
gemm_status pts_gemm_fp8(const void *a, int64_t lda, const float *a_scale, int64_t a_scale_stride_m,
                         int64_t a_scale_stride_k, const void *b, int64_t ldb, const float *b_scale,
                         int64_t b_scale_stride_n, int64_t b_scale_stride_k, int32_t b_block_n, void *d, int64_t ldd,
                         int32_t dtype_d, int64_t m, int64_t n, int64_t k, void *stream);

/*
 * The same product for each expert over its own rows: rows
 * [offsets[e], offsets[e + 1]) of D are (rows of A) . B_e.
 *
 * offsets: experts + 1 device int32, non-decreasing within [0, m]; rows of D in
 *   no expert's range (before the first offset, behind the last) are left as
 *   they were. Values outside [0, m] are taken as the nearest inside, and a
 *   table that decreases leaves D's first m rows undefined; neither leads
 *   outside the operands.
 * rows: device int32 [m], the row of A that each row of D reads (outside
 *   [0, a_rows): the nearest); NULL: row i of D reads row i of A (a_rows >= m).
 * b: expert e at b + e * b_stride_expert, each n x k as in pts_gemm_fp8, with
 *   128 x 128 blocks; b_stride_expert a multiple of 16 elements.
 * 1 <= experts <= PTS_MOE_MAX_EXPERTS. With `rows`, A must span less than 4 GiB
 *   and its scales 2 GiB (GEMM_ERR_UNSUPPORTED otherwise).
 */
gemm_status pts_gemm_fp8_experts(const void *a, int64_t a_rows, int64_t lda, const float *a_scale,
                                 int64_t a_scale_stride_m, int64_t a_scale_stride_k, const void *b, int64_t ldb,
                                 int64_t b_stride_expert, const float *b_scale, int64_t b_scale_stride_expert,
                                 int64_t b_scale_stride_n, int64_t b_scale_stride_k, int32_t experts,
                                 const int32_t *offsets, const int32_t *rows, void *d, int64_t ldd, int32_t dtype_d,
                                 int64_t m, int64_t n, int64_t k, void *stream);

/*
 * Choose `top` experts for each of m tokens from its logits (m x experts, bf16
 * or fp32, row stride ld), and put the m * top slots in order by expert.
 *   p = softmax(logits) or 1 / (1 + exp(-logits));  c = p + bias (bias may be NULL)
 *   groups > 1 (a divisor of experts): a group's score is the largest c of its
 *     experts / groups consecutive experts, or the sum of its two largest
 *     (group_top2); the topk_groups best groups stay, ties to the lower group
 *   ids[t][..] = the experts of the `top` largest c, largest first, ties to the
 *     lower index; c is compared in 64 bits (without a bias by the logits)
 *   weights[t][j] = scale * p / (sum of the chosen p + 1e-20) if renormalize,
 *     else scale * p
 * An expert whose logit or c is -inf or NaN is closed to the token. Slots left
 * without an open expert (a padded token's whole row, say) get id -1 and
 * weight 0. Where the softmax is not a number (a NaN or +inf logit) the choice
 * goes by the logits and the weights are NaN.
 *
 * The order (offsets NULL: not formed; then rows, positions and workspace are
 * not used): rows[p] = the token of the p-th row, positions[t][j] = the row of
 * slot (t, j); rows are by expert, then by slot. offsets[e] .. offsets[e + 1]
 * are expert e's rows (experts + 1 values). Slots without an expert take the
 * rows from offsets[experts] on, and their position is -2 - row.
 *
 * workspace: device memory of pts_moe_route_workspace() bytes (may be NULL where
 *   that is 0); calls that may overlap need one each.
 * top <= min(experts, PTS_MOE_MAX_TOP), experts <= PTS_MOE_MAX_EXPERTS,
 * groups <= PTS_MOE_MAX_GROUPS; m * top < 2^31.
 */
gemm_status pts_moe_route(const void *logits, int32_t dtype, int64_t ld, const float *bias, int64_t m, int32_t experts,
                          int32_t top, int32_t score, int32_t groups, int32_t topk_groups, int32_t group_top2,
                          int32_t renormalize, float scale, int32_t *ids, float *weights, int32_t *offsets,
                          int32_t *rows, int32_t *positions, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace pts_moe_route needs to form the order (0 for small m). */
int64_t pts_moe_route_workspace(int64_t m, int32_t experts, int32_t top);

/*
 * The gradient of the logits, from that of the weights (dweights, m x top, fp32)
 * and the choice `ids` (m x top; -1 or any value outside [0, experts): no
 * expert). dlogits has the logits' dtype, row stride ld_d; all of m x experts is
 * written. The choice has no gradient, so neither has the bias. An expert named
 * twice gets the sum. With sigmoid scores an expert that is not named gets 0,
 * whatever its logit (a NaN that closes it, say).
 */
gemm_status pts_moe_route_backward(const float *dweights, const void *logits, int32_t dtype, int64_t ld,
                                   const int32_t *ids, int64_t m, int32_t experts, int32_t top, int32_t score,
                                   int32_t renormalize, float scale, void *dlogits, int64_t ld_d, void *stream);

/*
 * out[t] = sum_j weights[t][j] * y[positions[t][j]], j ascending, in fp32; y
 * (rows x n) and out (m x n) bf16 or fp32, the same. A position outside
 * [0, rows) adds nothing (its weight is not looked at). m < 2^24, n <= 2^26 - 1024,
 * top <= PTS_MOE_MAX_TOP, for the gradients too.
 */
gemm_status pts_moe_combine(const void *y, int32_t dtype, int64_t ldy, int64_t rows, const float *weights,
                            const int32_t *positions, int64_t m, int64_t n, int32_t top, void *out, int64_t ld_out,
                            void *stream);

/*
 * Its gradients: dy[positions[t][j]] = weights[t][j] * dout[t] and
 * dweights[t][j] = sum over n of dout[t] * y[positions[t][j]] (fp32). A position
 * outside [0, rows) has dweights 0; a position -2 - p with p in [0, rows) sets
 * row p of dy to 0. Rows of dy that no position names are left as they were; no
 * two slots may name the same row. dy must not be y.
 */
gemm_status pts_moe_combine_backward(const void *dout, int64_t ld_dout, const void *y, int32_t dtype, int64_t ldy,
                                     int64_t rows, const float *weights, const int32_t *positions, int64_t m,
                                     int64_t n, int32_t top, void *dy, int64_t ld_dy, float *dweights, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PTS_EXPERTS_H */
