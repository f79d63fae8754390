/*
 * dspark_head.h - C ABI for training the drafter's head and for making the
 * hidden states that it reads.  Part of libdspark.so; the conventions of
 * dspark.h hold (caller-owned device memory, asynchronous on `stream`, host
 * validation before any launch, nothing allocated, DSPARK_DEV_* bits in the
 * status word at offset 0 of a workspace, a workspace zero-filled once).
 *
 *   r = residual + dropout(x)                    dspark_residual_norm
 *   h = r / rms(r) * gain                        (dspark_dropout by itself)
 *   z = h W^T + U[prev] V^T                      dspark_head_loss
 *   loss = log sum_v exp z_v - z[target]         and, with gradients,
 *                                                dspark_head_loss_grad
 *
 * z is the score that dspark_chain_lmhead maximises while drafting ("DSpark on
 * MAX", section "What DSpark is", items 2-3): the same factors, types and
 * layouts, so a head trained here is the head that drafts there.
 */
#ifndef DSPARK_HEAD_H_
#define DSPARK_HEAD_H_

#include "dspark.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Loss.  For each of M rows (request x position, any order):
 *     z_v  = h_i . W_v + U[prev_i] . V_v      (bf16 products, fp32 sums: the
 *            tensor cores', truncated, over up to 64 x 16 products at a time, and
 *            the chunks' rounded to nearest)
 *     lse  = log sum_v exp z_v
 *     loss = lse - z[target_i]
 * The scores are computed a 256-entry tile at a time and never stored.  A row
 * whose target is negative is ignored: its loss and lse are 0 and nothing else
 * that it holds has an effect (it costs no arithmetic either).  NaN or infinite
 * scores give the NaN or infinity of the formula in their own row.
 *
 * h           bf16 [M, d], row i at i*h_stride elements; h_stride >= d and a
 *             multiple of 8; 16-byte aligned.
 * W           bf16 [vocab, d] row-major, 16-byte aligned.
 * U, V        bf16 [vocab, rank] row-major, 16-byte aligned; rank 0 = no bias,
 *             then U, V and prev are not used and may be NULL.
 * prev        [M] int32.  Outside [0, vocab): 0 is used, DSPARK_DEV_TOKEN_OOR.
 * target      [M] int32.  >= vocab: ignored, DSPARK_DEV_TOKEN_OOR.
 * loss, lse   out [M] fp32.
 * workspace   >= dspark_head_workspace_size(M, vocab, d, rank, 0) bytes (a
 *             workspace for the gradient is large enough), 256-byte aligned.
 * Limits: 1 <= M <= 2^20, 1 <= vocab < 2^30, ceil(M / 256) ceil(vocab / 256) <=
 * 2^30, d a multiple of 8 in [8, 65536], rank a multiple of 8 in [0, 256].
 * The rows are gathered, and dU summed, by looking through all rows' tokens once
 * for each block of rows, and for each row: for M = 131072 with as many different
 * tokens that is some 6 ms, and four times as much for twice the rows.
 * ------------------------------------------------------------------------ */
DSPARK_API size_t dspark_head_workspace_size(int32_t M, int32_t vocab, int32_t d, int32_t rank,
                                             int32_t grad);

DSPARK_API dspark_status dspark_head_loss(
    const void *h, int64_t h_stride, const void *W, const void *U, const void *V,
    const int32_t *prev, const int32_t *target,
    int32_t M, int32_t vocab, int32_t d, int32_t rank,
    float *loss, float *lse,
    void *workspace, size_t workspace_bytes, dspark_stream_t stream);

/* Gradient.  With G[i, v] = dloss_i (exp(z_v - lse_i) - [v = target_i]):
 *     dh = G W     dW = G^T h     dV = G^T U[prev]
 *     dU[t] = sum of (G V)_i over the rows with prev_i = t
 * z is computed again, a piece of the vocabulary at a time; G is held in bf16
 * for one piece (relative to the largest |dloss|, so a mean's equal weights
 * round nothing), sums in fp32, and the results are rounded once.  Nothing
 * depends on the order in which blocks run: the same inputs give the same bits.
 * exp(z - lse) is as good as lse is in fp32: off by up to 2^-24 of |lse|, and 1
 * for every entry of a row whose scores are all one mask's value (as large as
 * bf16's lowest, lse does not hold log vocab beside it).
 *
 * h ... target   as above.
 * lse            [M] fp32, as written by dspark_head_loss.
 * dloss          [M] fp32: the derivative of the objective by each row's loss
 *                (1 / n for a mean over n rows).  Not read for ignored rows.
 * dh             out bf16 [M, d], row i at i*dh_stride elements (>= d, a
 *                multiple of 8), 16-byte aligned; 0 for ignored rows.
 * dW, dU, dV     out bf16, laid out as W, U and V, 16-byte aligned, written in
 *                full (0 where no row contributes); dU, dV not used at rank 0.
 * workspace      >= dspark_head_workspace_size(M, vocab, d, rank, 1) bytes.
 */
DSPARK_API dspark_status dspark_head_loss_grad(
    const void *h, int64_t h_stride, const void *W, const void *U, const void *V,
    const int32_t *prev, const int32_t *target, const float *lse, const float *dloss,
    int32_t M, int32_t vocab, int32_t d, int32_t rank,
    void *dh, int64_t dh_stride, void *dW, void *dU, void *dV,
    void *workspace, size_t workspace_bytes, dspark_stream_t stream);

/* ------------------------------------------------------------------------
 * Residual stream.  r = residual + dropout(x); y = r / sqrt(mean r^2 + eps) *
 * gain, row by row (sums in fp32, from the unrounded r).
 *
 * x, residual    [M, d] of dtype (DSPARK_BF16 or DSPARK_F32), rows x_stride /
 *                residual_stride elements apart (>= d); residual NULL = none.
 * gain           [d] of dtype.
 * r              out [M, d] of dtype, or NULL; may be x or residual itself.
 * y              out [M, d]: of dtype, or DSPARK_E4M3 (one byte each, y_dtype)
 *                with scales: group 0 = one scale for a row, group 128 = one
 *                for each 128 columns (the last may be narrower).  scale =
 *                max |y| / 448 over its columns (1 where that fp32 quotient is
 *                0), and the byte is y / scale, divided in fp32 too, rounded to
 *                nearest even; scale is fp32
 *                [M, ceil(d / 128)] or [M], contiguous.  group and scale are
 *                not used when y is of dtype.  (The 8-bit form is for a layer
 *                outside this library: dspark_head_loss and dspark_chain_lmhead
 *                read bf16.)
 * rstd           out [M] fp32: 1 / sqrt(mean r^2 + eps), or NULL.
 * p              probability of dropping an element of x, 0 <= p <= 1; 0 = none.
 *                Rounded so that T = round(65536 (1 - p)) of 65536 values are
 *                kept; what is kept is multiplied by 65536 / T.  Element (i, c)
 *                is kept iff lane c % 8 (16 bits each, low half of a word
 *                first) of the words of Philox4x32-10 with counter (c / 8, i,
 *                2^31, offset) and key (seed low, seed high) is below T.  The
 *                same (seed, offset) gives the same mask here, in the gradient
 *                and in dspark_dropout; use a new offset for every use.
 * Any d and alignment to the element works; rows that are 16-byte aligned with
 * d a multiple of 8 are faster.  A NaN or infinity stays in its own row (in
 * its own element where it is dropped).
 * Limits: 1 <= M <= 2^30, 1 <= d <= 32768.
 * ------------------------------------------------------------------------ */
#define DSPARK_E4M3 2

DSPARK_API dspark_status dspark_residual_norm(
    const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
    const void *gain, int32_t dtype, int32_t M, int32_t d, float eps,
    float p, uint64_t seed, uint32_t offset,
    void *r, int64_t r_stride, void *y, int64_t y_stride, int32_t y_dtype,
    int32_t group, float *scale, float *rstd, dspark_stream_t stream);

/* Gradient.  With a = dy gain, xh = r rstd:
 *     dr'   = dr + rstd (a - xh mean(a xh))
 *     dresidual = dr',  dx = dropout(dr'),  dgain = sum over rows of dy xh
 * dy             [M, d]: derivative by y.
 * dr             [M, d]: derivative by r from elsewhere, or NULL.
 * r, rstd        as written by dspark_residual_norm.
 * dx, dresidual  out [M, d], either may be NULL; dx may be dy itself and
 *                dresidual dr itself.
 * dgain          out [d], or NULL.
 * workspace      >= dspark_norm_workspace_size(M, d) bytes, 256-byte aligned.
 * All of dtype with strides as above; rstd fp32.  dgain is summed in an order
 * fixed by M, d, dtype and whether the rows are aligned to 16 bytes, d being a
 * multiple of 8. */
DSPARK_API size_t dspark_norm_workspace_size(int32_t M, int32_t d);

DSPARK_API dspark_status dspark_residual_norm_grad(
    const void *dy, int64_t dy_stride, const void *dr, int64_t dr_stride,
    const void *r, int64_t r_stride, const void *gain, const float *rstd,
    int32_t dtype, int32_t M, int32_t d, float p, uint64_t seed, uint32_t offset,
    void *dx, int64_t dx_stride, void *dresidual, int64_t dresidual_stride, void *dgain,
    void *workspace, size_t workspace_bytes, dspark_stream_t stream);

/* y = residual + dropout(x), elements, mask and arguments as above; residual
 * may be NULL, y may be x or residual itself.  Its gradient by x is
 * dspark_dropout of dy with residual = NULL. */
DSPARK_API dspark_status dspark_dropout(
    const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
    int32_t dtype, int32_t M, int32_t d, float p, uint64_t seed, uint32_t offset,
    void *y, int64_t y_stride, dspark_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DSPARK_HEAD_H_ */
