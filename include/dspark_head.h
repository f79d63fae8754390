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
 *     z_v  = h_i . W_v + U[prev_i] . V_v      (bf16 products, fp32 sums)
 *     lse  = log sum_v exp z_v
 *     loss = lse - z[target_i]
 * The scores are computed a 256-entry tile at a time and never stored.  A row
 * whose target is negative is ignored: its loss and lse are 0 and nothing else
 * of it is read (it costs no arithmetic either).  NaN or infinite scores give
 * the NaN or infinity of the formula in their own row.
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
 * Limits: 1 <= M <= 2^20, 1 <= vocab < 2^30, d a multiple of 8 in [8, 65536],
 * rank a multiple of 8 in [0, 256].
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

#ifdef __cplusplus
}
#endif
#endif /* DSPARK_HEAD_H_ */
