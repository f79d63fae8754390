/*
 * dspark_target.h - C ABI for the target's pass over the verify list: from the
 * scheduler's draft lengths to the logits that dspark_greedy_verify reads.
 * Part of libdspark.so; the conventions of dspark.h hold (caller-owned device
 * memory, asynchronous on `stream`, host validation before any launch, nothing
 * allocated, DSPARK_DEV_* bits in the status word at offset 0 of a workspace, a
 * workspace zero-filled once, calls that share one never overlapping).
 *
 *   draft_len, lengths  ->  rows, positions, pages, slots   dspark_step_rows
 *   q, k, v             ->  rotated q; k and v in the cache dspark_rotary_append
 *   q, cache            ->  attention of a request's rows   dspark_tree_attention
 *   logits              ->  penalties, biases, masks        dspark_adjust_logits
 *   logits              ->  accepted tokens                 dspark_greedy_verify
 *
 * Rows.  A step feeds the target R rows (tokens), request-major; request n has the
 * rows cu_rows[n] .. cu_rows[n+1].  Row 0 of a request that samples is its last
 * committed token, the rows after it are its drafts; a request that does not
 * sample has the next tokens of its prompt.  ctx_len[n] tokens of the request are
 * in the cache before the step, and row j's key and value go to index
 * ctx_len[n] + j of the request.
 *
 * Trees.  tree [N, tree_width] holds a 64-bit mask a row: row j of request n
 * attends row i of its own request iff bit i of tree[n, j] is set (a descendant's
 * mask is its parent's and its own bit).  A request is a tree iff tree is given,
 * it has at most tree_width rows, and bit 0 of tree[n, 0] is set; otherwise it is
 * a chain, whose row j attends its rows 0 .. j.  Bits past a request's rows are
 * ignored.  tree_width <= 64.
 *
 * Pages.  A cache holds num_pages pages of page_size tokens (a power of two from
 * 16 to 256); block_table [N, max_pages] int32 names the pages of each request in
 * order, and a slot is page * page_size + offset.
 */
#ifndef DSPARK_TARGET_H_
#define DSPARK_TARGET_H_

#include "dspark.h"

#ifdef __cplusplus
extern "C" {
#endif

/* more device status bits */
#define DSPARK_DEV_PAGES_SHORT 64u  /* the free list or the block table was too short */
#define DSPARK_DEV_ROWS_SHORT 128u  /* more rows than the buffers hold: cut off */
#define DSPARK_DEV_LEN_OOR    256u  /* a length was negative or past its buffer: clamped */
#define DSPARK_DEV_PAGE_OOR   512u  /* a page outside [0, num_pages): left out */

/* ------------------------------------------------------------------------
 * Rows, pages and slots of a step, from lengths on the GPU; nothing is read back.
 *
 * Request n has draft_len[n] + 1 rows if it samples (draft_len clamped to [0, K]),
 * chunk_len[n] otherwise.  Rows past max_rows are cut off (DSPARK_DEV_ROWS_SHORT).
 * It needs ceil((ctx_len[n] + rows) / page_size) pages; those past the
 * page_count[n] it has are popped off the end of free_pages, request by request
 * (the first one popped is free_pages[free_count - 1]), and written to
 * block_table.  Pages that are not there are -1 (DSPARK_DEV_PAGES_SHORT), as are
 * the slots of their rows; so are the slots of rows on a page outside [0, num_pages),
 * whose number stays in the table (DSPARK_DEV_PAGE_OOR).
 *
 * draft_len      [N]; sampling_mask [N] uint8 or NULL (all sample); chunk_len [N]
 *                or NULL (0).
 * ctx_len        [N]: tokens in the cache (negative: 0, DSPARK_DEV_LEN_OOR).
 * tree           [N, tree_width] uint64 or NULL.
 * tokens         [N, tokens_width], rows tokens_stride apart, or NULL: each
 *                request's committed tokens by index, the last one (not in the
 *                cache yet) at ctx_len[n].  draft_tokens [N, K].
 * page_count     [N], within [0, max_pages]; free_pages [free_max]; free_count device
 *                scalar, within [0, free_max].  Counts outside are clamped,
 *                DSPARK_DEV_LEN_OOR.
 * block_table    [N, max_pages], rows table_stride apart: entries from
 *                page_count[n] on are written where pages are added.
 * page_count_out [N], free_count_out scalar: after the step's pages are taken; may
 *                be page_count and free_count themselves.
 * cu_rows        out [N+1]; cu_out out [N+1]: offsets of the sampling requests'
 *                rows alone (dspark_greedy_verify's order).
 * row_request    out [max_rows]: n.   position out [max_rows]: ctx_len[n] + depth,
 *                depth being j in a chain and the number of other rows that row j
 *                attends in a tree.   slot out [max_rows], or -1.
 * row_token      out [max_rows] or NULL (tokens NULL): draft_tokens[n, j-1] for row
 *                j > 0 of a sampling request, tokens[n, ctx_len[n] + j] otherwise
 *                (0 and DSPARK_DEV_TOKEN_OOR past tokens_width).
 * out_row        out [max_rows]: the row of each entry of cu_out's order.
 * Entries past cu_rows[N] (out_row: cu_out[N]) are left as they are.
 * Limits: 1 <= N <= 16384, 1 <= K <= 63, 1 <= max_rows <= 2^22, num_pages *
 * page_size < 2^31, max_pages * page_size < 2^31.
 * ------------------------------------------------------------------------ */
DSPARK_API dspark_status dspark_step_rows(
    const int32_t *draft_len, const uint8_t *sampling_mask, const int32_t *chunk_len,
    const int32_t *ctx_len, const uint64_t *tree, int32_t tree_width,
    const int32_t *tokens, int64_t tokens_stride, int32_t tokens_width,
    const int32_t *draft_tokens, int32_t N, int32_t K,
    const int32_t *page_count, const int32_t *free_pages, int32_t free_max,
    const int32_t *free_count,
    int32_t page_size, int32_t num_pages,
    int32_t *block_table, int64_t table_stride, int32_t max_pages,
    int32_t *page_count_out, int32_t *free_count_out,
    int32_t *cu_rows, int32_t *cu_out, int32_t max_rows,
    int32_t *row_request, int32_t *position, int32_t *slot, int32_t *row_token,
    int32_t *out_row,
    void *workspace, size_t workspace_bytes, dspark_stream_t stream);

/* ------------------------------------------------------------------------
 * Rotary positions.  The first rot columns of every head are pairs (a, b):
 *     a' = amplitude (a cos t - b sin t),   b' = amplitude (b cos t + a sin t),
 * t = position * f_i for pair i; the others are copied.  Columns i and i + rot / 2
 * make a pair, or 2i and 2i + 1 where interleaved.  inverse turns the other way,
 * which is the gradient: of q' = dspark_rotary(q), dq = dspark_rotary(dq',
 * inverse), with the same amplitude.
 *
 * dspark_rotary_table writes f_i as a fraction of a turn a position, in units of
 * 2^-64, to HOST memory (turns [rot / 2], copied to the device by the caller), so
 * that position * turns mod 2^64 is the angle at any position, to the 53 bits that
 * f_i is computed with:
 *     f_i = base^(-2i / rot)
 *     DSPARK_ROPE_LINEAR    f_i / factor
 *     DSPARK_ROPE_BY_PARTS  f_i (1 - w) + f_i / factor w, w a ramp over i from 0 at
 *                           lo = max(floor e(high), 0) to 1 at
 *                           hi = min(ceil e(low), rot - 1), with
 *                           e(b) = rot ln(original / (2 pi b)) / (2 ln base); a step
 *                           after lo where hi <= lo
 *     DSPARK_ROPE_BY_TURNS  f_i s + f_i / factor (1 - s), s = (u - low) / (high -
 *                           low) clamped to [0, 1], u = original f_i / (2 pi)
 * A factor so small that f_i is not finite is refused.
 *
 * q, q_out   [R, Hq, d] of dtype (DSPARK_BF16 or DSPARK_F32): row strides and head
 *            strides in elements, columns contiguous.  k, k_out [R, Hk, d] alike.
 *            q with Hq = 0, or k with Hk = 0, may be NULL.  The outputs may be the
 *            inputs themselves, with the same strides; else they do not overlap.
 * position   [R] int32, taken as it is (negative ones turn backwards).
 * n_rows     device scalar or NULL (R): rows from it on are left as they are.
 * turns      [rot / 2] uint64 device memory.
 * fp32 arithmetic, one rounding; sin and cos of the angle's nearest fp32 fraction of
 * a turn.  Rows that are 16-byte aligned, with d and the halves of rot multiples of
 * 16 bytes, are faster.
 * Limits: 0 <= R <= 2^22, Hq, Hk <= 1024, 2 <= rot <= d <= 1024, rot even.
 *
 * dspark_rotary_append also copies v and writes the rotated k, and v, to slot[row]
 * of a cache (a slot outside [0, num_pages * page_size) is not written; slots are
 * distinct): element (page, offset, head, column) at page * page_stride + offset *
 * token_stride + head * head_stride + column of k_cache and of v_cache (elements),
 * both of dtype.  Limits as above, and those of dspark_step_rows on pages.
 * ------------------------------------------------------------------------ */
#define DSPARK_ROPE_PLAIN    0
#define DSPARK_ROPE_LINEAR   1
#define DSPARK_ROPE_BY_PARTS 2
#define DSPARK_ROPE_BY_TURNS 3

DSPARK_API dspark_status dspark_rotary_table(int32_t rot, double base, int32_t scaling,
                                             double factor, double original, double low,
                                             double high, uint64_t *turns);

DSPARK_API dspark_status dspark_rotary(
    const void *q, int64_t q_stride, int64_t q_head_stride, int32_t Hq,
    const void *k, int64_t k_stride, int64_t k_head_stride, int32_t Hk,
    int32_t dtype, int32_t R, int32_t d, const int32_t *position, const int32_t *n_rows,
    const uint64_t *turns, int32_t rot, int32_t interleaved, int32_t inverse,
    float amplitude, void *q_out, int64_t q_out_stride, int64_t q_out_head_stride,
    void *k_out, int64_t k_out_stride, int64_t k_out_head_stride, dspark_stream_t stream);

DSPARK_API dspark_status dspark_rotary_append(
    const void *q, int64_t q_stride, int64_t q_head_stride, int32_t Hq,
    const void *k, int64_t k_stride, int64_t k_head_stride,
    const void *v, int64_t v_stride, int64_t v_head_stride, int32_t Hk,
    int32_t dtype, int32_t R, int32_t d, const int32_t *position, const int32_t *slot,
    const int32_t *n_rows, const uint64_t *turns, int32_t rot, int32_t interleaved,
    float amplitude, void *q_out, int64_t q_out_stride, int64_t q_out_head_stride,
    void *k_cache, void *v_cache, int64_t page_stride, int64_t token_stride,
    int64_t head_stride, int32_t page_size, int32_t num_pages, dspark_stream_t stream);

/* ------------------------------------------------------------------------
 * Attention of a step's rows over the paged cache, which holds the step's own keys
 * and values already.  For row j of request n and query head h, with the key head
 * h / (Hq / Hk):
 *     s_t = scale q . k_t  over the ctx_len[n] cached tokens and those of the
 *           request's rows that row j attends (see Trees)
 *     out = sum_t exp(s_t) v_t / sum_t exp(s_t),   lse = log sum_t exp(s_t)
 * bf16 products, fp32 sums and softmax; exp(s_t - m) is rounded to bf16 for the
 * product with v and summed unrounded.  A row that attends nothing (or only tokens
 * whose score is -inf) is 0, its lse -inf.  What a row does not attend has no effect
 * on it, NaN and infinities included; nor have tokens on pages outside [0,
 * num_pages) or past the table (left out, DSPARK_DEV_PAGE_OOR).
 *
 * q, out     bf16 [R, Hq, d], row and head strides in elements; out overlaps nothing
 *            that is read.
 * k_cache, v_cache  bf16, element (page, offset, head, column) as in
 *            dspark_rotary_append.
 * block_table [N, max_pages], rows table_stride apart.   ctx_len [N] (negative: 0,
 *            DSPARK_DEV_LEN_OOR).
 * cu_rows    [N+1]: as written by dspark_step_rows; rows past cu_rows[N] are left as
 *            they are.
 * max_len    no request has more rows (more: left as they are, DSPARK_DEV_LEN_OOR).
 * lse        out fp32 [R, Hq], contiguous, or NULL.
 * workspace  >= dspark_attention_workspace_size(N, max_len, Hq, Hk, d) bytes,
 *            256-byte aligned.
 * scale      positive, a normal number below 2^127.
 * All strides multiples of 8, all bases 16-byte aligned.
 * Limits: 1 <= N <= 16384, 1 <= R <= 2^22, Hq a multiple of Hk, Hq / Hk <= 128, Hq <=
 * 1024, d a multiple of 8 in [8, 256], num_pages * page_size < 2^31, max_pages *
 * page_size < 2^30.
 * ------------------------------------------------------------------------ */
DSPARK_API size_t dspark_attention_workspace_size(int32_t N, int32_t max_len, int32_t Hq,
                                                  int32_t Hk, int32_t d);

DSPARK_API dspark_status dspark_tree_attention(
    const void *q, int64_t q_stride, int64_t q_head_stride,
    const void *k_cache, const void *v_cache, int64_t page_stride, int64_t token_stride,
    int64_t head_stride, int32_t page_size, int32_t num_pages,
    const int32_t *block_table, int64_t table_stride, int32_t max_pages,
    const int32_t *ctx_len, const int32_t *cu_rows, const uint64_t *tree, int32_t tree_width,
    int32_t N, int32_t R, int32_t max_len, int32_t Hq, int32_t Hk, int32_t d, float scale,
    void *out, int64_t out_stride, int64_t out_head_stride, float *lse,
    void *workspace, size_t workspace_bytes, dspark_stream_t stream);

/* ------------------------------------------------------------------------
 * Penalties for repeated tokens, biases and masks on the logits of each request's
 * rows, in this order, for token v of row j of request n:
 *     x = logits
 *     x = x > 0 ? x / repetition[n] : x * repetition[n]   if v was seen
 *     x = x - frequency[n] * c                            c times generated
 *     x = x - presence[n]                                 if c > 0
 *     x = x + sum of bias_value[n, i] over bias_token[n, i] = v
 *     x = -inf                                            if masked
 * in fp32, each operation rounded, and rounded once more to the logits' type.  Seen:
 * among the request's hist_len[n] committed tokens, or generated on row j's path.
 * Generated (c): committed at prompt_len[n] or later, and the drafts on row j's
 * path: draft_tokens[n, i-1] for every row i >= 1 that row j attends (see Trees).
 *
 * logits, out  [R, vocab] of dtype (DSPARK_BF16 or DSPARK_F32), rows stride elements
 *              apart.  out may be logits: then only what changes is written; else
 *              they do not overlap.
 * cu_rows      [N+1]: the requests' rows among the logits' (cu_out of
 *              dspark_step_rows).  Rows past cu_rows[N] are left as they are.
 * tokens       [N, tokens_width], rows tokens_stride apart: the buffer's first columns,
 *              as many as hist_len may reach (more than 10900 less K and bias_width take
 *              a slower way, whatever hist_len).  hist_len [N]; prompt_len
 *              [N] or NULL (0).  draft_tokens [N, K] or NULL (K = 0).  A token
 *              outside [0, vocab) is skipped, DSPARK_DEV_TOKEN_OOR.  hist_len outside
 *              [0, tokens_width] and bias_count outside [0, bias_width] are clamped,
 *              DSPARK_DEV_LEN_OOR.
 * repetition, frequency, presence  [N] fp32, each may be NULL (1, 0, 0).
 * bias_token [N, bias_width], bias_value fp32, bias_count [N]; or NULL, bias_width 0.
 *              A token more than once: its values are added up in order first.
 * mask         [mask_rows, mask_stride] 32-bit words or NULL: bit v % 32 of word v /
 *              32 is 1 where token v is allowed.
 * mask_index   [R]: a row's row of mask, negative = none masked; or NULL: the row
 *              itself.  An index >= mask_rows masks nothing, DSPARK_DEV_LEN_OOR.
 * workspace    256 bytes (the status word).
 * Limits: 1 <= N <= 16384, 0 <= K <= 63, 1 <= vocab < 2^30, bias_width <= 1024,
 * tokens_width <= 2^26, 0 < R <= 2^22.
 * ------------------------------------------------------------------------ */
DSPARK_API dspark_status dspark_adjust_logits(
    const void *logits, int64_t stride, int32_t dtype, int32_t R, int32_t vocab,
    const int32_t *cu_rows, int32_t N,
    const int32_t *tokens, int64_t tokens_stride, int32_t tokens_width,
    const int32_t *hist_len, const int32_t *prompt_len,
    const int32_t *draft_tokens, int32_t K, const uint64_t *tree, int32_t tree_width,
    const float *repetition, const float *frequency, const float *presence,
    const int32_t *bias_token, const float *bias_value, const int32_t *bias_count,
    int32_t bias_width, const uint32_t *mask, int64_t mask_stride, int32_t mask_rows,
    const int32_t *mask_index, void *out, int64_t out_stride,
    void *workspace, size_t workspace_bytes, dspark_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DSPARK_TARGET_H_ */
