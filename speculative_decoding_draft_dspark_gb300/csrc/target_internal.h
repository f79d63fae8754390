// Internal interface between the C-ABI layer (target_api.cu) and the kernels of the
// target's step (rows.cu, rotary.cu, attention.cu, adjust.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/dspark_target.h"
#include "dspark_internal.h"

namespace dspark {

constexpr int kMaxRequests = 16384;
constexpr int kMaxStepRows = 1 << 22;
constexpr int kMaxTreeRows = 64;
constexpr int kMaxStepDrafts = kMaxTreeRows - 1;
constexpr int kMaxBias = 1024;
constexpr int kMaxHistory = 1 << 26;
constexpr int kMaxAttentionHead = 256;

struct RowsArgs {
  const int32_t *draft_len;
  const uint8_t *mask;
  const int32_t *chunk_len, *ctx_len;
  const uint64_t *tree;
  int32_t tree_width;
  const int32_t *tokens;
  int64_t tokens_stride;
  int32_t tokens_width;
  const int32_t *draft;
  int32_t N, K;
  const int32_t *page_count, *free_pages;
  int32_t free_max;
  const int32_t *free_count;
  int32_t page_shift, num_pages;
  int32_t *block_table;
  int64_t table_stride;
  int32_t max_pages;
  int32_t *page_count_out, *free_count_out, *cu_rows, *cu_out;
  int32_t max_rows;
  int32_t *row_request, *position, *slot, *row_token, *out_row;
  uint32_t *status;
};
dspark_status rows_launch(const RowsArgs &a, cudaStream_t stream);

// a [rows, heads, d] tensor (elements)
struct HeadRows {
  void *p;
  int64_t stride, head_stride;
};

struct RotaryArgs {
  HeadRows q, k, v, q_out, k_out;  // v, caches: appending only
  int32_t Hq, Hk, f32, R, d;
  const int32_t *position, *slot, *n_rows;
  const uint64_t *turns;
  int32_t rot, interleaved, inverse;
  float amplitude;
  void *k_cache, *v_cache;
  int64_t page_stride, token_stride, head_stride;
  int32_t page_shift, num_pages;
};
dspark_status rotary_launch(const RotaryArgs &a, cudaStream_t stream);

struct AttentionArgs {
  HeadRows q, out;
  const void *k_cache, *v_cache;
  int64_t page_stride, token_stride, head_stride;
  int32_t page_shift, num_pages;
  const int32_t *block_table;
  int64_t table_stride;
  int32_t max_pages;
  const int32_t *ctx_len, *cu_rows;
  const uint64_t *tree;
  int32_t tree_width, N, R, max_len, Hq, Hk, d;
  float scale;
  float *lse;
  uint8_t *workspace;
};
size_t attention_workspace_bytes(int32_t max_len, int32_t Hq, int32_t Hk, int32_t d);
dspark_status attention_launch(const AttentionArgs &a, cudaStream_t stream);

struct AdjustArgs {
  const void *logits;
  int64_t stride;
  int32_t f32, R, vocab;
  const int32_t *cu_rows;
  int32_t N;
  const int32_t *tokens;
  int64_t tokens_stride;
  int32_t tokens_width;
  const int32_t *hist_len, *prompt_len, *draft;
  int32_t K;
  const uint64_t *tree;
  int32_t tree_width;
  const float *repetition, *frequency, *presence;
  const int32_t *bias_token;
  const float *bias_value;
  const int32_t *bias_count;
  int32_t bias_width;
  const uint32_t *mask;
  int64_t mask_stride;
  int32_t mask_rows;
  const int32_t *mask_index;
  void *out;
  int64_t out_stride;
  uint32_t *status;
};
dspark_status adjust_launch(const AdjustArgs &a, cudaStream_t stream);

#ifdef __CUDACC__
// The rows of one request among a step's: cu_rows with every offset inside [0, R].
struct RowSpan {
  int first, count;
};
__device__ __forceinline__ RowSpan row_span(const int32_t *cu_rows, int n, int R) {
  const int a = min(max(cu_rows[n], 0), R);
  return {a, max(min(cu_rows[n + 1], R) - a, 0)};
}

// Whether a request of `count` rows is a tree.
__device__ __forceinline__ bool is_tree(const uint64_t *tree, int tree_width, int n, int count) {
  return tree != nullptr && count > 0 && count <= tree_width &&
         (tree[static_cast<int64_t>(n) * tree_width] & 1ull) != 0;
}

// The lowest n bits.
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull;
}

// The rows of its request that a row of a tree attends.
__device__ __forceinline__ uint64_t tree_bits(const uint64_t *tree, int tree_width, int n, int j,
                                              int count) {
  return tree[static_cast<int64_t>(n) * tree_width + j] & low_bits(count);
}
#endif

}  // namespace dspark
