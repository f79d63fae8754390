// C entry points of include/dspark_target.h: host-side validation, then the
// launches.  Nothing here allocates device memory or synchronises.
#include <cmath>
#include <cstdint>
#include <utility>

#include "target_internal.h"

namespace dspark {
namespace {

bool aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// a required array, or one that may be NULL, of elements of `size` bytes
bool given(const void *p, uintptr_t size) { return p != nullptr && aligned(p, size); }
bool optional(const void *p, uintptr_t size) { return aligned(p, size); }

dspark_status check_pages(int32_t page_size, int32_t num_pages) {
  if (page_size <= 0 || num_pages <= 0) return DSPARK_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0)
    return DSPARK_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_pages) * page_size >= (1ll << 31)) return DSPARK_ERR_UNSUPPORTED;
  return DSPARK_OK;
}

int32_t log2_of(int32_t page_size) {
  int32_t s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

dspark_status check_tree(const uint64_t *tree, int32_t tree_width) {
  if (tree == nullptr) return DSPARK_OK;
  if (!aligned(tree, 8) || tree_width <= 0) return DSPARK_ERR_INVALID_ARG;
  return tree_width > kMaxTreeRows ? DSPARK_ERR_UNSUPPORTED : DSPARK_OK;
}

dspark_status check_ws(const void *ws, size_t bytes, size_t need) {
  return ws == nullptr || !aligned(ws, 256) || bytes < need ? DSPARK_ERR_WORKSPACE : DSPARK_OK;
}

// Whether d contiguous elements at every index of three dimensions share none.
bool distinct(int64_t d, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2 = 1,
              int64_t s2 = 0) {
  int64_t n[3] = {n0, n1, n2}, s[3] = {s0, s1, s2};
  double extent = static_cast<double>(d);  // 64 bits do not hold every product
  for (int k = 0; k < 3; ++k) {
    int low = k;
    for (int j = k + 1; j < 3; ++j)
      if (s[j] < s[low]) low = j;
    std::swap(n[k], n[low]);
    std::swap(s[k], s[low]);
    if (n[k] <= 1) continue;
    if (static_cast<double>(s[k]) < extent) return false;
    extent += static_cast<double>(n[k] - 1) * static_cast<double>(s[k]);
  }
  return true;
}

// The pointer and strides of a [rows, heads, d] tensor.
bool heads_ok(const void *p, int64_t stride, int64_t head_stride, int32_t heads, int32_t d,
              uintptr_t align, int64_t multiple) {
  if (heads == 0) return true;
  return given(p, align) && head_stride >= d && stride >= d && stride % multiple == 0 &&
         head_stride % multiple == 0;
}

// The same of one that is written.
bool heads_out_ok(const HeadRows &t, int32_t rows, int32_t heads, int32_t d, uintptr_t align,
                  int64_t multiple) {
  return heads == 0 || (heads_ok(t.p, t.stride, t.head_stride, heads, d, align, multiple) &&
                        distinct(d, rows, t.stride, heads, t.head_stride));
}

// In place: every element where it was.
bool in_place_ok(const HeadRows &in, const HeadRows &out, int32_t rows, int32_t heads) {
  return heads == 0 || in.p != out.p ||
         ((rows == 1 || in.stride == out.stride) &&
          (heads == 1 || in.head_stride == out.head_stride));
}

// The strides of a cache: any order of pages, tokens and heads, one element a place.
bool cache_ok(int64_t page_stride, int64_t token_stride, int64_t head_stride, int32_t num_pages,
              int32_t page_size, int32_t heads, int32_t d, int64_t multiple) {
  return page_stride >= d && token_stride >= d && head_stride >= d &&
         page_stride % multiple == 0 && token_stride % multiple == 0 &&
         head_stride % multiple == 0 &&
         distinct(d, num_pages, page_stride, page_size, token_stride, heads, head_stride);
}

dspark_status check_rotary(const RotaryArgs &a, int32_t dtype) {
  if (dtype != DSPARK_BF16 && dtype != DSPARK_F32) return DSPARK_ERR_INVALID_ARG;
  if (a.R < 0 || a.Hq < 0 || a.Hk < 0 || a.d <= 0 || a.rot < 2 || a.rot > a.d || a.rot % 2 != 0)
    return DSPARK_ERR_INVALID_ARG;
  if (a.R > kMaxStepRows || a.Hq > 1024 || a.Hk > 1024 || a.d > 1024)
    return DSPARK_ERR_UNSUPPORTED;
  if (a.R == 0) return DSPARK_OK;  // an empty tensor has no pointer
  const int e = dtype == DSPARK_F32 ? 4 : 2;
  if (!heads_ok(a.q.p, a.q.stride, a.q.head_stride, a.Hq, a.d, e, 1) ||
      !heads_out_ok(a.q_out, a.R, a.Hq, a.d, e, 1) || !in_place_ok(a.q, a.q_out, a.R, a.Hq) ||
      !heads_ok(a.k.p, a.k.stride, a.k.head_stride, a.Hk, a.d, e, 1))
    return DSPARK_ERR_INVALID_ARG;
  if (!given(a.position, 4) || !given(a.turns, 8) || !optional(a.n_rows, 4) ||
      !std::isfinite(a.amplitude))
    return DSPARK_ERR_INVALID_ARG;
  return DSPARK_OK;
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

dspark_status dspark_step_rows(
    const int32_t *draft_len, const uint8_t *sampling_mask, const int32_t *chunk_len,
    const int32_t *ctx_len, const uint64_t *tree, int32_t tree_width, const int32_t *tokens,
    int64_t tokens_stride, int32_t tokens_width, const int32_t *draft_tokens, int32_t N,
    int32_t K, const int32_t *page_count, const int32_t *free_pages, int32_t free_max,
    const int32_t *free_count, int32_t page_size, int32_t num_pages, int32_t *block_table,
    int64_t table_stride, int32_t max_pages, int32_t *page_count_out, int32_t *free_count_out,
    int32_t *cu_rows, int32_t *cu_out, int32_t max_rows, int32_t *row_request,
    int32_t *position, int32_t *slot, int32_t *row_token, int32_t *out_row, void *workspace,
    size_t workspace_bytes, dspark_stream_t stream) {
  if (N <= 0 || K <= 0 || max_rows <= 0 || max_pages <= 0 || free_max < 0)
    return DSPARK_ERR_INVALID_ARG;
  if (N > kMaxRequests || K > kMaxStepDrafts || max_rows > kMaxStepRows)
    return DSPARK_ERR_UNSUPPORTED;
  dspark_status s = check_pages(page_size, num_pages);
  if (s != DSPARK_OK) return s;
  if (static_cast<int64_t>(max_pages) * page_size >= (1ll << 31)) return DSPARK_ERR_UNSUPPORTED;
  if ((s = check_tree(tree, tree_width)) != DSPARK_OK) return s;
  if (!given(draft_len, 4) || !optional(chunk_len, 4) || !given(ctx_len, 4) ||
      !given(draft_tokens, 4) || !given(page_count, 4) || !given(free_count, 4) ||
      !given(block_table, 4) || !given(page_count_out, 4) || !given(free_count_out, 4) ||
      !given(cu_rows, 4) || !given(cu_out, 4) || !given(row_request, 4) || !given(position, 4) ||
      !given(slot, 4) || !given(out_row, 4) || !optional(row_token, 4) || !optional(tokens, 4))
    return DSPARK_ERR_INVALID_ARG;
  if (free_max > 0 && !given(free_pages, 4)) return DSPARK_ERR_INVALID_ARG;
  if (row_token != nullptr &&
      (tokens == nullptr || tokens_width <= 0 || tokens_stride < tokens_width))
    return DSPARK_ERR_INVALID_ARG;
  if (table_stride < max_pages) return DSPARK_ERR_INVALID_ARG;
  if ((s = check_ws(workspace, workspace_bytes, 256)) != DSPARK_OK) return s;
  RowsArgs a = {};
  a.draft_len = draft_len;
  a.mask = sampling_mask;
  a.chunk_len = chunk_len;
  a.ctx_len = ctx_len;
  a.tree = tree;
  a.tree_width = tree_width;
  a.tokens = tokens;
  a.tokens_stride = tokens_stride;
  a.tokens_width = tokens_width;
  a.draft = draft_tokens;
  a.N = N;
  a.K = K;
  a.page_count = page_count;
  a.free_pages = free_pages;
  a.free_max = free_max;
  a.free_count = free_count;
  a.page_shift = log2_of(page_size);
  a.num_pages = num_pages;
  a.block_table = block_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.page_count_out = page_count_out;
  a.free_count_out = free_count_out;
  a.cu_rows = cu_rows;
  a.cu_out = cu_out;
  a.max_rows = max_rows;
  a.row_request = row_request;
  a.position = position;
  a.slot = slot;
  a.row_token = row_token;
  a.out_row = out_row;
  a.status = static_cast<uint32_t *>(workspace);
  return rows_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

dspark_status dspark_rotary_table(int32_t rot, double base, int32_t scaling, double factor,
                                  double original, double low, double high, uint64_t *turns) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (rot < 2 || rot % 2 != 0 || turns == nullptr) return DSPARK_ERR_INVALID_ARG;
  if (rot > 1024) return DSPARK_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !std::isfinite(base)) return DSPARK_ERR_INVALID_ARG;
  if (scaling < DSPARK_ROPE_PLAIN || scaling > DSPARK_ROPE_BY_TURNS)
    return DSPARK_ERR_INVALID_ARG;
  if (scaling != DSPARK_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor)))
    return DSPARK_ERR_INVALID_ARG;
  const bool ramp = scaling == DSPARK_ROPE_BY_PARTS || scaling == DSPARK_ROPE_BY_TURNS;
  if (ramp && (!(original > 0.0) || !std::isfinite(original) || !(low > 0.0) || !(high > low) ||
               !std::isfinite(high)))
    return DSPARK_ERR_INVALID_ARG;
  double first = 0.0, last = 0.0;
  if (scaling == DSPARK_ROPE_BY_PARTS) {
    auto edge = [&](double b) {
      return rot * std::log(original / (b * kTwoPi)) / (2.0 * std::log(base));
    };
    first = std::fmax(std::floor(edge(high)), 0.0);
    // the end may lie behind the last pair, which is then within the ramp
    last = std::fmin(std::ceil(edge(low)), rot - 1.0);
  }
  for (int32_t i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == DSPARK_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == DSPARK_ROPE_BY_PARTS) {
      // the ramp is a step where it has no width
      const double w = std::fmin(1.0, std::fmax(0.0, (i - first) / std::fmax(last - first, 1e-3)));
      f = f * (1.0 - w) + f / factor * w;
    } else if (scaling == DSPARK_ROPE_BY_TURNS) {
      const double s =
          std::fmin(1.0, std::fmax(0.0, (original * f / kTwoPi - low) / (high - low)));
      f = f * s + f / factor * (1.0 - s);
    }
    const double t = f / kTwoPi;
    if (!std::isfinite(t)) return DSPARK_ERR_INVALID_ARG;  // a factor too small for f / factor
    turns[i] = static_cast<uint64_t>(std::ldexp(t - std::floor(t), 64));
  }
  return DSPARK_OK;
}

dspark_status dspark_rotary(const void *q, int64_t q_stride, int64_t q_head_stride, int32_t Hq,
                            const void *k, int64_t k_stride, int64_t k_head_stride, int32_t Hk,
                            int32_t dtype, int32_t R, int32_t d, const int32_t *position,
                            const int32_t *n_rows, const uint64_t *turns, int32_t rot,
                            int32_t interleaved, int32_t inverse, float amplitude, void *q_out,
                            int64_t q_out_stride, int64_t q_out_head_stride, void *k_out,
                            int64_t k_out_stride, int64_t k_out_head_stride,
                            dspark_stream_t stream) {
  RotaryArgs a = {};
  a.q = {const_cast<void *>(q), q_stride, q_head_stride};
  a.k = {const_cast<void *>(k), k_stride, k_head_stride};
  a.q_out = {q_out, q_out_stride, q_out_head_stride};
  a.k_out = {k_out, k_out_stride, k_out_head_stride};
  a.Hq = Hq;
  a.Hk = Hk;
  a.f32 = dtype == DSPARK_F32;
  a.R = R;
  a.d = d;
  a.position = position;
  a.n_rows = n_rows;
  a.turns = turns;
  a.rot = rot;
  a.interleaved = interleaved != 0;
  a.inverse = inverse != 0;
  a.amplitude = amplitude;
  const dspark_status s = check_rotary(a, dtype);
  if (s != DSPARK_OK || R == 0) return s;
  if (!heads_out_ok(a.k_out, R, Hk, d, a.f32 ? 4 : 2, 1) || !in_place_ok(a.k, a.k_out, R, Hk))
    return DSPARK_ERR_INVALID_ARG;
  return rotary_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

dspark_status dspark_rotary_append(
    const void *q, int64_t q_stride, int64_t q_head_stride, int32_t Hq, const void *k,
    int64_t k_stride, int64_t k_head_stride, const void *v, int64_t v_stride,
    int64_t v_head_stride, int32_t Hk, int32_t dtype, int32_t R, int32_t d,
    const int32_t *position, const int32_t *slot, const int32_t *n_rows, const uint64_t *turns,
    int32_t rot, int32_t interleaved, float amplitude, void *q_out, int64_t q_out_stride,
    int64_t q_out_head_stride, void *k_cache, void *v_cache, int64_t page_stride,
    int64_t token_stride, int64_t head_stride, int32_t page_size, int32_t num_pages,
    dspark_stream_t stream) {
  RotaryArgs a = {};
  a.q = {const_cast<void *>(q), q_stride, q_head_stride};
  a.k = {const_cast<void *>(k), k_stride, k_head_stride};
  a.v = {const_cast<void *>(v), v_stride, v_head_stride};
  a.q_out = {q_out, q_out_stride, q_out_head_stride};
  a.Hq = Hq;
  a.Hk = Hk;
  a.f32 = dtype == DSPARK_F32;
  a.R = R;
  a.d = d;
  a.position = position;
  a.slot = slot;
  a.n_rows = n_rows;
  a.turns = turns;
  a.rot = rot;
  a.interleaved = interleaved != 0;
  a.amplitude = amplitude;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.page_stride = page_stride;
  a.token_stride = token_stride;
  a.head_stride = head_stride;
  a.num_pages = num_pages;
  dspark_status s = check_rotary(a, dtype);
  if (s != DSPARK_OK || R == 0) return s;
  if ((s = check_pages(page_size, num_pages)) != DSPARK_OK) return s;
  const int e = a.f32 ? 4 : 2;
  if (Hk == 0 || !heads_ok(v, v_stride, v_head_stride, Hk, d, e, 1) || !given(slot, 4) ||
      !given(k_cache, e) || !given(v_cache, e) ||
      !cache_ok(page_stride, token_stride, head_stride, num_pages, page_size, Hk, d, 1))
    return DSPARK_ERR_INVALID_ARG;
  a.page_shift = log2_of(page_size);
  return rotary_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

static dspark_status check_attention_dims(int32_t N, int32_t max_len, int32_t Hq, int32_t Hk,
                                          int32_t d) {
  if (N <= 0 || max_len <= 0 || Hq <= 0 || Hk <= 0 || d <= 0 || Hq % Hk != 0)
    return DSPARK_ERR_INVALID_ARG;
  if (N > kMaxRequests || max_len > kMaxStepRows || Hq > 1024 || Hq / Hk > 128)
    return DSPARK_ERR_UNSUPPORTED;
  if (d % 8 != 0 || d > kMaxAttentionHead) return DSPARK_ERR_UNSUPPORTED;
  return DSPARK_OK;
}

size_t dspark_attention_workspace_size(int32_t N, int32_t max_len, int32_t Hq, int32_t Hk,
                                       int32_t d) {
  if (check_attention_dims(N, max_len, Hq, Hk, d) != DSPARK_OK) return 0;
  return attention_workspace_bytes(max_len, Hq, Hk, d);
}

dspark_status dspark_tree_attention(
    const void *q, int64_t q_stride, int64_t q_head_stride, const void *k_cache,
    const void *v_cache, int64_t page_stride, int64_t token_stride, int64_t head_stride,
    int32_t page_size, int32_t num_pages, const int32_t *block_table, int64_t table_stride,
    int32_t max_pages, const int32_t *ctx_len, const int32_t *cu_rows, const uint64_t *tree,
    int32_t tree_width, int32_t N, int32_t R, int32_t max_len, int32_t Hq, int32_t Hk,
    int32_t d, float scale, void *out, int64_t out_stride, int64_t out_head_stride, float *lse,
    void *workspace, size_t workspace_bytes, dspark_stream_t stream) {
  dspark_status s = check_attention_dims(N, max_len, Hq, Hk, d);
  if (s != DSPARK_OK) return s;
  if (R <= 0 || max_pages <= 0) return DSPARK_ERR_INVALID_ARG;
  if (R > kMaxStepRows) return DSPARK_ERR_UNSUPPORTED;
  if ((s = check_pages(page_size, num_pages)) != DSPARK_OK) return s;
  if (static_cast<int64_t>(max_pages) * page_size >= (1ll << 30)) return DSPARK_ERR_UNSUPPORTED;
  if ((s = check_tree(tree, tree_width)) != DSPARK_OK) return s;
  if (!heads_ok(q, q_stride, q_head_stride, Hq, d, 16, 8) ||
      !heads_out_ok({out, out_stride, out_head_stride}, R, Hq, d, 16, 8) ||
      !given(k_cache, 16) || !given(v_cache, 16) ||
      !cache_ok(page_stride, token_stride, head_stride, num_pages, page_size, Hk, d, 8))
    return DSPARK_ERR_INVALID_ARG;
  // strides of a tensor map
  if (page_stride >= (1ll << 38) || token_stride >= (1ll << 38) || head_stride >= (1ll << 38))
    return DSPARK_ERR_UNSUPPORTED;
  if (!given(block_table, 4) || table_stride < max_pages || !given(ctx_len, 4) ||
      !given(cu_rows, 4) || !optional(lse, 4) || !(scale > 0.0f) ||
      !std::isnormal(scale) || !std::isfinite(scale * 2.0f))
    return DSPARK_ERR_INVALID_ARG;
  if ((s = check_ws(workspace, workspace_bytes, attention_workspace_bytes(max_len, Hq, Hk, d))) !=
      DSPARK_OK)
    return s;
  AttentionArgs a = {};
  a.q = {const_cast<void *>(q), q_stride, q_head_stride};
  a.out = {out, out_stride, out_head_stride};
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.page_stride = page_stride;
  a.token_stride = token_stride;
  a.head_stride = head_stride;
  a.page_shift = log2_of(page_size);
  a.num_pages = num_pages;
  a.block_table = block_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.ctx_len = ctx_len;
  a.cu_rows = cu_rows;
  a.tree = tree;
  a.tree_width = tree_width;
  a.N = N;
  a.R = R;
  a.max_len = max_len;
  a.Hq = Hq;
  a.Hk = Hk;
  a.d = d;
  a.scale = scale;
  a.lse = lse;
  a.workspace = static_cast<uint8_t *>(workspace);
  return attention_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

dspark_status dspark_adjust_logits(
    const void *logits, int64_t stride, int32_t dtype, int32_t R, int32_t vocab,
    const int32_t *cu_rows, int32_t N, const int32_t *tokens, int64_t tokens_stride,
    int32_t tokens_width, const int32_t *hist_len, const int32_t *prompt_len,
    const int32_t *draft_tokens, int32_t K, const uint64_t *tree, int32_t tree_width,
    const float *repetition, const float *frequency, const float *presence,
    const int32_t *bias_token, const float *bias_value, const int32_t *bias_count,
    int32_t bias_width, const uint32_t *mask, int64_t mask_stride, int32_t mask_rows,
    const int32_t *mask_index, void *out, int64_t out_stride, void *workspace,
    size_t workspace_bytes, dspark_stream_t stream) {
  if (dtype != DSPARK_BF16 && dtype != DSPARK_F32) return DSPARK_ERR_INVALID_ARG;
  if (R <= 0 || vocab <= 0 || N <= 0 || K < 0 || tokens_width <= 0 || bias_width < 0)
    return DSPARK_ERR_INVALID_ARG;
  if (R > kMaxStepRows || vocab >= (1 << 30) || N > kMaxRequests || K > kMaxStepDrafts ||
      bias_width > kMaxBias || tokens_width > kMaxHistory)
    return DSPARK_ERR_UNSUPPORTED;
  dspark_status s = check_tree(tree, tree_width);
  if (s != DSPARK_OK) return s;
  const int e = dtype == DSPARK_F32 ? 4 : 2;
  if (!given(logits, e) || !given(out, e) || (R > 1 && (stride < vocab || out_stride < vocab)))
    return DSPARK_ERR_INVALID_ARG;
  // in place: row on row
  if (out == logits && out_stride != stride) return DSPARK_ERR_INVALID_ARG;
  if (!given(cu_rows, 4) || !given(tokens, 4) || tokens_stride < tokens_width ||
      !given(hist_len, 4) || !optional(prompt_len, 4) || !optional(repetition, 4) ||
      !optional(frequency, 4) || !optional(presence, 4) || !optional(mask_index, 4))
    return DSPARK_ERR_INVALID_ARG;
  if (K > 0 && !given(draft_tokens, 4)) return DSPARK_ERR_INVALID_ARG;
  if (bias_width > 0 && (!given(bias_token, 4) || !given(bias_value, 4) || !given(bias_count, 4)))
    return DSPARK_ERR_INVALID_ARG;
  if (mask != nullptr && (!aligned(mask, 4) || mask_rows <= 0 || mask_stride < (vocab + 31) / 32))
    return DSPARK_ERR_INVALID_ARG;
  if ((s = check_ws(workspace, workspace_bytes, 256)) != DSPARK_OK) return s;
  AdjustArgs a = {};
  a.logits = logits;
  a.stride = stride;
  a.f32 = dtype == DSPARK_F32;
  a.R = R;
  a.vocab = vocab;
  a.cu_rows = cu_rows;
  a.N = N;
  a.tokens = tokens;
  a.tokens_stride = tokens_stride;
  a.tokens_width = tokens_width;
  a.hist_len = hist_len;
  a.prompt_len = prompt_len;
  a.draft = draft_tokens;
  a.K = K;
  a.tree = tree;
  a.tree_width = tree_width;
  a.repetition = repetition;
  a.frequency = frequency;
  a.presence = presence;
  a.bias_token = bias_token;
  a.bias_value = bias_value;
  a.bias_count = bias_count;
  a.bias_width = bias_width;
  a.mask = mask;
  a.mask_stride = mask_stride;
  a.mask_rows = mask_rows;
  a.mask_index = mask_index;
  a.out = out;
  a.out_stride = out_stride;
  a.status = static_cast<uint32_t *>(workspace);
  return adjust_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
