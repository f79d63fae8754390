// Attention of a step's rows over the paged cache: a warp for each row and query
// head, the running maximum and sum of a softmax in fp32.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.cuh"
#include "target_internal.h"

namespace dspark {

constexpr int AT_WARPS = 4;

__global__ void __launch_bounds__(AT_WARPS * 32) attention_kernel(const AttentionArgs p) {
  wait_for_earlier_kernel();
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y * AT_WARPS + (threadIdx.x >> 5);
  const int r = blockIdx.x;
  if (h >= p.Hq) return;
  // the request of this row
  int lo = 0, hi = p.N;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_rows[mid] <= r) lo = mid;
    else hi = mid;
  }
  const int n = lo;
  const RowSpan rows = row_span(p.cu_rows, n, p.R);
  const int j = r - rows.first;
  if (j < 0 || j >= rows.count) return;
  if (j >= p.max_len) {
    raise_status(reinterpret_cast<uint32_t *>(p.workspace), DSPARK_DEV_LEN_OOR);
    return;
  }
  const int count = min(rows.count, p.max_len);
  const int ctx = max(p.ctx_len[n], 0);
  const bool tree = is_tree(p.tree, p.tree_width, n, count);
  const uint64_t bits = tree ? tree_bits(p.tree, p.tree_width, n, j, count) : 0ull;
  const int kh = h / (p.Hq / p.Hk);
  const int page = 1 << p.page_shift;
  constexpr int E = kMaxAttentionHead / 32;
  float q[E], acc[E];
  const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(p.q.p) + r * p.q.stride + h * p.q.head_stride;
  for (int e = 0; e < E; ++e) {
    const int c = e * 32 + lane;
    q[e] = c < p.d ? __bfloat162float(qp[c]) : 0.0f;
    acc[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const int64_t end = min(static_cast<int64_t>(ctx) + (tree ? count : j + 1),
                          static_cast<int64_t>(p.max_pages) << p.page_shift);
  for (int64_t t = 0; t < end; ++t) {
    if (tree && t >= ctx && (bits >> (t - ctx) & 1ull) == 0ull) continue;
    const int id = p.block_table[n * p.table_stride + (t >> p.page_shift)];
    if (id < 0 || id >= p.num_pages) {
      raise_status(reinterpret_cast<uint32_t *>(p.workspace), DSPARK_DEV_PAGE_OOR);
      continue;
    }
    const int64_t at = id * p.page_stride + (t & (page - 1)) * p.token_stride + kh * p.head_stride;
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(p.k_cache) + at;
    const __nv_bfloat16 *vp = static_cast<const __nv_bfloat16 *>(p.v_cache) + at;
    float s = 0.0f;
    for (int e = 0; e < E; ++e) {
      const int c = e * 32 + lane;
      if (c < p.d) s += q[e] * __bfloat162float(kp[c]);
    }
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= p.scale;
    if (s == -INFINITY) continue;
    const float top = fmaxf(m, s), w = expf(s - top), keep = m == -INFINITY ? 0.0f : expf(m - top);
    l = l * keep + w;
    for (int e = 0; e < E; ++e) {
      const int c = e * 32 + lane;
      if (c < p.d) acc[e] = acc[e] * keep + w * __bfloat162float(vp[c]);
    }
    m = top;
  }
  if (end < static_cast<int64_t>(ctx) + (tree ? count : j + 1))
    raise_status(reinterpret_cast<uint32_t *>(p.workspace), DSPARK_DEV_PAGE_OOR);
  __nv_bfloat16 *op = static_cast<__nv_bfloat16 *>(p.out.p) + r * p.out.stride + h * p.out.head_stride;
  const bool none = m == -INFINITY;
  for (int e = 0; e < E; ++e) {
    const int c = e * 32 + lane;
    if (c < p.d) op[c] = __float2bfloat16_rn(none ? 0.0f : acc[e] / l);
  }
  if (p.lse != nullptr && lane == 0)
    p.lse[static_cast<int64_t>(r) * p.Hq + h] = none ? -INFINITY : m + logf(l);
}

size_t attention_workspace_bytes(int32_t, int32_t, int32_t, int32_t) { return 256; }

dspark_status attention_launch(const AttentionArgs &a, cudaStream_t stream) {
  const dim3 grid(a.R, (a.Hq + AT_WARPS - 1) / AT_WARPS);
  return launch_overlapped(attention_kernel, grid, dim3(AT_WARPS * 32), 0, stream, a) ==
                 cudaSuccess
             ? DSPARK_OK
             : DSPARK_ERR_CUDA;
}

}  // namespace dspark
