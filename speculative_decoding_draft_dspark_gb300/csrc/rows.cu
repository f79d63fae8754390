// The rows of a target step: offsets, pages, positions, slots and input tokens from
// lengths that are on the GPU.
//
// Everything follows from two prefix sums over the requests, of their rows and of
// the pages they need.  One cluster does the whole call: every CTA computes both
// sums for itself (a few loads a thread), keeps them in shared memory, and takes a
// share of the rows, each row looking its request up there.  What is read and may be
// written in place (page counts, the free list's length) is read before the
// cluster's barrier and written after it.  The call moves a few hundred kilobytes at
// most: it is bound by the latency of its dependent steps, not by bytes (1024 requests,
// 9440 rows: 10 us on a GB300; a call of 8 requests 6-8 us, less than the host needs
// to make it).
#include <mutex>

#include "common.cuh"
#include "ptx_pair.cuh"
#include "target_internal.h"

namespace dspark {

constexpr int RW_THREADS = 1024;
constexpr int RW_CTAS = 8;           // a cluster, where there are many rows
constexpr int RW_ALONE = 4096;       // rows up to which one CTA does without
constexpr uint32_t kManyRows = 1u << 30;

// Sums that stop at 2^30, so that lengths of any size add up to "too many".
__device__ __forceinline__ uint32_t add_capped(uint32_t a, uint32_t b) {
  return min(a + b, kManyRows);
}

// Exclusive prefix sum over the block of one value a thread; *total: over all.
__device__ __forceinline__ uint32_t scan_block(uint32_t v, uint32_t *warp_sums, uint32_t *total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x = add_capped(x, y);
  }
  __syncthreads();  // the sums of the scan before have been read
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  uint32_t s = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s = add_capped(s, y);
  }
  const uint32_t upto = __shfl_sync(0xFFFFFFFFu, s, max(w - 1, 0));
  *total = __shfl_sync(0xFFFFFFFFu, s, 31);
  const uint32_t left = __shfl_up_sync(0xFFFFFFFFu, x, 1);
  return add_capped(w > 0 ? upto : 0u, lane > 0 ? left : 0u);
}

__global__ void __launch_bounds__(RW_THREADS) rows_kernel(const RowsArgs p) {
  extern __shared__ int32_t rw_sm[];
  __shared__ uint32_t warp_sums[32];
  int32_t *cu = rw_sm;                // [N + 1]
  int32_t *first_page = cu + p.N + 1;  // [N]: pages that earlier requests take
  int32_t *owned = first_page + p.N;   // [N]
  const int tid = threadIdx.x;
  const int rank = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
  const int page = 1 << p.page_shift;

  const int C = (p.N + RW_THREADS - 1) / RW_THREADS;
  const int n0 = min(p.N, tid * C), n1 = min(p.N, n0 + C);
  uint32_t flags = 0u;
  auto samples = [&](int n) { return p.mask == nullptr || p.mask[n] != 0; };
  auto rows_of = [&](int n) -> uint32_t {
    int v;
    if (samples(n)) {
      v = p.draft_len[n];
      if (v < 0 || v > p.K) flags |= DSPARK_DEV_LEN_OOR;
      v = min(max(v, 0), p.K) + 1;
    } else {
      v = p.chunk_len != nullptr ? p.chunk_len[n] : 0;
      if (v < 0) flags |= DSPARK_DEV_LEN_OOR;
      v = max(v, 0);
    }
    return min(static_cast<uint32_t>(v), kManyRows);
  };
  // rows
  uint32_t mine = 0u, total;
  for (int n = n0; n < n1; ++n) mine = add_capped(mine, rows_of(n));
  uint32_t at = scan_block(mine, warp_sums, &total);
  const uint32_t most = static_cast<uint32_t>(p.max_rows);
  if (total > most) flags |= DSPARK_DEV_ROWS_SHORT;
  for (int n = n0; n < n1; ++n) {
    cu[n] = static_cast<int32_t>(min(at, most));
    at = add_capped(at, rows_of(n));
  }
  const int rows = static_cast<int>(min(total, most));
  if (tid == 0) cu[p.N] = rows;
  __syncthreads();
  // pages, and the rows of sampling requests
  uint32_t pages = 0u, outs = 0u;
  auto need_of = [&](int n) -> uint32_t {
    const int said = p.page_count[n], have = min(max(said, 0), p.max_pages);
    if (have != said) flags |= DSPARK_DEV_LEN_OOR;
    owned[n] = have;
    const int count = cu[n + 1] - cu[n];
    if (count == 0) return 0u;
    int ctx = p.ctx_len[n];
    if (ctx < 0) flags |= DSPARK_DEV_LEN_OOR;
    const int64_t end = static_cast<int64_t>(max(ctx, 0)) + count;
    int64_t want = (end + page - 1) >> p.page_shift;
    if (want > p.max_pages) {
      flags |= DSPARK_DEV_PAGES_SHORT;
      want = p.max_pages;
    }
    return static_cast<uint32_t>(max(static_cast<int>(want) - have, 0));
  };
  for (int n = n0; n < n1; ++n) {
    pages = add_capped(pages, need_of(n));
    if (samples(n)) outs += cu[n + 1] - cu[n];
  }
  uint32_t all_pages, all_outs;
  uint32_t page_at = scan_block(pages, warp_sums, &all_pages);
  uint32_t out_at = scan_block(outs, warp_sums, &all_outs);
  const int said_free = *p.free_count, have_free = min(max(said_free, 0), p.free_max);
  if (have_free != said_free) flags |= DSPARK_DEV_LEN_OOR;
  if (all_pages > static_cast<uint32_t>(have_free)) flags |= DSPARK_DEV_PAGES_SHORT;
  for (int n = n0; n < n1; ++n) {
    first_page[n] = static_cast<int32_t>(page_at);
    page_at = add_capped(page_at, need_of(n));
    if (rank == 0) {
      p.cu_rows[n] = cu[n];
      p.cu_out[n] = static_cast<int32_t>(out_at);
    }
    if (samples(n)) out_at += cu[n + 1] - cu[n];
  }
  if (rank == 0 && tid == 0) {
    p.cu_rows[p.N] = rows;
    p.cu_out[p.N] = static_cast<int32_t>(all_outs);
  }
  // the counts may be given back in place: all CTAs have read them
  if (ctas > 1) cluster_sync_all();
  else __syncthreads();
  if (rank == 0) {
    for (int n = tid; n < p.N; n += RW_THREADS) {
      const uint32_t end =
          n + 1 < p.N ? static_cast<uint32_t>(first_page[n + 1]) : all_pages;
      const int need = static_cast<int>(end) - first_page[n];
      p.page_count_out[n] = owned[n] + min(need, max(have_free - first_page[n], 0));
    }
    if (tid == 0)
      *p.free_count_out = max(have_free - static_cast<int>(min(all_pages, kManyRows)), 0);
  }

  for (int r = rank * RW_THREADS + tid; r < rows; r += ctas * RW_THREADS) {
    int lo = 0, hi = p.N;  // cu[lo] <= r < cu[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= r) lo = mid;
      else hi = mid;
    }
    const int n = lo, j = r - cu[n], count = cu[n + 1] - cu[n];
    const int ctx = max(p.ctx_len[n], 0);
    const bool samp = samples(n);
    int depth = j;
    if (is_tree(p.tree, p.tree_width, n, count))
      depth = __popcll(tree_bits(p.tree, p.tree_width, n, j, count) & ~(1ull << j));
    p.row_request[r] = n;
    p.position[r] = static_cast<int>(min(static_cast<int64_t>(ctx) + depth,
                                         static_cast<int64_t>(INT32_MAX)));

    // the page of this row's token: an old one, or one popped off the free list
    const int64_t index = static_cast<int64_t>(ctx) + j;
    int32_t *table = p.block_table + static_cast<int64_t>(n) * p.table_stride;
    auto fresh = [&](int64_t k) {
      const int64_t pick = static_cast<int64_t>(have_free) - 1 - first_page[n] - (k - owned[n]);
      if (pick < 0) return -1;  // the list ran out, which has a bit of its own
      const int id = p.free_pages[pick];
      if (id < 0 || id >= p.num_pages) flags |= DSPARK_DEV_PAGE_OOR;
      return id;
    };
    const int64_t k = index >> p.page_shift;
    int id = -1;
    if (k < p.max_pages) {
      // a request's first row writes the pages that are missing up to its own,
      // a page's first row that page
      if (j == 0)
        for (int64_t m = owned[n]; m < k; ++m) table[m] = fresh(m);
      if (k < owned[n]) {
        id = table[k];
      } else {
        id = fresh(k);
        if (j == 0 || (index & (page - 1)) == 0) table[k] = id;
      }
    } else if (j == 0) {
      for (int64_t m = owned[n]; m < p.max_pages; ++m) table[m] = fresh(m);
    }
    if (id >= p.num_pages || (id < 0 && k < owned[n])) {
      flags |= DSPARK_DEV_PAGE_OOR;
      id = -1;
    }
    p.slot[r] = id < 0 ? -1 : (id << p.page_shift) + static_cast<int>(index & (page - 1));

    if (p.row_token != nullptr) {
      int t = 0;
      if (samp && j > 0) {
        t = p.draft[static_cast<int64_t>(n) * p.K + j - 1];
      } else if (index < p.tokens_width) {
        t = p.tokens[static_cast<int64_t>(n) * p.tokens_stride + index];
      } else {
        flags |= DSPARK_DEV_TOKEN_OOR;
      }
      p.row_token[r] = t;
    }
    if (samp) p.out_row[p.cu_out[n] + j] = r;
  }
  if (flags != 0u) raise_status(p.status, flags);
}

static std::mutex g_rows_mu;
static bool g_rows_attr[128];

dspark_status rows_launch(const RowsArgs &a, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return DSPARK_ERR_CUDA;
  const int most = (3 * kMaxRequests + 1) * 4;
  {
    std::lock_guard<std::mutex> lk(g_rows_mu);
    if (!g_rows_attr[dev]) {
      if (cudaFuncSetAttribute(rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) !=
          cudaSuccess)
        return DSPARK_ERR_CUDA;
      g_rows_attr[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  const int ctas = a.max_rows > RW_ALONE ? RW_CTAS : 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(RW_THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(3 * a.N + 1) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rows_kernel, a) == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // namespace dspark
