// Penalties, biases and masks on logits.
//
// Few of a row's logits change: the tokens of the request's history and drafts, its
// biases, and what a mask forbids.  A CTA takes one request and a slice of the
// vocabulary that fits into shared memory: it counts the history's tokens there (a
// word an entry, no hashing, whole numbers, so their order does not matter) and lists
// the entries that any row may change, then goes through the request's rows (a share
// of them, where there are few CTAs): the listed entries one by one, and the slice 16
// bytes at a time.  In place, vectors that the mask forbids whole are written unread
// and those that it allows whole are left alone; elsewhere all are copied.
#include <algorithm>
#include <cuda_bf16.h>
#include <type_traits>

#include "common.cuh"
#include "launch.cuh"
#include "target_internal.h"

namespace dspark {

constexpr int AJ_THREADS = 512;
constexpr int AJ_SLICE = 8192;             // vocabulary entries of a CTA
constexpr int AJ_CTAS = 4 * 152;           // aimed at, by giving a CTA fewer rows
constexpr int AJ_ROWS = 64;                // rows that are masked together
constexpr uint32_t kListed = 1u << 31;
constexpr uint32_t kInPrompt = 1u << 30;
constexpr uint32_t kBiased = 1u << 29;
constexpr uint32_t kCount = kBiased - 1;

template <typename T>
__device__ __forceinline__ T minus_infinity();
template <>
__device__ __forceinline__ float minus_infinity<float>() {
  return __uint_as_float(0xFF800000u);
}
template <>
__device__ __forceinline__ __nv_bfloat16 minus_infinity<__nv_bfloat16>() {
  return __ushort_as_bfloat16(0xFF80u);
}
__device__ __forceinline__ float logit_f32(float x) { return x; }
__device__ __forceinline__ float logit_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void logit_set(float v, float *x) { *x = v; }
__device__ __forceinline__ void logit_set(float v, __nv_bfloat16 *x) {
  *x = __float2bfloat16_rn(v);
}

// V bits of a row of mask words from entry i on, and beyond its end none.
template <int V>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t *mask, int i, int words) {
  const int w = i >> 5, shift = i & 31;
  const uint32_t lo = mask[w];
  const uint32_t hi = shift > 32 - V && w + 1 < words ? mask[w + 1] : 0u;
  return __funnelshift_r(lo, hi, shift) & ((1u << V) - 1u);
}

// What the vectors of a row need, once for the CTA.
template <typename T>
struct MaskRow {
  const T *src;
  T *dst;
  const uint32_t *mask;
  int32_t lead, vectors;  // entries up to the first 16-byte boundary; then so many
};

// The entries of a vector whose bits are 0 become -inf.
template <typename T>
__device__ __forceinline__ void forbid(uint4 &w, uint32_t keep) {
  uint32_t *x = &w.x;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // two bits to two half words of ones
      const uint32_t ones = ((keep >> (2 * e) & 3u) * 0x8001u & 0x10001u) * 0xFFFFu;
      x[e] = (x[e] & ones) | (0xFF80FF80u & ~ones);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((keep >> e & 1u) == 0u) x[e] = 0xFF800000u;
  }
}

// What the masks of `count` rows forbid in the slice, and where `copies` the rest.
template <typename T, bool COPIES>
__device__ __forceinline__ void mask_rows(const MaskRow<T> *row, int count, int size, int words) {
  constexpr int V = 16 / sizeof(T), VECTORS = AJ_SLICE / V, UNROLL = 4;
  constexpr uint32_t ALL = (1u << V) - 1u;
  const int total = count * VECTORS;
  for (int x0 = threadIdx.x; x0 < total; x0 += UNROLL * AJ_THREADS) {
    uint4 x[UNROLL];
    T *at[UNROLL];
    uint32_t keep[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int i = x0 + u * AJ_THREADS;
      at[u] = nullptr;
      keep[u] = ALL;
      if (i >= total) continue;
      const MaskRow<T> &r = row[i / VECTORS];
      const int v = i % VECTORS, e = r.lead + v * V;
      if (v >= r.vectors) continue;
      if (r.mask != nullptr) keep[u] = mask_bits<V>(r.mask, e, words);
      if (!COPIES && keep[u] == ALL) continue;
      at[u] = r.dst + e;
      if (keep[u] != 0u) x[u] = *reinterpret_cast<const uint4 *>(r.src + e);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (at[u] == nullptr) continue;
      forbid<T>(x[u], keep[u]);
      *reinterpret_cast<uint4 *>(at[u]) = x[u];
    }
  }
  // the entries that no vector held: a warp a row
  for (int j = threadIdx.x >> 5; j < count; j += AJ_THREADS / 32) {
    const MaskRow<T> r = row[j];
    const int held = r.vectors * V;
    for (int k = threadIdx.x & 31; k < size - held; k += 32) {
      const int i = k < r.lead ? k : k + held;
      if (r.mask != nullptr && (r.mask[i >> 5] >> (i & 31) & 1u) == 0u)
        r.dst[i] = minus_infinity<T>();
      else if (COPIES)
        r.dst[i] = r.src[i];
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(AJ_THREADS, 3) adjust_kernel(const AdjustArgs p) {
  extern __shared__ __align__(16) uint8_t aj_sm[];
  uint32_t *count = reinterpret_cast<uint32_t *>(aj_sm);           // [slice]
  uint16_t *list = reinterpret_cast<uint16_t *>(count + AJ_SLICE);  // [slice]
  // the slice's biases, in order, if there are any: each one's value, the sum of its
  // token's, its entry
  float *bias = reinterpret_cast<float *>(list + AJ_SLICE);
  float *bias_sum = bias + p.bias_width;
  uint16_t *bias_entry = reinterpret_cast<uint16_t *>(bias_sum + p.bias_width);
  __shared__ int listed, drafts_here, masked_rows, warp_biases[AJ_THREADS / 32];
  __shared__ MaskRow<T> mask_row[AJ_ROWS];
  const int tid = threadIdx.x;
  wait_for_earlier_kernel();
  const int n = blockIdx.y;
  const RowSpan rows = row_span(p.cu_rows, n, p.R);
  // this CTA's share of them
  const int share = (rows.count + gridDim.z - 1) / gridDim.z;
  const int j0 = blockIdx.z * share, j1 = min(rows.count, j0 + share);
  if (j0 >= j1) return;
  const int lo = blockIdx.x * AJ_SLICE, size = min(AJ_SLICE, p.vocab - lo);
  const int words = (size + 31) / 32;
  uint32_t flags = 0u;

  for (int i = tid; i < AJ_SLICE / 4; i += AJ_THREADS)
    reinterpret_cast<uint4 *>(count)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) listed = drafts_here = 0;
  __syncthreads();
  int hist = p.hist_len[n];
  if (hist < 0 || hist > p.tokens_width) flags |= DSPARK_DEV_LEN_OOR;
  hist = min(max(hist, 0), p.tokens_width);
  const int prompt = p.prompt_len != nullptr ? p.prompt_len[n] : 0;
  auto in_slice = [&](int t) {
    if (t < 0 || t >= p.vocab) flags |= DSPARK_DEV_TOKEN_OOR;
    return t >= lo && t - lo < size;
  };
  // the first to touch an entry lists it
  auto first_touch = [&](int i) {
    if ((atomicOr(&count[i], kListed) & kListed) == 0u)
      list[atomicAdd(&listed, 1)] = static_cast<uint16_t>(i);
  };
  const int32_t *text = p.tokens + n * p.tokens_stride;
  for (int i0 = tid; i0 < hist; i0 += 4 * AJ_THREADS) {
    int t[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      t[u] = i0 + u * AJ_THREADS < hist ? text[i0 + u * AJ_THREADS] : lo + size;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * AJ_THREADS;
      if (i >= hist || !in_slice(t[u])) continue;
      const int e = t[u] - lo;
      if (i < prompt) atomicOr(&count[e], kInPrompt);
      else atomicAdd(&count[e], 1u);
      first_touch(e);
    }
  }
  const int drafts = min(p.K, rows.count - 1);
  const int32_t *draft = p.draft + static_cast<int64_t>(n) * p.K;
  if (tid < drafts) {
    const int t = draft[tid];
    if (in_slice(t)) {
      first_touch(t - lo);
      drafts_here = 1;
    }
  }
  if (p.bias_width > 0) {
    const int biases = min(max(p.bias_count[n], 0), p.bias_width);
    const int32_t *token = p.bias_token + static_cast<int64_t>(n) * p.bias_width;
    const float *value = p.bias_value + static_cast<int64_t>(n) * p.bias_width;
    int here = 0;  // in the slice, so far
    for (int i0 = 0; i0 < biases; i0 += AJ_THREADS) {
      const int i = i0 + tid;
      const int t = i < biases ? token[i] : lo + size;
      const bool in = i < biases && in_slice(t);
      const uint32_t votes = __ballot_sync(0xFFFFFFFFu, in);
      if ((tid & 31) == 0) warp_biases[tid >> 5] = __popc(votes);
      __syncthreads();
      int at = here;
      for (int w = 0; w < AJ_THREADS / 32; ++w) {
        if (w < tid >> 5) at += warp_biases[w];
        here += warp_biases[w];
      }
      if (in) {
        at += __popc(votes & ((1u << (tid & 31)) - 1u));
        bias[at] = value[i];
        bias_entry[at] = static_cast<uint16_t>(t - lo);
        atomicOr(&count[t - lo], kBiased);
        first_touch(t - lo);
      }
      __syncthreads();
    }
    // a token's first bias adds up all of them, in order
    for (int i = tid; i < here; i += AJ_THREADS) {
      const int e = bias_entry[i];
      int k = 0;
      while (bias_entry[k] != e) ++k;
      if (k < i) continue;
      float sum = bias[i];
      for (k = i + 1; k < here; ++k)
        if (bias_entry[k] == e) sum = __fadd_rn(sum, bias[k]);
      bias_sum[i] = sum;
    }
  }
  __syncthreads();
  const int entries = listed;
  const bool by_row = drafts_here != 0;  // counts that differ from row to row

  const float rep = p.repetition != nullptr ? p.repetition[n] : 1.0f;
  const float freq = p.frequency != nullptr ? p.frequency[n] : 0.0f;
  const float pres = p.presence != nullptr ? p.presence[n] : 0.0f;
  auto source = [&](int j) {
    return static_cast<const T *>(p.logits) + (rows.first + j) * p.stride + lo;
  };
  auto target = [&](int j) {
    return static_cast<T *>(p.out) + (rows.first + j) * p.out_stride + lo;
  };
  auto mask_of = [&](int j) -> const uint32_t * {
    if (p.mask == nullptr) return nullptr;
    const int64_t row = rows.first + j;
    const int64_t m = p.mask_index != nullptr ? p.mask_index[row] : row;
    if (m >= p.mask_rows) flags |= DSPARK_DEV_LEN_OOR;
    return m >= 0 && m < p.mask_rows ? p.mask + m * p.mask_stride + lo / 32 : nullptr;
  };
  auto adjust = [&](int j, int e) {
    const int i = list[e];
    const uint32_t *mask = mask_of(j);
    if (mask != nullptr && (mask[i >> 5] >> (i & 31) & 1u) == 0u) return;
    const uint32_t word = count[i], c = word & kCount;
    float x = logit_f32(source(j)[i]);
    if (c != 0u || (word & kInPrompt) != 0u) x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
    if (c != 0u) {
      x = __fsub_rn(x, __fmul_rn(freq, static_cast<float>(c)));
      x = __fsub_rn(x, pres);
    }
    if ((word & kBiased) != 0u) {
      int k = 0;
      while (bias_entry[k] != i) ++k;
      x = __fadd_rn(x, bias_sum[k]);
    }
    logit_set(x, target(j) + i);
  };
  const bool copies = p.out != p.logits;
  // rows that have something for mask_rows, AJ_ROWS at a time
  auto mask_all = [&](auto copying) {
    constexpr bool COPIES = decltype(copying)::value;
    constexpr int V = 16 / sizeof(T);
    for (int b0 = j0; b0 < j1; b0 += AJ_ROWS) {
      __syncthreads();
      if (tid == 0) masked_rows = 0;
      __syncthreads();
      const int j = b0 + tid;
      if (tid < AJ_ROWS && j < j1) {
        MaskRow<T> r;
        r.src = source(j);
        r.dst = target(j);
        r.mask = mask_of(j);
        const uintptr_t off = reinterpret_cast<uintptr_t>(r.dst) & 15;
        r.lead = min(size, static_cast<int>((16 - off) & 15) / static_cast<int>(sizeof(T)));
        // rows whose two sides are not aligned alike have no vectors
        r.vectors = off == (reinterpret_cast<uintptr_t>(r.src) & 15) ? (size - r.lead) / V : 0;
        if (COPIES || r.mask != nullptr) mask_row[atomicAdd(&masked_rows, 1)] = r;
      }
      __syncthreads();
      mask_rows<T, COPIES>(mask_row, masked_rows, size, words);
    }
  };
  if (copies) {
    mask_all(std::true_type());
    __syncthreads();
  }
  if (!by_row) {
    for (int x = tid; x < entries * (j1 - j0); x += AJ_THREADS) {
      const int j = x / entries;
      adjust(j0 + j, x - j * entries);
    }
  } else {
    const bool tree = is_tree(p.tree, p.tree_width, n, rows.count);
    uint64_t path = 0ull;  // the rows whose drafts are counted
    for (int j = j0; j < j1; ++j) {
      const uint64_t now =
          (tree ? tree_bits(p.tree, p.tree_width, n, j, rows.count) : low_bits(j + 1)) & ~1ull;
      if (tid >= 1 && tid <= drafts && ((now ^ path) >> tid & 1ull) != 0ull) {
        const int t = draft[tid - 1];
        if (t >= lo && t - lo < size)
          atomicAdd(&count[t - lo], (now >> tid & 1ull) != 0ull ? 1u : ~0u);
      }
      path = now;
      __syncthreads();
      for (int e = tid; e < entries; e += AJ_THREADS) adjust(j, e);
      __syncthreads();
    }
  }
  // vectors that are allowed in part are read again, with what was changed above
  if (!copies && p.mask != nullptr) mask_all(std::false_type());
  if (flags != 0u) raise_status(p.status, flags);
}

template <typename T>
static dspark_status launch(const AdjustArgs &a, cudaStream_t stream) {
  const size_t smem = AJ_SLICE * 6 + static_cast<size_t>(a.bias_width) * 10;
  if (cudaFuncSetAttribute(adjust_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           AJ_SLICE * 6 + kMaxBias * 10) != cudaSuccess ||
      cudaFuncSetAttribute(adjust_kernel<T>, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  const int slices = (a.vocab + AJ_SLICE - 1) / AJ_SLICE;
  // rows a request, as far as the host knows
  const int64_t rows = (static_cast<int64_t>(a.R) + a.N - 1) / a.N;
  const int64_t shares =
      std::min(rows, (AJ_CTAS + static_cast<int64_t>(slices) * a.N - 1) /
                         (static_cast<int64_t>(slices) * a.N));
  const dim3 grid(slices, a.N, static_cast<unsigned>(std::max<int64_t>(1, shares)));
  return launch_overlapped(adjust_kernel<T>, grid, dim3(AJ_THREADS), smem, stream, a) ==
                 cudaSuccess
             ? DSPARK_OK
             : DSPARK_ERR_CUDA;
}

dspark_status adjust_launch(const AdjustArgs &a, cudaStream_t stream) {
  return a.f32 ? launch<float>(a, stream) : launch<__nv_bfloat16>(a, stream);
}

}  // namespace dspark
