// Penalties, biases and masks on logits, in two kernels.
//
// mask_kernel streams what a mask forbids, 16 bytes at a time: in place, vectors that
// are forbidden whole are written unread and those that are allowed whole are left
// alone; elsewhere all are copied.  Logits pass through L2 as what is not used again, so
// that the masks stay there for the second kernel.
//
// adjust_kernel changes the few entries of a row that can change otherwise: the tokens
// of the request's history and drafts, and its biases.  A CTA counts the tokens of one
// request in shared memory, lists the distinct ones, and then takes a share of the
// request's rows, entry by entry.  The counts are whole numbers, so their order does
// not matter.  They are in a hash table where one holds every token that a request can
// have, which the host knows by the text buffer's width; wider buffers go through the
// vocabulary a slice at a time, a CTA each, with a word for every entry, whatever the
// histories in them.  (A slice costs the whole history again.  262144 entries, 256
// requests x 8 rows, half of them masked, in place, in a graph: with a buffer of 4096
// tokens and histories up to that 207 us, up to 100 tokens 176; with a buffer of 131072
// 289 and 272, and 417 with histories up to 32768.)
//
// Measured on a GB300, that case with a buffer of 4096, call after call: 197-199 us, of
// which masks 143 (0.74 of HBM's cycles: 537 MB written, half of it read), then counts
// and entries 42 (some 600000 single logits, a sector each).  561 rows x 50003 fp32
// elsewhere: 49 us, the copy 37 (0.91 of measured HBM), counts and entries 10.
#include <algorithm>
#include <cuda_bf16.h>
#include <mutex>

#include "common.cuh"
#include "launch.cuh"
#include "target_internal.h"

namespace dspark {

constexpr int MK_THREADS = 256;
constexpr int MK_CHUNK = 32768;            // entries of a CTA
constexpr int AJ_THREADS = 512;
constexpr int AJ_SLICE = 8192;             // vocabulary entries of a CTA without hashing
constexpr int AJ_MOST_SLOTS = 16384;       // of a hash table
constexpr int AJ_CTAS = 2 * 152;           // that run at once: a CTA gets fewer rows up to there
constexpr uint32_t kEmpty = 0xFFFFFFFFu;
constexpr uint32_t kListed = 1u << 31;
constexpr uint32_t kInPrompt = 1u << 30;
constexpr uint32_t kBiased = 1u << 29;
constexpr uint32_t kBiases = 1u << 28;     // more than one
constexpr uint32_t kDraft = 1u << 27;
constexpr uint32_t kCount = kDraft - 1;

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

// ------------------------------------------------------------------- masks
template <typename T>
__global__ void __launch_bounds__(MK_THREADS) mask_kernel(const AdjustArgs p) {
  constexpr int V = 16 / sizeof(T), UNROLL = 4;
  constexpr uint32_t ALL = (1u << V) - 1u;
  constexpr uint32_t NONE = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
  __shared__ uint4 ones[1 << V];  // a vector's bits, each as wide as an entry
  const int tid = threadIdx.x;
  if (tid < 1 << V) {
    uint32_t m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m[k] = V == 8 ? (tid >> (2 * k) & 1u) * 0xFFFFu | (tid >> (2 * k + 1) & 1u) * 0xFFFF0000u
                    : (tid >> k & 1u) * 0xFFFFFFFFu;
    ones[tid] = make_uint4(m[0], m[1], m[2], m[3]);
  }
  wait_for_earlier_kernel();
  allow_next_kernel();
  const int64_t row = blockIdx.x;
  if (row < max(p.cu_rows[0], 0) || row >= p.cu_rows[p.N]) return;
  const bool copies = p.out != p.logits;
  const uint32_t *mask = nullptr;
  if (p.mask != nullptr) {
    const int64_t m = p.mask_index != nullptr ? p.mask_index[row] : row;
    if (m >= p.mask_rows) raise_status(p.status, DSPARK_DEV_LEN_OOR);
    else if (m >= 0) mask = p.mask + m * p.mask_stride;
  }
  if (!copies && mask == nullptr) return;
  __syncthreads();
  const int lo = blockIdx.y * MK_CHUNK, size = min(MK_CHUNK, p.vocab - lo);
  const int words = (size + 31) / 32;
  if (mask != nullptr) mask += lo / 32;
  const T *src = static_cast<const T *>(p.logits) + row * p.stride + lo;
  T *dst = static_cast<T *>(p.out) + row * p.out_stride + lo;
  // entries up to the first 16-byte boundary, vectors, and those left; none of them
  // vectors where the two sides are not aligned alike
  const uintptr_t off = reinterpret_cast<uintptr_t>(dst) & 15;
  const int lead = min(size, static_cast<int>((16 - off) & 15) / static_cast<int>(sizeof(T)));
  const int vectors = off == (reinterpret_cast<uintptr_t>(src) & 15) ? (size - lead) / V : 0;
  const uint8_t *bytes = reinterpret_cast<const uint8_t *>(mask);
  for (int v0 = tid; v0 < vectors; v0 += UNROLL * MK_THREADS) {
    uint4 x[UNROLL];
    uint32_t keep[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int v = v0 + u * MK_THREADS;
      keep[u] = ALL;
      if (mask != nullptr && v < vectors) {
        if (lead == 0) keep[u] = V == 8 ? bytes[v] : bytes[v >> 1] >> (4 * (v & 1)) & ALL;
        else keep[u] = mask_bits<V>(mask, lead + v * V, words);
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int v = v0 + u * MK_THREADS;
      if (v < vectors && keep[u] != 0u && (copies || keep[u] != ALL))
        x[u] = __ldcs(reinterpret_cast<const uint4 *>(src + lead + v * V));
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int v = v0 + u * MK_THREADS;
      if (v >= vectors || (!copies && keep[u] == ALL)) continue;
      const uint4 m = ones[keep[u]];
      x[u].x = (x[u].x & m.x) | (NONE & ~m.x);
      x[u].y = (x[u].y & m.y) | (NONE & ~m.y);
      x[u].z = (x[u].z & m.z) | (NONE & ~m.z);
      x[u].w = (x[u].w & m.w) | (NONE & ~m.w);
      __stcs(reinterpret_cast<uint4 *>(dst + lead + v * V), x[u]);
    }
  }
  const int held = vectors * V;
  for (int k = tid; k < size - held; k += MK_THREADS) {
    const int i = k < lead ? k : k + held;
    if (mask != nullptr && (mask[i >> 5] >> (i & 31) & 1u) == 0u) dst[i] = minus_infinity<T>();
    else if (copies) dst[i] = src[i];
  }
}

// ------------------------------------------------- penalties and biases
// Shared memory of adjust_kernel: a word a slot for its count and flags; the token
// (hashing); a bias's place; the list of slots in use.
struct AdjustShape {
  int slots;   // a power of two when hashing, AJ_SLICE otherwise
  int slices;  // of the vocabulary: 1 when hashing
  __host__ __device__ int bytes(bool hash, bool biases) const {
    return slots * (4 + (hash ? 4 : 0) + 2 + (biases ? 2 : 0));
  }
};

template <typename T, bool HASH>
__global__ void __launch_bounds__(AJ_THREADS, 2)
    adjust_kernel(const AdjustArgs p, const AdjustShape shape) {
  extern __shared__ __align__(16) uint8_t aj_sm[];
  uint32_t *count = reinterpret_cast<uint32_t *>(aj_sm);
  uint32_t *key = count + shape.slots;                                   // hashing
  uint16_t *list = reinterpret_cast<uint16_t *>(HASH ? key + shape.slots : key);
  uint16_t *bias_at = list + shape.slots;                                // with biases
  __shared__ int listed;
  __shared__ int32_t draft[kMaxStepDrafts + 1];  // [i]: the token of the request's row i
  const int tid = threadIdx.x;
  const int n = blockIdx.y;
  for (int i = tid; i < shape.slots / 4; i += AJ_THREADS) {
    reinterpret_cast<uint4 *>(count)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (HASH) reinterpret_cast<uint4 *>(key)[i] = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
  }
  if (tid == 0) listed = 0;
  wait_for_earlier_kernel();
  const RowSpan rows = row_span(p.cu_rows, n, p.R);
  // this CTA's share of them
  const int share = (rows.count + gridDim.z - 1) / gridDim.z;
  const int j0 = blockIdx.z * share, j1 = min(rows.count, j0 + share);
  if (j0 >= j1) return;
  int hist = p.hist_len[n];
  const int prompt = p.prompt_len != nullptr ? p.prompt_len[n] : 0;
  const int said = p.bias_width > 0 ? p.bias_count[n] : 0;
  const int biases = min(max(said, 0), p.bias_width);
  const int32_t *bias_token = p.bias_token + static_cast<int64_t>(n) * p.bias_width;
  const float *bias_value = p.bias_value + static_cast<int64_t>(n) * p.bias_width;
  const int drafts = min(p.K, rows.count - 1);
  const int lo = HASH ? 0 : blockIdx.x * AJ_SLICE;
  const int size = HASH ? p.vocab : min(AJ_SLICE, p.vocab - lo);
  uint32_t flags = 0u;
  if (hist < 0 || hist > p.tokens_width || said != biases) flags |= DSPARK_DEV_LEN_OOR;
  hist = min(max(hist, 0), p.tokens_width);
  __syncthreads();

  // the slot of a token that this CTA has, listed on first touch; -1 otherwise
  auto slot_of = [&](int t) -> int {
    if (t < 0 || t >= p.vocab) flags |= DSPARK_DEV_TOKEN_OOR;
    if (t < lo || t - lo >= size) return -1;
    int s = t - lo;
    if constexpr (HASH) {
      const uint32_t key_t = static_cast<uint32_t>(t);
      s = static_cast<int>((key_t * 2654435769u) >> 16) & (shape.slots - 1);
      while (true) {
        const uint32_t old = atomicCAS(&key[s], kEmpty, key_t);
        if (old == kEmpty || old == key_t) break;
        s = (s + 1) & (shape.slots - 1);
      }
    }
    return s;
  };
  auto touch = [&](int s, uint32_t flag) -> uint32_t {
    const uint32_t old = atomicOr(&count[s], flag | kListed);
    if ((old & kListed) == 0u) list[atomicAdd(&listed, 1)] = static_cast<uint16_t>(s);
    return old;
  };
  const int32_t *text = p.tokens + n * p.tokens_stride;
  constexpr int UNROLL = 4;
  for (int i0 = tid; i0 < hist; i0 += UNROLL * AJ_THREADS) {
    int t[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (i0 + u * AJ_THREADS < hist) t[u] = text[i0 + u * AJ_THREADS];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int i = i0 + u * AJ_THREADS;
      if (i >= hist) continue;
      const int s = slot_of(t[u]);
      if (s < 0) continue;
      touch(s, i < prompt ? kInPrompt : 0u);
      if (i >= prompt) atomicAdd(&count[s], 1u);
    }
  }
  if (tid < drafts) {
    const int t = p.draft[static_cast<int64_t>(n) * p.K + tid];
    draft[tid + 1] = t;
    const int s = slot_of(t);
    if (s >= 0) touch(s, kDraft);
  }
  for (int i = tid; i < biases; i += AJ_THREADS) {
    const int s = slot_of(bias_token[i]);
    if (s < 0) continue;
    if ((touch(s, kBiased) & kBiased) != 0u) touch(s, kBiases);
    bias_at[s] = static_cast<uint16_t>(i);
  }
  __syncthreads();
  const int entries = listed;
  const float rep = p.repetition != nullptr ? p.repetition[n] : 1.0f;
  const float freq = p.frequency != nullptr ? p.frequency[n] : 0.0f;
  const float pres = p.presence != nullptr ? p.presence[n] : 0.0f;
  const bool tree = is_tree(p.tree, p.tree_width, n, rows.count);

  // Entries that are allowed: in place their logits are as they were.  Four at a time, so
  // that their loads (a mask's row, its word, the logit) overlap.
  const int total = entries * (j1 - j0);
  constexpr int ITEMS = 4;
  for (int x0 = tid; x0 < total; x0 += ITEMS * AJ_THREADS) {
    int slot[ITEMS], row_j[ITEMS], token[ITEMS];
    int64_t mask_row[ITEMS];
    float logit[ITEMS];
    bool allowed[ITEMS];
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
      const int x = x0 + u * AJ_THREADS;
      allowed[u] = x < total;
      if (!allowed[u]) continue;
      const int r = x / entries;
      row_j[u] = j0 + r;
      slot[u] = list[x - r * entries];
      token[u] = HASH ? static_cast<int>(key[slot[u]]) : lo + slot[u];
      const int64_t row = rows.first + row_j[u];
      mask_row[u] = p.mask == nullptr ? -1 : p.mask_index != nullptr ? p.mask_index[row] : row;
    }
#pragma unroll
    for (int u = 0; u < ITEMS; ++u)
      if (allowed[u] && mask_row[u] >= 0 && mask_row[u] < p.mask_rows)
        allowed[u] = (p.mask[mask_row[u] * p.mask_stride + (token[u] >> 5)] >> (token[u] & 31) &
                      1u) != 0u;
#pragma unroll
    for (int u = 0; u < ITEMS; ++u)
      if (allowed[u])
        logit[u] = logit_f32(
            static_cast<const T *>(p.logits)[(rows.first + row_j[u]) * p.stride + token[u]]);
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
      if (!allowed[u]) continue;
      const int s = slot[u], t = token[u], j = row_j[u];
      float v = logit[u];
      const uint32_t word = count[s];
      uint32_t c = word & kCount;
      if ((word & kDraft) != 0u) {
        // on row j's path: the rows that it attends, without row 0
        const uint64_t path =
            tree ? tree_bits(p.tree, p.tree_width, n, j, rows.count) : low_bits(j + 1);
        for (int i = 1; i <= drafts; ++i)
          if (draft[i] == t) c += static_cast<uint32_t>(path >> i) & 1u;
      }
      if (c != 0u || (word & kInPrompt) != 0u)
        v = v > 0.0f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
      if (c != 0u) {
        v = __fsub_rn(v, __fmul_rn(freq, static_cast<float>(c)));
        v = __fsub_rn(v, pres);
      }
      if ((word & kBiases) != 0u) {
        // several: their sum, in order
        bool any = false;
        float sum = 0.0f;
        for (int i = 0; i < biases; ++i) {
          if (bias_token[i] != t) continue;
          sum = any ? __fadd_rn(sum, bias_value[i]) : bias_value[i];
          any = true;
        }
        v = __fadd_rn(v, sum);
      } else if ((word & kBiased) != 0u) {
        v = __fadd_rn(v, bias_value[bias_at[s]]);
      }
      logit_set(v, static_cast<T *>(p.out) + (rows.first + j) * p.out_stride + t);
    }
  }
  if (flags != 0u) raise_status(p.status, flags);
}

static std::mutex g_aj_mu;

template <typename T, bool HASH>
static dspark_status launch_adjust(const AdjustArgs &a, const AdjustShape &shape,
                                   cudaStream_t stream) {
  const bool biases = a.bias_width > 0;
  const AdjustShape most = {HASH ? AJ_MOST_SLOTS : AJ_SLICE, 1};
  static bool attr[128];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return DSPARK_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lk(g_aj_mu);
    if (!attr[dev]) {
      if (cudaFuncSetAttribute(adjust_kernel<T, HASH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               most.bytes(HASH, true)) != cudaSuccess ||
          cudaFuncSetAttribute(adjust_kernel<T, HASH>,
                               cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared) != cudaSuccess)
        return DSPARK_ERR_CUDA;
      attr[dev] = true;
    }
  }
  // rows a request, as far as the host knows
  const int64_t rows = (static_cast<int64_t>(a.R) + a.N - 1) / a.N;
  const int64_t each = static_cast<int64_t>(shape.slices) * a.N;
  // one request may have all rows: a CTA's entries are counted in 31 bits
  const int64_t least = (static_cast<int64_t>(a.R) * shape.slots >> 30) + 1;
  const int64_t shares = std::max(least, std::min(rows, AJ_CTAS / each));
  const dim3 grid(shape.slices, a.N, static_cast<unsigned>(shares));
  return launch_overlapped(adjust_kernel<T, HASH>, grid, dim3(AJ_THREADS),
                           shape.bytes(HASH, biases), stream, a, shape) == cudaSuccess
             ? DSPARK_OK
             : DSPARK_ERR_CUDA;
}

template <typename T>
static dspark_status launch(const AdjustArgs &a, cudaStream_t stream) {
  if (a.out != a.logits || a.mask != nullptr) {
    const dim3 grid(a.R, (a.vocab + MK_CHUNK - 1) / MK_CHUNK);
    if (launch_overlapped(mask_kernel<T>, grid, dim3(MK_THREADS), 0, stream, a) != cudaSuccess)
      return DSPARK_ERR_CUDA;
  }
  // every token that a request can have, in two thirds of a table
  const int64_t most = std::min<int64_t>(
      a.vocab, static_cast<int64_t>(a.tokens_width) + a.K + a.bias_width);
  AdjustShape shape = {256, 1};
  while (shape.slots < AJ_MOST_SLOTS && 2ll * shape.slots < 3 * most) shape.slots *= 2;
  if (2ll * shape.slots >= 3 * most) return launch_adjust<T, true>(a, shape, stream);
  shape = {AJ_SLICE, (a.vocab + AJ_SLICE - 1) / AJ_SLICE};
  return launch_adjust<T, false>(a, shape, stream);
}

dspark_status adjust_launch(const AdjustArgs &a, cudaStream_t stream) {
  return a.f32 ? launch<float>(a, stream) : launch<__nv_bfloat16>(a, stream);
}

}  // namespace dspark
