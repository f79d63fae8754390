// Penalties, biases and masks on logits.
//
// Few of a row's logits change: the tokens of the request's history and drafts, its
// biases, and what a mask forbids.  A CTA takes one request and a slice of the
// vocabulary that fits into shared memory: it counts the history's tokens there (a
// word an entry, no hashing, whole numbers, so their order does not matter), lists
// the entries that any row may change, and then goes through the request's rows.  In
// place a row costs its listed entries and what its mask forbids, 16 bytes at a time
// where eight (four) neighbours are; the masked logits are never read.  Elsewhere the
// slice is copied first.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.cuh"
#include "target_internal.h"

namespace dspark {

constexpr int AJ_THREADS = 256;
constexpr int AJ_SLICE = 8192;             // vocabulary entries of a CTA
constexpr uint32_t kListed = 1u << 31;     // a draft or a bias: listed whatever its count
constexpr uint32_t kInPrompt = 1u << 30;
constexpr uint32_t kCount = kInPrompt - 1;

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

template <typename T>
__global__ void __launch_bounds__(AJ_THREADS) adjust_kernel(const AdjustArgs p) {
  extern __shared__ __align__(16) uint8_t aj_sm[];
  uint32_t *count = reinterpret_cast<uint32_t *>(aj_sm);           // [slice]
  uint16_t *list = reinterpret_cast<uint16_t *>(count + AJ_SLICE);  // [slice]
  float *bias = reinterpret_cast<float *>(list + AJ_SLICE);         // [slice], if there are any
  __shared__ uint32_t listed;
  const int tid = threadIdx.x, lane = tid & 31;
  wait_for_earlier_kernel();
  const int n = blockIdx.y;
  const RowSpan rows = row_span(p.cu_rows, n, p.R);
  if (rows.count == 0) return;
  const int lo = blockIdx.x * AJ_SLICE, size = min(AJ_SLICE, p.vocab - lo);
  const bool has_bias = p.bias_width > 0;
  uint32_t flags = 0u;

  // count
  for (int i = tid; i < AJ_SLICE; i += AJ_THREADS) {
    count[i] = 0u;
    if (has_bias) bias[i] = 0.0f;
  }
  if (tid == 0) listed = 0u;
  __syncthreads();
  int hist = p.hist_len[n];
  if (hist < 0 || hist > p.tokens_width) flags |= DSPARK_DEV_LEN_OOR;
  hist = min(max(hist, 0), p.tokens_width);
  const int prompt = p.prompt_len != nullptr ? p.prompt_len[n] : 0;
  auto in_slice = [&](int t) {
    if (t < 0 || t >= p.vocab) flags |= DSPARK_DEV_TOKEN_OOR;
    return t >= lo && t - lo < size;
  };
  const int32_t *text = p.tokens + n * p.tokens_stride;
  for (int i = tid; i < hist; i += AJ_THREADS) {
    const int t = text[i];
    if (!in_slice(t)) continue;
    if (i < prompt) atomicOr(&count[t - lo], kInPrompt);
    else atomicAdd(&count[t - lo], 1u);
  }
  const int drafts = min(p.K, rows.count - 1);
  const int32_t *draft = p.draft + static_cast<int64_t>(n) * p.K;
  if (tid < drafts) {
    const int t = draft[tid];
    if (in_slice(t)) atomicOr(&count[t - lo], kListed);
  }
  if (has_bias) {
    const int biases = min(max(p.bias_count[n], 0), p.bias_width);
    const int32_t *token = p.bias_token + static_cast<int64_t>(n) * p.bias_width;
    const float *value = p.bias_value + static_cast<int64_t>(n) * p.bias_width;
    for (int i = tid; i < biases; i += AJ_THREADS) {
      const int t = token[i];
      if (!in_slice(t)) continue;
      // a token's first place adds up all of its values, in order
      bool first = true;
      for (int k = 0; k < i && first; ++k) first = token[k] != t;
      if (!first) continue;
      float sum = value[i];
      for (int k = i + 1; k < biases; ++k)
        if (token[k] == t) sum = __fadd_rn(sum, value[k]);
      bias[t - lo] = sum;
      atomicOr(&count[t - lo], kListed);
    }
  }
  __syncthreads();
  for (int i = tid; i < AJ_SLICE; i += AJ_THREADS) {
    const bool on = count[i] != 0u;
    const uint32_t votes = __ballot_sync(0xFFFFFFFFu, on);
    uint32_t base = 0u;
    if (lane == 0 && votes != 0u) base = atomicAdd(&listed, __popc(votes));
    base = __shfl_sync(0xFFFFFFFFu, base, 0);
    if (on) list[base + __popc(votes & ((1u << lane) - 1u))] = static_cast<uint16_t>(i);
  }
  __syncthreads();
  const int entries = static_cast<int>(listed);

  const float rep = p.repetition != nullptr ? p.repetition[n] : 1.0f;
  const float freq = p.frequency != nullptr ? p.frequency[n] : 0.0f;
  const float pres = p.presence != nullptr ? p.presence[n] : 0.0f;
  const bool tree = is_tree(p.tree, p.tree_width, n, rows.count);
  const bool copies = p.out != p.logits;
  uint64_t path = 0ull;  // the rows whose drafts are counted
  for (int j = 0; j < rows.count; ++j) {
    const int64_t row = rows.first + j;
    const T *src = static_cast<const T *>(p.logits) + row * p.stride + lo;
    T *dst = static_cast<T *>(p.out) + row * p.out_stride + lo;
    const uint32_t *mask = nullptr;
    if (p.mask != nullptr) {
      const int64_t m = p.mask_index != nullptr ? p.mask_index[row] : row;
      if (m >= p.mask_rows) flags |= DSPARK_DEV_LEN_OOR;
      else if (m >= 0) mask = p.mask + m * p.mask_stride + lo / 32;
    }
    const uint64_t now =
        (tree ? tree_bits(p.tree, p.tree_width, n, j, rows.count) : low_bits(j + 1)) & ~1ull;
    if (tid >= 1 && tid <= drafts && ((now ^ path) >> tid & 1ull) != 0ull) {
      const int t = draft[tid - 1] - lo;
      if (t >= 0 && t < size && draft[tid - 1] >= 0)
        atomicAdd(&count[t], (now >> tid & 1ull) != 0ull ? 1u : ~0u);
    }
    path = now;
    // what the mask forbids, and a copy of the rest
    for (int i = tid; i < size; i += AJ_THREADS) {
      const bool forbidden = mask != nullptr && (mask[i >> 5] >> (i & 31) & 1u) == 0u;
      if (forbidden) dst[i] = minus_infinity<T>();
      else if (copies) dst[i] = src[i];
    }
    __syncthreads();
    for (int e = tid; e < entries; e += AJ_THREADS) {
      const int i = list[e];
      if (mask != nullptr && (mask[i >> 5] >> (i & 31) & 1u) == 0u) continue;
      const uint32_t seen = count[i] & ~kListed, c = seen & kCount;
      float x = logit_f32(src[i]);
      if (seen != 0u) x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
      if (c != 0u) {
        x = __fsub_rn(x, __fmul_rn(freq, static_cast<float>(c)));
        x = __fsub_rn(x, pres);
      }
      if (has_bias) x = __fadd_rn(x, bias[i]);
      logit_set(x, dst + i);
    }
    __syncthreads();
  }
  if (flags != 0u) raise_status(p.status, flags);
}

template <typename T>
static dspark_status launch(const AdjustArgs &a, cudaStream_t stream) {
  const size_t smem = AJ_SLICE * (a.bias_width > 0 ? 10 : 6);
  if (cudaFuncSetAttribute(adjust_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           AJ_SLICE * 10) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  const dim3 grid((a.vocab + AJ_SLICE - 1) / AJ_SLICE, a.N);
  return launch_overlapped(adjust_kernel<T>, grid, dim3(AJ_THREADS), smem, stream, a) ==
                 cudaSuccess
             ? DSPARK_OK
             : DSPARK_ERR_CUDA;
}

dspark_status adjust_launch(const AdjustArgs &a, cudaStream_t stream) {
  return a.f32 ? launch<float>(a, stream) : launch<__nv_bfloat16>(a, stream);
}

}  // namespace dspark
