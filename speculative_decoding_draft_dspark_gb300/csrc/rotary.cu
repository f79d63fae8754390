// Rotary positions, and their keys and values into the paged cache.
//
// A pair's angle is position * f_i.  f_i comes as a fraction of a turn in units of
// 2^-64, so that the product's low 64 bits are the angle's fraction of a turn, exact
// at any position; its upper 32 bits, signed, go to sincospi.  A CTA takes one row:
// its rot / 2 sines and cosines are computed once, into shared memory, and serve all
// its heads.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.cuh"
#include "target_internal.h"

namespace dspark {

constexpr int RT_THREADS = 256;

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T x[V];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float v, float &x) { x = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16 &x) { x = __float2bfloat16_rn(v); }

// One unit of a head: V pairs (halves), or V columns of whole pairs (interleaved; a
// single pair for V = 1), or V columns that are copied.
template <typename T, int V, bool INTER>
__device__ __forceinline__ void rotate_unit(const T *src, T *dst, int u, int rot,
                                            const float2 *turn) {
  using P = Pack<T, V>;
  const int half = rot >> 1;
  if constexpr (!INTER) {
    const int units = half / V;
    if (u < units) {
      const P a = *reinterpret_cast<const P *>(src + u * V);
      const P b = *reinterpret_cast<const P *>(src + half + u * V);
      P ya, yb;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 cs = turn[u * V + e];
        const float fa = to_f32(a.x[e]), fb = to_f32(b.x[e]);
        from_f32(fa * cs.x - fb * cs.y, ya.x[e]);
        from_f32(fb * cs.x + fa * cs.y, yb.x[e]);
      }
      *reinterpret_cast<P *>(dst + u * V) = ya;
      *reinterpret_cast<P *>(dst + half + u * V) = yb;
      return;
    }
    const int c = rot + (u - units) * V;
    *reinterpret_cast<P *>(dst + c) = *reinterpret_cast<const P *>(src + c);
  } else if constexpr (V == 1) {
    if (u < half) {
      const float2 cs = turn[u];
      const float fa = to_f32(src[2 * u]), fb = to_f32(src[2 * u + 1]);
      from_f32(fa * cs.x - fb * cs.y, dst[2 * u]);
      from_f32(fb * cs.x + fa * cs.y, dst[2 * u + 1]);
      return;
    }
    dst[rot + u - half] = src[rot + u - half];
  } else {
    const P a = *reinterpret_cast<const P *>(src + u * V);
    P y = a;
    if (u * V < rot) {
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float2 cs = turn[(u * V + e) >> 1];
        const float fa = to_f32(a.x[e]), fb = to_f32(a.x[e + 1]);
        from_f32(fa * cs.x - fb * cs.y, y.x[e]);
        from_f32(fb * cs.x + fa * cs.y, y.x[e + 1]);
      }
    }
    *reinterpret_cast<P *>(dst + u * V) = y;
  }
}

template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(RT_THREADS) rotary_kernel(const RotaryArgs p) {
  __shared__ float2 turn[512];
  wait_for_earlier_kernel();
  const int r = blockIdx.x;
  if (p.n_rows != nullptr && r >= *p.n_rows) return;
  const int half = p.rot >> 1;
  const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(p.position[r]));
  for (int i = threadIdx.x; i < half; i += RT_THREADS) {
    const int32_t t = static_cast<int32_t>((pos * p.turns[i]) >> 32);
    float s, c;
    sincospif(static_cast<float>(t) * 0x1p-31f, &s, &c);
    turn[i] = make_float2(c * p.amplitude, (p.inverse ? -s : s) * p.amplitude);
  }
  __syncthreads();
  const int units = INTER ? (V == 1 ? p.d - half : p.d / V) : (p.d - half) / V;
  const T *q = static_cast<const T *>(p.q.p) + r * p.q.stride;
  T *qo = static_cast<T *>(p.q_out.p) + r * p.q_out.stride;
  for (int i = threadIdx.x; i < p.Hq * units; i += RT_THREADS) {
    const int h = i / units, u = i - h * units;
    rotate_unit<T, V, INTER>(q + h * p.q.head_stride, qo + h * p.q_out.head_stride, u, p.rot,
                             turn);
  }
  if (p.Hk == 0) return;
  const T *k = static_cast<const T *>(p.k.p) + r * p.k.stride;
  T *ko = static_cast<T *>(p.k_out.p) + r * p.k_out.stride;
  int64_t ko_head = p.k_out.head_stride;
  if (p.slot != nullptr) {
    const int slot = p.slot[r];
    if (slot < 0 || (slot >> p.page_shift) >= p.num_pages) return;
    const int64_t at = (slot >> p.page_shift) * p.page_stride +
                       (slot & ((1 << p.page_shift) - 1)) * p.token_stride;
    ko = static_cast<T *>(p.k_cache) + at;
    ko_head = p.head_stride;
    const T *v = static_cast<const T *>(p.v.p) + r * p.v.stride;
    T *vo = static_cast<T *>(p.v_cache) + at;
    using P = Pack<T, V>;
    const int columns = p.d / V;
    for (int i = threadIdx.x; i < p.Hk * columns; i += RT_THREADS) {
      const int h = i / columns, c = (i - h * columns) * V;
      *reinterpret_cast<P *>(vo + h * ko_head + c) =
          *reinterpret_cast<const P *>(v + h * p.v.head_stride + c);
    }
  }
  for (int i = threadIdx.x; i < p.Hk * units; i += RT_THREADS) {
    const int h = i / units, u = i - h * units;
    rotate_unit<T, V, INTER>(k + h * p.k.head_stride, ko + h * ko_head, u, p.rot, turn);
  }
}

template <typename T, int V, bool INTER>
static dspark_status launch(const RotaryArgs &a, cudaStream_t stream) {
  return launch_overlapped(rotary_kernel<T, V, INTER>, dim3(a.R), dim3(RT_THREADS), 0, stream,
                           a) == cudaSuccess
             ? DSPARK_OK
             : DSPARK_ERR_CUDA;
}

// Whether a tensor's vectors of `v` elements are 16-byte aligned.
static bool wide(const HeadRows &t, int heads, int v) {
  return heads == 0 || ((reinterpret_cast<uintptr_t>(t.p) & 15) == 0 && t.stride % v == 0 &&
                        t.head_stride % v == 0);
}

template <typename T>
static dspark_status launch_type(const RotaryArgs &a, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  bool vectors = a.d % V == 0 && (a.interleaved ? a.rot : a.rot / 2) % V == 0 &&
                 wide(a.q, a.Hq, V) && wide(a.q_out, a.Hq, V) && wide(a.k, a.Hk, V);
  if (a.slot != nullptr)
    vectors = vectors && wide(a.v, a.Hk, V) && wide({a.k_cache, a.token_stride, a.head_stride}, 1, V) &&
              wide({a.v_cache, a.page_stride, a.head_stride}, 1, V);
  else
    vectors = vectors && wide(a.k_out, a.Hk, V);
  if (vectors)
    return a.interleaved ? launch<T, V, true>(a, stream) : launch<T, V, false>(a, stream);
  return a.interleaved ? launch<T, 1, true>(a, stream) : launch<T, 1, false>(a, stream);
}

dspark_status rotary_launch(const RotaryArgs &a, cudaStream_t stream) {
  if (a.Hq + a.Hk == 0) return DSPARK_OK;
  return a.f32 ? launch_type<float>(a, stream) : launch_type<__nv_bfloat16>(a, stream);
}

}  // namespace dspark
