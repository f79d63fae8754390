// Rotary positions, and their keys and values into the paged cache.
//
// A pair's angle is position * f_i.  f_i comes as a fraction of a turn in units of
// 2^-64, so that the product's low 64 bits are the angle's fraction of a turn, exact
// at any position; signed, and rounded to fp32, it goes to sincospi.  A CTA takes a few rows:
// their sines and cosines are computed once, an angle a thread, into shared memory, and
// serve all heads.  The rest is a copy, bound by memory: 8192 rows of 32 + 2 x 8 heads x
// 128 columns in 37 us, 5.4 TB/s, 0.81 of measured HBM (GB300).  A row a CTA, its first
// loads before the sines, took 66 us, without them 47: the sines of one row keep a
// quarter of the threads busy.
#include <algorithm>
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.cuh"
#include "target_internal.h"

namespace dspark {

constexpr int RT_THREADS = 256;
constexpr int RT_ROWS = 8;         // of a CTA, at most
constexpr int RT_ANGLES = 512;     // of its rows: one row's at least
constexpr int RT_CTAS = 4 * 152;   // below which rows are not put together

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T x[V];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float v, float &x) { x = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16 &x) { x = __float2bfloat16_rn(v); }
// neighbours, in one conversion
__device__ __forceinline__ void from_f32(float v, float w, float *x) {
  x[0] = v;
  x[1] = w;
}
__device__ __forceinline__ void from_f32(float v, float w, __nv_bfloat16 *x) {
  *reinterpret_cast<__nv_bfloat162 *>(x) = __floats2bfloat162_rn(v, w);
}

// One unit of a head: V pairs (halves), or V columns of whole pairs (interleaved; a
// single pair for V = 1), or V columns that are copied.
template <typename T, int V, bool INTER>
struct Unit {
  using P = Pack<T, V>;
  P a, b;  // b: the pairs' second halves
  __host__ __device__ __forceinline__ static int pairs(int rot) {  // units with pairs
    return INTER ? (V == 1 ? rot >> 1 : rot / V) : (rot >> 1) / V;
  }
  __host__ __device__ __forceinline__ static int count(int rot, int d) {
    return INTER && V > 1 ? d / V : pairs(rot) + (d - rot) / V;
  }
  __device__ __forceinline__ static int column(int u, int rot) {
    if (INTER && V > 1) return u * V;
    const int n = pairs(rot);
    return u < n ? (INTER ? 2 * u : u * V) : rot + (u - n) * V;
  }
  __device__ __forceinline__ static int second(int rot) { return INTER ? 1 : rot >> 1; }
  __device__ __forceinline__ void load(const T *src, int u, int rot) {
    const int c = column(u, rot);
    a = *reinterpret_cast<const P *>(src + c);
    if ((!INTER || V == 1) && u < pairs(rot))
      b = *reinterpret_cast<const P *>(src + c + second(rot));
  }
  __device__ __forceinline__ void store(T *dst, int u, int rot, const float2 *turn) {
    const int c = column(u, rot);
    if (u < pairs(rot)) {
      if constexpr (V == 1) {
        const float2 cs = turn[u];
        const float fa = to_f32(a.x[0]), fb = to_f32(b.x[0]);
        from_f32(fa * cs.x - fb * cs.y, a.x[0]);
        from_f32(fb * cs.x + fa * cs.y, b.x[0]);
        *reinterpret_cast<P *>(dst + c + second(rot)) = b;
      } else if constexpr (INTER) {
        const float4 *t = reinterpret_cast<const float4 *>(turn + (c >> 1));  // two pairs
#pragma unroll
        for (int e = 0; e < V; e += 4) {
          const float4 cs = t[e >> 2];
          const float a0 = to_f32(a.x[e]), b0 = to_f32(a.x[e + 1]);
          const float a1 = to_f32(a.x[e + 2]), b1 = to_f32(a.x[e + 3]);
          from_f32(a0 * cs.x - b0 * cs.y, b0 * cs.x + a0 * cs.y, a.x + e);
          from_f32(a1 * cs.z - b1 * cs.w, b1 * cs.z + a1 * cs.w, a.x + e + 2);
        }
      } else {
        const float4 *t = reinterpret_cast<const float4 *>(turn + u * V);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float4 cs = t[e >> 1];
          const float a0 = to_f32(a.x[e]), b0 = to_f32(b.x[e]);
          const float a1 = to_f32(a.x[e + 1]), b1 = to_f32(b.x[e + 1]);
          from_f32(a0 * cs.x - b0 * cs.y, a1 * cs.z - b1 * cs.w, a.x + e);
          from_f32(b0 * cs.x + a0 * cs.y, b1 * cs.z + a1 * cs.w, b.x + e);
        }
        *reinterpret_cast<P *>(dst + c + second(rot)) = b;
      }
    }
    *reinterpret_cast<P *>(dst + c) = a;
  }
};

// Division of numbers below 2^29 by one that the host knows.
struct Divisor {
  uint32_t magic, shift;
  int32_t by;
  __host__ explicit Divisor(int32_t d) : magic(0), shift(0), by(d) {
    while ((1ll << shift) < d) ++shift;
    if (d > 1) {
      --shift;
      magic = static_cast<uint32_t>(((1ull << (32 + shift)) + d - 1) / d);
    }
  }
  __device__ __forceinline__ int operator()(int m, int &rest) const {
    const int q =
        by == 1 ? m : static_cast<int>(__umulhi(static_cast<uint32_t>(m), magic) >> shift);
    rest = m - q * by;
    return q;
  }
};
struct RotaryShape {
  int32_t rows;                        // of a CTA
  Divisor half, heads_q, heads_k;      // pairs; a row's units of q, and of k
  Divisor units, heads_v, columns;     // a head's units; a row's columns of v, and a head's
};

template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(RT_THREADS, 6)
    rotary_kernel(const RotaryArgs p, const RotaryShape shape) {
  using U = Unit<T, V, INTER>;
  using P = Pack<T, V>;
  constexpr int UNROLL = 2;
  __shared__ __align__(16) float2 turn[RT_ANGLES];
  __shared__ int64_t place[RT_ROWS];  // of a row in the cache, or -1
  wait_for_earlier_kernel();
  const int tid = threadIdx.x, r0 = blockIdx.x * shape.rows, half = p.rot >> 1;
  int rows = min(shape.rows, p.R - r0);
  if (p.n_rows != nullptr) rows = min(rows, *p.n_rows - r0);
  if (rows <= 0) return;
  for (int i = tid; i < rows * half; i += RT_THREADS) {
    int pair;
    const int r = r0 + shape.half(i, pair);
    const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(p.position[r]));
    // signed, and all 64 bits to the nearest float: a small angle keeps its 24 bits
    const int64_t t = static_cast<int64_t>(pos * p.turns[pair]);
    float s, c;
    sincospif(static_cast<float>(t) * 0x1p-63f, &s, &c);
    turn[i] = make_float2(c * p.amplitude, (p.inverse ? -s : s) * p.amplitude);
  }
  if (p.slot != nullptr && tid < rows) {
    const int slot = p.slot[r0 + tid];
    place[tid] = slot < 0 || (slot >> p.page_shift) >= p.num_pages
                     ? -1
                     : (slot >> p.page_shift) * p.page_stride +
                           (slot & ((1 << p.page_shift) - 1)) * p.token_stride;
  }
  __syncthreads();
  // q, then k: several units of a thread at a time, their loads first
  auto rotate = [&](const HeadRows &from, const HeadRows &to, bool cached, const Divisor &row_units,
                    int heads) {
    const int total = rows * row_units.by;
    for (int i0 = tid; heads > 0 && i0 < total; i0 += UNROLL * RT_THREADS) {
      U x[UNROLL];
      T *dst[UNROLL];
      int u[UNROLL], r[UNROLL];
#pragma unroll
      for (int e = 0; e < UNROLL; ++e) {
        const int i = i0 + e * RT_THREADS;
        dst[e] = nullptr;
        if (i >= total) continue;
        int rest;
        r[e] = row_units(i, rest);
        const int h = shape.units(rest, u[e]);
        x[e].load(static_cast<const T *>(from.p) + (r0 + r[e]) * from.stride +
                      h * from.head_stride,
                  u[e], p.rot);
        if (!cached)
          dst[e] = static_cast<T *>(to.p) + (r0 + r[e]) * to.stride + h * to.head_stride;
        else if (place[r[e]] >= 0)
          dst[e] = static_cast<T *>(to.p) + place[r[e]] + h * to.head_stride;
      }
#pragma unroll
      for (int e = 0; e < UNROLL; ++e)
        if (dst[e] != nullptr) x[e].store(dst[e], u[e], p.rot, turn + r[e] * half);
    }
  };
  rotate(p.q, p.q_out, false, shape.heads_q, p.Hq);
  if (p.slot == nullptr) {
    rotate(p.k, p.k_out, false, shape.heads_k, p.Hk);
    return;
  }
  rotate(p.k, {p.k_cache, 0, p.head_stride}, true, shape.heads_k, p.Hk);
  const int total = rows * shape.heads_v.by;
  for (int i0 = tid; i0 < total; i0 += UNROLL * RT_THREADS) {
    P x[UNROLL];
    T *dst[UNROLL];
#pragma unroll
    for (int e = 0; e < UNROLL; ++e) {
      const int i = i0 + e * RT_THREADS;
      dst[e] = nullptr;
      if (i >= total) continue;
      int rest, c;
      const int r = shape.heads_v(i, rest), h = shape.columns(rest, c);
      if (place[r] < 0) continue;
      x[e] = *reinterpret_cast<const P *>(static_cast<const T *>(p.v.p) + (r0 + r) * p.v.stride +
                                          h * p.v.head_stride + c * V);
      dst[e] = static_cast<T *>(p.v_cache) + place[r] + h * p.head_stride + c * V;
    }
#pragma unroll
    for (int e = 0; e < UNROLL; ++e)
      if (dst[e] != nullptr) *reinterpret_cast<P *>(dst[e]) = x[e];
  }
}

template <typename T, int V, bool INTER>
static dspark_status launch(const RotaryArgs &a, cudaStream_t stream) {
  const int units = Unit<T, V, INTER>::count(a.rot, a.d), half = a.rot / 2;
  // a sine for every thread, where there are rows enough for all SMs
  int rows = std::min(RT_ROWS, std::max(1, RT_THREADS / half));
  while (rows > 1 && a.R < rows * RT_CTAS) --rows;
  const RotaryShape shape = {rows,
                             Divisor(half),
                             Divisor(std::max(1, a.Hq * units)),
                             Divisor(std::max(1, a.Hk * units)),
                             Divisor(units),
                             Divisor(std::max(1, a.Hk * (a.d / V))),
                             Divisor(a.d / V)};
  return launch_overlapped(rotary_kernel<T, V, INTER>, dim3((a.R + rows - 1) / rows),
                           dim3(RT_THREADS), 0, stream, a, shape) == cudaSuccess
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
