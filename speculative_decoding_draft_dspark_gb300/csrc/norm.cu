// The residual stream's addition, dropout and root-mean-square norm, and their
// gradient.
//
//   r = residual + dropout(x)      rstd = (mean r^2 + eps)^-1/2
//   y = r rstd gain, in the type of x, or as e4m3 numbers with a scale for a
//       row or for 128 columns: scale = max |y| / 448, q = y / scale
//
//   a = dy gain    xh = r rstd     dr' = dr + rstd (a - xh mean(a xh))
//   dresidual = dr'    dx = dropout(dr')    dgain = sum over rows of dy xh
//
// Dropout keeps an element iff its 16-bit lane is below T = round(65536 (1 -
// p)), and scales by 65536 / T.  The lanes of columns 8g .. 8g+7 of a row are
// the four words of Philox4x32-10 (Salmon et al., SC 2011) with counter (g,
// row, 2^31, offset): no mask is stored, the gradient draws the same one.
//
// Every kernel reads its inputs once and writes its outputs once, so HBM
// bounds all of them; a row stays in registers between its sum and its use.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "launch.cuh"
#include "norm_internal.h"

namespace dspark {

namespace {

// ---------------------------------------------------------------- dropout
struct Philox4 {
  uint32_t w[4];
};

__device__ __forceinline__ Philox4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2,
                                                 uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint32_t h0 = __umulhi(0xD2511F53u, c0), l0 = 0xD2511F53u * c0;
    const uint32_t h1 = __umulhi(0xCD9E8D57u, c2), l1 = 0xCD9E8D57u * c2;
    c0 = h1 ^ c1 ^ k0;
    c1 = l1;
    c2 = h0 ^ c3 ^ k1;
    c3 = l0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

__device__ __forceinline__ Philox4 drop_words(const DropArgs &d, int group, int row) {
  return philox4x32_10(static_cast<uint32_t>(group), static_cast<uint32_t>(row), 0x80000000u,
                       d.offset, d.seed_lo, d.seed_hi);
}

// ----------------------------------------------------- eight columns a lane
// A warp holds 256 columns of a row.  Aligned rows (VEC): lane l has columns
// 8l .. 8l+7, one or two 16-byte accesses.  Other rows: lane l has columns l,
// 32 + l, ..., 224 + l, so that every access of the warp is contiguous.
template <bool VEC>
__device__ __forceinline__ int column(int base, int lane, int e) {
  return VEC ? base + lane * 8 + e : base + e * 32 + lane;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint16_t to_bf16(float v) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
  return r;
}

// eight values as they lie in memory
template <bool F32>
struct Raw {
  uint32_t w[F32 ? 8 : 4];
};

template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void *row, int base, int lane, int d, Raw<F32> &r) {
  if (VEC) {
    const int c = base + lane * 8;
    if (c < d) {
      const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(row) +
                                                       static_cast<size_t>(c) * (F32 ? 4 : 2));
#pragma unroll
      for (int j = 0; j < (F32 ? 2 : 1); ++j) {
        const uint4 v = p[j];
        r.w[4 * j] = v.x;
        r.w[4 * j + 1] = v.y;
        r.w[4 * j + 2] = v.z;
        r.w[4 * j + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < (F32 ? 8 : 4); ++j) r.w[j] = 0u;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = base + e * 32 + lane;
      if (F32) {
        r.w[e] = c < d ? static_cast<const uint32_t *>(row)[c] : 0u;
      } else {
        const uint32_t v = c < d ? static_cast<const uint16_t *>(row)[c] : 0u;
        if (e & 1)
          r.w[e / 2] |= v << 16;
        else
          r.w[e / 2] = v;
      }
    }
  }
}

template <bool F32>
__device__ __forceinline__ void unpack8(const Raw<F32> &r, float (&v)[8]) {
  if (F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r.w[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = bf16_lo(r.w[e]);
      v[2 * e + 1] = bf16_hi(r.w[e]);
    }
  }
}

template <bool F32, bool VEC>
__device__ __forceinline__ void store8(void *row, int base, int lane, int d,
                                       const float (&v)[8]) {
  if (VEC) {
    const int c = base + lane * 8;
    if (c >= d) return;
    uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(row) +
                                         static_cast<size_t>(c) * (F32 ? 4 : 2));
    if (F32) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        p[j] = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                          __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
    } else {
      p[0] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                        pack_bf16(v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = base + e * 32 + lane;
      if (c < d) {
        if (F32)
          static_cast<float *>(row)[c] = v[e];
        else
          static_cast<uint16_t *>(row)[c] = to_bf16(v[e]);
      }
    }
  }
}

// v = dropout(v); a select, so that what a dropped element holds (NaN,
// infinity) is gone
template <bool VEC>
__device__ __forceinline__ void drop8(const DropArgs &dr, int base, int lane, int row,
                                      float (&v)[8]) {
  const Philox4 p = drop_words(dr, base / 8 + lane, row);
  if (VEC) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t x = (p.w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
      v[e] = x < dr.keep ? v[e] * dr.scale : 0.0f;
    }
  } else {
    // lane l drew the words of columns 8l .. 8l+7; column 32e + l is lane
    // (l % 8) of group 4e + l / 8
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int src = 4 * e + (lane >> 3);
      const uint32_t a = __shfl_sync(0xFFFFFFFFu, p.w[0], src);
      const uint32_t b = __shfl_sync(0xFFFFFFFFu, p.w[1], src);
      const uint32_t c = __shfl_sync(0xFFFFFFFFu, p.w[2], src);
      const uint32_t f = __shfl_sync(0xFFFFFFFFu, p.w[3], src);
      const uint32_t lo = lane & 2 ? b : a, hi = lane & 2 ? f : c;
      const uint32_t w = lane & 4 ? hi : lo;
      const uint32_t x = (lane & 1 ? w >> 16 : w) & 0xFFFFu;
      v[e] = x < dr.keep ? v[e] * dr.scale : 0.0f;
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmax_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// A row's warps share values through `slots` (warps per row of them); all of
// the CTA's threads call this together.
__device__ __forceinline__ float row_sum(float v, float *slots, int w, int warps, int lane) {
  v = warp_sum(v);
  if (warps == 1) return v;
  if (lane == 0) slots[w] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < warps; ++i) s += slots[i];
  return s;
}
__device__ __forceinline__ float row_max_nan(float v, float *slots, int w, int warps, int lane) {
  v = warp_max_nan(v);
  if (warps == 1) return v;
  if (lane == 0) slots[w] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < warps; ++i) s = fmax_nan(s, slots[i]);
  return s;
}

// eight e4m3 numbers of y / scale
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

constexpr float kE4m3Max = 448.0f;

__device__ __forceinline__ float scale_of(float top) {
  return top == 0.0f ? 1.0f : top / kE4m3Max;
}

// q = y / scale.  The product with the reciprocal is within an ulp of it, and
// e4m3 keeps 4 bits; where the reciprocal would overflow it divides.
__device__ __forceinline__ void over_scale(float (&y)[8], float scale) {
  if (scale > 1e-35f || scale != scale) {
    const float inv = 1.0f / scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= inv;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] /= scale;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8_e4m3(uint8_t *row, int base, int lane, int d,
                                            const float (&q)[8]) {
  if (VEC) {
    const int c = base + lane * 8;
    if (c >= d) return;
    *reinterpret_cast<uint2 *>(row + c) = make_uint2(e4m3x2(q[0], q[1]) | e4m3x2(q[2], q[3]) << 16,
                                                     e4m3x2(q[4], q[5]) | e4m3x2(q[6], q[7]) << 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = base + e * 32 + lane;
      if (c < d) row[c] = static_cast<uint8_t>(e4m3x2(q[e], 0.0f) & 0xFFu);
    }
  }
}

// y -> y / scale with a scale for 128 columns: 16 lanes if a lane's columns are
// neighbours, else the warp's first or last four
template <bool VEC>
__device__ __forceinline__ void by_groups(const NormArgs &a, int64_t row, int base, int lane,
                                          float (&y)[8]) {
  float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) t0 = fmax_nan(t0, fabsf(y[e]));
#pragma unroll
  for (int e = 4; e < 8; ++e) t1 = fmax_nan(t1, fabsf(y[e]));
  if (VEC) {
    t0 = fmax_nan(t0, t1);
#pragma unroll
    for (int o = 8; o; o >>= 1) t0 = fmax_nan(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, o));
    const float s = scale_of(t0);
    if ((lane & 15) == 0 && base + lane * 8 < a.d)
      a.scale[row * a.groups + (base + lane * 8) / 128] = s;
    over_scale(y, s);
  } else {
    const float s0 = scale_of(warp_max_nan(t0)), s1 = scale_of(warp_max_nan(t1));
    if (lane == 0 && base < a.d) a.scale[row * a.groups + base / 128] = s0;
    if (lane == 0 && base + 128 < a.d) a.scale[row * a.groups + base / 128 + 1] = s1;
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = y[e];
    over_scale(q, s0);
    over_scale(y, s1);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = q[e];
  }
}

// ---------------------------------------------------------------- forward
// `warps` warps hold a row, NV x 256 columns each (chunk i of a warp starts at
// column 256 (i warps + w)); a CTA has as many rows as fit.
template <bool F32, bool VEC, int NV>
__global__ void __launch_bounds__(256) norm_kernel(const NormArgs a, int warps) {
  allow_next_kernel();
  wait_for_earlier_kernel();
  __shared__ float slots[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / warps, w = warp - group * warps;
  const int rows_per_cta = (blockDim.x >> 5) / warps;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_cta + group;
  const bool live = row < a.M;
  constexpr int E = F32 ? 4 : 2;
  const uint8_t *x = static_cast<const uint8_t *>(a.x) + row * a.x_stride * E;
  const uint8_t *res = static_cast<const uint8_t *>(a.residual) + row * a.residual_stride * E;

  float r[NV][8];
  float sum = 0.0f;
  if (live) {
    Raw<F32> rx[NV], rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) load8<F32, VEC>(x, (i * warps + w) * 256, lane, a.d, rx[i]);
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < NV; ++i) load8<F32, VEC>(res, (i * warps + w) * 256, lane, a.d, rr[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack8<F32>(rx[i], r[i]);
      if (a.drop.on) drop8<VEC>(a.drop, (i * warps + w) * 256, lane, static_cast<int>(row), r[i]);
      if (a.residual) {
        float t[8];
        unpack8<F32>(rr[i], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] += t[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(r[i][e], r[i][e], sum);
    }
  }
  sum = row_sum(sum, slots[0] + group * warps, w, warps, lane);
  const float rstd = rsqrtf(sum / static_cast<float>(a.d) + a.eps);
  float top = 0.0f;
  if (live) {
    if (a.rstd && w == 0 && lane == 0) a.rstd[row] = rstd;
    uint8_t *ro = static_cast<uint8_t *>(a.r) + row * a.r_stride * E;
    uint8_t *yo = static_cast<uint8_t *>(a.y) + row * a.y_stride * (a.e4m3 ? 1 : E);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int base = (i * warps + w) * 256;
      if (a.r) store8<F32, VEC>(ro, base, lane, a.d, r[i]);
      Raw<F32> g;
      float t[8];
      load8<F32, VEC>(a.gain, base, lane, a.d, g);
      unpack8<F32>(g, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] = r[i][e] * rstd * t[e];
      if (!a.e4m3) {
        store8<F32, VEC>(yo, base, lane, a.d, r[i]);
      } else if (a.group == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmax_nan(top, fabsf(r[i][e]));
      } else {
        by_groups<VEC>(a, row, base, lane, r[i]);
        store8_e4m3<VEC>(yo, base, lane, a.d, r[i]);
      }
    }
  }
  if (a.e4m3 && a.group == 0) {
    const float s = scale_of(row_max_nan(top, slots[1] + group * warps, w, warps, lane));
    if (live) {
      if (w == 0 && lane == 0) a.scale[row] = s;
      uint8_t *yo = static_cast<uint8_t *>(a.y) + row * a.y_stride;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        over_scale(r[i], s);
        store8_e4m3<VEC>(yo, (i * warps + w) * 256, lane, a.d, r[i]);
      }
    }
  }
}

// Rows too wide to hold: a CTA to a row, which is read again (from L2) for
// every use of it.
constexpr int WIDE_WARPS = 16;

template <bool F32, bool VEC>
__device__ __forceinline__ void stream8(const NormArgs &a, const uint8_t *x, const uint8_t *res,
                                        int64_t row, int base, int lane, float (&r)[8]) {
  Raw<F32> rx, rr;
  load8<F32, VEC>(x, base, lane, a.d, rx);
  if (a.residual) load8<F32, VEC>(res, base, lane, a.d, rr);
  unpack8<F32>(rx, r);
  if (a.drop.on) drop8<VEC>(a.drop, base, lane, static_cast<int>(row), r);
  if (a.residual) {
    float t[8];
    unpack8<F32>(rr, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] += t[e];
  }
}

template <bool F32, bool VEC>
__device__ __forceinline__ void times_gain(const NormArgs &a, float rstd, int base, int lane,
                                           float (&r)[8]) {
  Raw<F32> g;
  float t[8];
  load8<F32, VEC>(a.gain, base, lane, a.d, g);
  unpack8<F32>(g, t);
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = r[e] * rstd * t[e];
}

template <bool F32, bool VEC>
__global__ void __launch_bounds__(WIDE_WARPS * 32) norm_wide_kernel(const NormArgs a) {
  allow_next_kernel();
  wait_for_earlier_kernel();
  __shared__ float slots[2][32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  constexpr int E = F32 ? 4 : 2;
  const uint8_t *x = static_cast<const uint8_t *>(a.x) + row * a.x_stride * E;
  const uint8_t *res = static_cast<const uint8_t *>(a.residual) + row * a.residual_stride * E;
  float sum = 0.0f;
  for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256) {
    float r[8];
    stream8<F32, VEC>(a, x, res, row, base, lane, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(r[e], r[e], sum);
  }
  sum = row_sum(sum, slots[0], w, WIDE_WARPS, lane);
  const float rstd = rsqrtf(sum / static_cast<float>(a.d) + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  float s = 1.0f;
  if (a.e4m3 && a.group == 0) {
    float top = 0.0f;
    for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256) {
      float r[8];
      stream8<F32, VEC>(a, x, res, row, base, lane, r);
      times_gain<F32, VEC>(a, rstd, base, lane, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmax_nan(top, fabsf(r[e]));
    }
    s = scale_of(row_max_nan(top, slots[1], w, WIDE_WARPS, lane));
    if (threadIdx.x == 0) a.scale[row] = s;
  }
  uint8_t *ro = static_cast<uint8_t *>(a.r) + row * a.r_stride * E;
  uint8_t *yo = static_cast<uint8_t *>(a.y) + row * a.y_stride * (a.e4m3 ? 1 : E);
  for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256) {
    float r[8];
    stream8<F32, VEC>(a, x, res, row, base, lane, r);
    if (a.r) store8<F32, VEC>(ro, base, lane, a.d, r);
    times_gain<F32, VEC>(a, rstd, base, lane, r);
    if (!a.e4m3) {
      store8<F32, VEC>(yo, base, lane, a.d, r);
      continue;
    }
    if (a.group == 0)
      over_scale(r, s);
    else
      by_groups<VEC>(a, row, base, lane, r);
    store8_e4m3<VEC>(yo, base, lane, a.d, r);
  }
}

// --------------------------------------------------------------- backward
// A row as in the forward kernel, with the next row's loads issued before the
// current row's sum is waited for.  A CTA goes over rows and keeps dgain's sums
// of its columns in registers, joins its row groups in order and writes one
// fp32 line of partial sums.  dgain_kernel adds the lines up in order.
template <bool F32, int NV>
struct GradRow {
  Raw<F32> dy[NV], r[NV], dr[NV];
  float rstd;
};

template <bool F32, bool VEC, int NV>
__device__ __forceinline__ void load_row(const NormGradArgs &a, int64_t row, int warps, int w,
                                         int lane, GradRow<F32, NV> &x) {
  constexpr int E = F32 ? 4 : 2;
  if (row >= a.M) return;
  const uint8_t *py = static_cast<const uint8_t *>(a.dy) + row * a.dy_stride * E;
  const uint8_t *pr = static_cast<const uint8_t *>(a.r) + row * a.r_stride * E;
  const uint8_t *pd = static_cast<const uint8_t *>(a.dr) + row * a.dr_stride * E;
#pragma unroll
  for (int i = 0; i < NV; ++i) load8<F32, VEC>(py, (i * warps + w) * 256, lane, a.d, x.dy[i]);
#pragma unroll
  for (int i = 0; i < NV; ++i) load8<F32, VEC>(pr, (i * warps + w) * 256, lane, a.d, x.r[i]);
  if (a.dr) {
#pragma unroll
    for (int i = 0; i < NV; ++i) load8<F32, VEC>(pd, (i * warps + w) * 256, lane, a.d, x.dr[i]);
  }
  x.rstd = a.rstd[row];
}

template <bool F32, bool VEC, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_grad_kernel(const NormGradArgs a, int warps) {
  allow_next_kernel();
  wait_for_earlier_kernel();
  __shared__ float slots[2][32];
  extern __shared__ float lines[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / warps, w = warp - group * warps;
  const int groups = (blockDim.x >> 5) / warps;
  constexpr int E = F32 ? 4 : 2;
  float dg[NV][8] = {};
  Raw<F32> g[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) load8<F32, VEC>(a.gain, (i * warps + w) * 256, lane, a.d, g[i]);

  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t r0 = static_cast<int64_t>(blockIdx.x) * groups;
  GradRow<F32, NV> cur, next;
  load_row<F32, VEC, NV>(a, r0 + group, warps, w, lane, cur);
  for (int turn = 0; r0 < a.M; r0 += step, turn ^= 1) {
    const int64_t row = r0 + group;
    const bool live = row < a.M;
    load_row<F32, VEC, NV>(a, row + step, warps, w, lane, next);
    float dot = 0.0f;
    const float rstd = cur.rstd;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float y[8], x[8], t[8];
        unpack8<F32>(cur.dy[i], y);
        unpack8<F32>(cur.r[i], x);
        unpack8<F32>(g[i], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = y[e] * (x[e] * rstd);
          dg[i][e] += s;
          dot = fmaf(s, t[e], dot);
        }
      }
    }
    // two sets of slots: a row's sums are read while the next row's are written
    dot = row_sum(dot, slots[turn] + group * warps, w, warps, lane) / static_cast<float>(a.d);
    if (live) {
      uint8_t *px = static_cast<uint8_t *>(a.dx) + row * a.dx_stride * E;
      uint8_t *ps = static_cast<uint8_t *>(a.dresidual) + row * a.dresidual_stride * E;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int base = (i * warps + w) * 256;
        float y[8], x[8], t[8], o[8];
        unpack8<F32>(cur.dy[i], y);
        unpack8<F32>(cur.r[i], x);
        unpack8<F32>(g[i], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = rstd * (y[e] * t[e] - x[e] * rstd * dot);
        if (a.dr) {
          unpack8<F32>(cur.dr[i], t);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += t[e];
        }
        if (a.dresidual) store8<F32, VEC>(ps, base, lane, a.d, o);
        if (a.dx) {
          if (a.drop.on) drop8<VEC>(a.drop, base, lane, static_cast<int>(row), o);
          store8<F32, VEC>(px, base, lane, a.d, o);
        }
      }
    }
    cur = next;
  }
  if (!a.dgain) return;
  // the row groups' sums, joined in order
  float *line = a.partial + static_cast<int64_t>(blockIdx.x) * a.d;
  for (int k = 0; k < groups; ++k) {
    if (group == k) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = column<VEC>((i * warps + w) * 256, lane, e);
          if (c < a.d) {
            if (groups == 1)
              line[c] = dg[i][e];
            else if (k == 0)
              lines[c] = dg[i][e];
            else if (k < groups - 1)
              lines[c] += dg[i][e];
            else
              line[c] = lines[c] + dg[i][e];
          }
        }
    }
    __syncthreads();
  }
}

// Rows too wide to hold: a CTA to a row, read twice; dgain's sums stay in
// shared memory, every column with one thread.
template <bool F32, bool VEC>
__global__ void __launch_bounds__(WIDE_WARPS * 32) norm_grad_wide_kernel(const NormGradArgs a) {
  allow_next_kernel();
  wait_for_earlier_kernel();
  __shared__ float slots[2][32];
  extern __shared__ float line[];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int E = F32 ? 4 : 2;
  if (a.dgain)
    for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<VEC>(base, lane, e);
        if (c < a.d) line[c] = 0.0f;
      }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
    const uint8_t *py = static_cast<const uint8_t *>(a.dy) + row * a.dy_stride * E;
    const uint8_t *pr = static_cast<const uint8_t *>(a.r) + row * a.r_stride * E;
    const uint8_t *pd = static_cast<const uint8_t *>(a.dr) + row * a.dr_stride * E;
    const float rstd = a.rstd[row];
    float dot = 0.0f;
    for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256) {
      Raw<F32> raw;
      float y[8], x[8], t[8];
      load8<F32, VEC>(py, base, lane, a.d, raw);
      unpack8<F32>(raw, y);
      load8<F32, VEC>(pr, base, lane, a.d, raw);
      unpack8<F32>(raw, x);
      load8<F32, VEC>(a.gain, base, lane, a.d, raw);
      unpack8<F32>(raw, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = y[e] * (x[e] * rstd);
        const int c = column<VEC>(base, lane, e);
        if (a.dgain && c < a.d) line[c] += s;
        dot = fmaf(s, t[e], dot);
      }
    }
    dot = row_sum(dot, slots[turn], w, WIDE_WARPS, lane) / static_cast<float>(a.d);
    uint8_t *px = static_cast<uint8_t *>(a.dx) + row * a.dx_stride * E;
    uint8_t *ps = static_cast<uint8_t *>(a.dresidual) + row * a.dresidual_stride * E;
    for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256) {
      Raw<F32> raw;
      float y[8], x[8], o[8];
      load8<F32, VEC>(a.gain, base, lane, a.d, raw);
      unpack8<F32>(raw, o);
      load8<F32, VEC>(py, base, lane, a.d, raw);
      unpack8<F32>(raw, y);
      load8<F32, VEC>(pr, base, lane, a.d, raw);
      unpack8<F32>(raw, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = rstd * (y[e] * o[e] - x[e] * rstd * dot);
      if (a.dr) {
        load8<F32, VEC>(pd, base, lane, a.d, raw);
        unpack8<F32>(raw, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += y[e];
      }
      if (a.dresidual) store8<F32, VEC>(ps, base, lane, a.d, o);
      if (a.dx) {
        if (a.drop.on) drop8<VEC>(a.drop, base, lane, static_cast<int>(row), o);
        store8<F32, VEC>(px, base, lane, a.d, o);
      }
    }
  }
  if (!a.dgain) return;
  float *out = a.partial + static_cast<int64_t>(blockIdx.x) * a.d;
  for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<VEC>(base, lane, e);
      if (c < a.d) out[c] = line[c];
    }
}

template <bool F32>
__global__ void __launch_bounds__(1024)
    dgain_kernel(const float *partial, int lines, int d, void *dgain) {
  allow_next_kernel();
  wait_for_earlier_kernel();
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < d)
    for (int i = w; i < lines; i += 32) s += partial[static_cast<int64_t>(i) * d + c];
  part[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < d) {
    s = 0.0f;
    for (int i = 0; i < 32; ++i) s += part[i][lane];
    if (F32)
      static_cast<float *>(dgain)[c] = s;
    else
      static_cast<uint16_t *>(dgain)[c] = to_bf16(s);
  }
}

// ------------------------------------------------- dropout by itself
// A CTA takes `rows_per_cta` rows of `chunks` 256-column chunks; warps go over
// them in order.
template <bool F32, bool VEC>
__global__ void __launch_bounds__(256) dropout_kernel(const DropoutArgs a, int rows_per_cta,
                                                      int chunks) {
  allow_next_kernel();
  wait_for_earlier_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int E = F32 ? 4 : 2;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * rows_per_cta;
  const int n = static_cast<int>(min(static_cast<int64_t>(rows_per_cta), a.M - r0)) * chunks;
  for (int i = warp; i < n; i += 8) {
    const int rr = i / chunks, base = (i - rr * chunks) * 256;
    const int64_t row = r0 + rr;
    Raw<F32> rx, rs;
    load8<F32, VEC>(static_cast<const uint8_t *>(a.x) + row * a.x_stride * E, base, lane, a.d, rx);
    if (a.residual)
      load8<F32, VEC>(static_cast<const uint8_t *>(a.residual) + row * a.residual_stride * E, base,
                      lane, a.d, rs);
    float v[8];
    unpack8<F32>(rx, v);
    if (a.drop.on) drop8<VEC>(a.drop, base, lane, static_cast<int>(row), v);
    if (a.residual) {
      float t[8];
      unpack8<F32>(rs, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += t[e];
    }
    store8<F32, VEC>(static_cast<uint8_t *>(a.y) + row * a.y_stride * E, base, lane, a.d, v);
  }
}

// ------------------------------------------------------------------ host
bool wide(const void *p, int64_t stride, int esz, int bytes) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0 &&
                          (stride * esz) % bytes == 0);
}

// How a row is spread: chunks of 256 columns, nv of them a warp; nv = 0: rows
// too wide to hold, a CTA to a row.
struct RowPlan {
  int nv, warps, rows_per_cta, threads;
};

constexpr int kHeldColumns = 8192;

RowPlan row_plan(int d, int nv) {
  if (d > kHeldColumns) return {0, WIDE_WARPS, 1, WIDE_WARPS * 32};
  RowPlan p;
  const int chunks = (d + 255) / 256;
  p.nv = std::min(nv, chunks >= 4 ? 4 : chunks >= 2 ? 2 : 1);
  p.warps = (chunks + p.nv - 1) / p.nv;
  p.rows_per_cta = std::max(1, 4 / p.warps);
  p.threads = p.rows_per_cta * p.warps * 32;
  return p;
}

// forward: two chunks a warp
RowPlan norm_plan(int d) { return row_plan(d, 4); }

// gradient: one chunk a warp, so that the sums and two rows fit 64 registers;
// in the odd layout two, where addresses take more of them
RowPlan norm_grad_plan(int d, bool vec) { return row_plan(d, vec ? 1 : 2); }

// CTAs go over the rows: as many as a GB300 holds at 64 registers a thread.
int grad_grid(int32_t M, const RowPlan &p) {
  const int64_t most = 152 * std::max(1, 1024 / p.threads);
  return static_cast<int>(
      std::min<int64_t>((static_cast<int64_t>(M) + p.rows_per_cta - 1) / p.rows_per_cta, most));
}

template <bool F32, bool VEC>
cudaError_t norm_launch_t(const NormArgs &a, cudaStream_t st) {
  const RowPlan p = norm_plan(a.d);
  const unsigned grid = (static_cast<int64_t>(a.M) + p.rows_per_cta - 1) / p.rows_per_cta;
  switch (p.nv) {
    case 0: return launch_overlapped(norm_wide_kernel<F32, VEC>, grid, p.threads, 0, st, a);
    case 1: return launch_overlapped(norm_kernel<F32, VEC, 1>, grid, p.threads, 0, st, a, p.warps);
    case 2: return launch_overlapped(norm_kernel<F32, VEC, 2>, grid, p.threads, 0, st, a, p.warps);
    default: return launch_overlapped(norm_kernel<F32, VEC, 4>, grid, p.threads, 0, st, a, p.warps);
  }
}

template <bool F32, bool VEC>
cudaError_t norm_grad_launch_t(const NormGradArgs &a, cudaStream_t st) {
  const RowPlan p = norm_grad_plan(a.d, VEC);
  const int grid = grad_grid(a.M, p);
  const size_t line = static_cast<size_t>(a.d) * 4;
  const size_t sm = p.rows_per_cta > 1 ? line : 0;
  cudaError_t e;
  if (p.nv == 0) {
    const auto kernel = norm_grad_wide_kernel<F32, VEC>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxNormColumns * 4);
    if (e == cudaSuccess)
      e = launch_overlapped(kernel, grid, p.threads, a.dgain ? line : 0, st, a);
  } else if (p.nv == 1) {
    e = launch_overlapped(norm_grad_kernel<F32, VEC, 1, 1024>, grid, p.threads, sm, st, a, p.warps);
  } else {
    e = launch_overlapped(norm_grad_kernel<F32, VEC, 2, 512>, grid, p.threads, sm, st, a, p.warps);
  }
  if (e != cudaSuccess || !a.dgain) return e;
  return launch_overlapped(dgain_kernel<F32>, (a.d + 31) / 32, 1024, 0, st,
                           static_cast<const float *>(a.partial), grid, a.d, a.dgain);
}

template <bool F32, bool VEC>
cudaError_t dropout_launch_t(const DropoutArgs &a, cudaStream_t st) {
  const int chunks = (a.d + 255) / 256;
  const int rows = std::max(1, 16 / chunks);
  const unsigned grid = (static_cast<int64_t>(a.M) + rows - 1) / rows;
  return launch_overlapped(dropout_kernel<F32, VEC>, grid, 256, 0, st, a, rows, chunks);
}

dspark_status result(cudaError_t e) { return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA; }

}  // namespace

size_t norm_workspace_bytes(int32_t M, int32_t d) {
  // either layout's lines
  const int lines =
      std::max(grad_grid(M, norm_grad_plan(d, true)), grad_grid(M, norm_grad_plan(d, false)));
  return kNormPartialOffset + static_cast<size_t>(lines) * d * 4;
}

dspark_status norm_launch(const NormArgs &a, cudaStream_t st) {
  const int e = a.f32 ? 4 : 2;
  const bool vec = a.d % 8 == 0 && wide(a.x, a.x_stride, e, 16) &&
                   wide(a.residual, a.residual_stride, e, 16) && wide(a.r, a.r_stride, e, 16) &&
                   wide(a.gain, 0, e, 16) &&
                   wide(a.y, a.y_stride, a.e4m3 ? 1 : e, a.e4m3 ? 8 : 16);
  if (a.f32) return result(vec ? norm_launch_t<true, true>(a, st) : norm_launch_t<true, false>(a, st));
  return result(vec ? norm_launch_t<false, true>(a, st) : norm_launch_t<false, false>(a, st));
}

dspark_status norm_grad_launch(const NormGradArgs &a, cudaStream_t st) {
  const int e = a.f32 ? 4 : 2;
  const bool vec = a.d % 8 == 0 && wide(a.dy, a.dy_stride, e, 16) &&
                   wide(a.dr, a.dr_stride, e, 16) && wide(a.r, a.r_stride, e, 16) &&
                   wide(a.gain, 0, e, 16) && wide(a.dx, a.dx_stride, e, 16) &&
                   wide(a.dresidual, a.dresidual_stride, e, 16);
  if (a.f32)
    return result(vec ? norm_grad_launch_t<true, true>(a, st) : norm_grad_launch_t<true, false>(a, st));
  return result(vec ? norm_grad_launch_t<false, true>(a, st) : norm_grad_launch_t<false, false>(a, st));
}

dspark_status dropout_launch(const DropoutArgs &a, cudaStream_t st) {
  const int e = a.f32 ? 4 : 2;
  const bool vec = a.d % 8 == 0 && wide(a.x, a.x_stride, e, 16) &&
                   wide(a.residual, a.residual_stride, e, 16) && wide(a.y, a.y_stride, e, 16);
  if (a.f32)
    return result(vec ? dropout_launch_t<true, true>(a, st) : dropout_launch_t<true, false>(a, st));
  return result(vec ? dropout_launch_t<false, true>(a, st) : dropout_launch_t<false, false>(a, st));
}

}  // namespace dspark
