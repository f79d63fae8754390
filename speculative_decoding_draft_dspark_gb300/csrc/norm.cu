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

__device__ __forceinline__ Philox4 drop_words(const DropArgs &d, int group, int row) {
  uint32_t c0 = static_cast<uint32_t>(group), c1 = static_cast<uint32_t>(row);
  uint32_t c2 = 0x80000000u, c3 = d.offset, k0 = d.seed_lo, k1 = d.seed_hi;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(p1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

// ----------------------------------------------------- eight columns a lane
// A warp holds 256 columns of a row, in one of four layouts for all tensors of a
// call:
//   kWide   rows at 16 bytes, d a multiple of 8: lane l has columns 8l .. 8l+7,
//           one or two 16-byte accesses
//   kPairs  bf16 rows at 4 bytes: columns 2l, 64 + 2l, 128 + 2l, 192 + 2l and
//           their neighbours, four accesses (at 15360 x 2044 the norm takes 42 us,
//           107 by single columns)
//   kShifted other bf16 rows: the same columns; where a row begins in the middle
//           of a word its words are columns 2l - 1 and 2l, and the lanes hand
//           halves on (at 15360 x 2047 the norm takes 70 us and dropout 48, by
//           single columns 111 and 57; not for the gradient, 86 us by single
//           columns and 111 so: the 64 registers that its launch bound leaves do not
//           hold it)
//   kSingle anything: columns l, 32 + l, ..., 224 + l, eight accesses
// Every access of the warp is to neighbouring words.
enum Layout { kWide = 0, kPairs = 1, kShifted = 2, kSingle = 3 };

template <int L>
__device__ __forceinline__ int column(int base, int lane, int e) {
  return L == kWide     ? base + lane * 8 + e
         : L != kSingle ? base + (e >> 1) * 64 + lane * 2 + (e & 1)
                        : base + e * 32 + lane;
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

// Eight values as four pairs: the packed fp32 instructions do two at once.
struct V8 {
  uint64_t p[4];
};

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void halves(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void split8(const V8 &v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) halves(v.p[i], f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ V8 join8(const float (&f)[8]) {
  V8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = pair(f[2 * i], f[2 * i + 1]);
  return v;
}

// eight values as they lie in memory; kShifted rows that begin in the middle of a
// word are still a half off, until settle()
template <bool F32>
struct Raw {
  uint32_t w[F32 ? 8 : 5];
  bool off;
};

// A row at 2 bytes: no half word of another row is touched.  Where the row is a half
// off, a lane's words are columns c - 1 and c, and lane 0 has the last word's next
// column as well.
__device__ __forceinline__ void load_shifted(const uint16_t *row, int base, int lane, int d,
                                             Raw<false> &r) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1) & 1;
  const int c = base + lane * 2 - off;
  const uint16_t *p = row + c;
  r.off = off;
  r.w[4] = 0u;
  if (base + 256 <= d && base >= off) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = *reinterpret_cast<const uint32_t *>(p + i * 64);
    if (lane == 0) r.w[4] = row[base + 255];
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = c + i * 64 >= 0 && c + i * 64 < d, hi = c + i * 64 + 1 < d;
    r.w[i] = 0u;
    if (lo && hi)
      r.w[i] = *reinterpret_cast<const uint32_t *>(p + i * 64);
    else if (hi)
      r.w[i] = static_cast<uint32_t>(p[i * 64 + 1]) << 16;
    else if (lo)
      r.w[i] = p[i * 64];
  }
  if (lane == 0 && base + 255 < d) r.w[4] = row[base + 255];
}

// After the loads, by all lanes: the halves to where they belong.
template <int L>
__device__ __forceinline__ void settle(Raw<false> &r, int lane) {
  if constexpr (L == kShifted) {
    if (!r.off) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t next =
          __shfl_sync(0xFFFFFFFFu, lane == 0 ? r.w[i + 1] : r.w[i], (lane + 1) & 31);
      r.w[i] = __byte_perm(r.w[i], next, 0x5432);
    }
  }
}
template <int L>
__device__ __forceinline__ void settle(Raw<true> &, int) {}

// Pairs of columns, a word W of two halves H each, likewise.
template <class H, class W>
__device__ __forceinline__ void store_shifted(H *row, int base, int lane, int d,
                                              const uint32_t (&w)[4]) {
  constexpr int B = sizeof(H) * 8;
  const int c = base + lane * 2;
  if (!(reinterpret_cast<uintptr_t>(row) & sizeof(H))) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      H *p = row + c + i * 64;
      if (c + i * 64 + 1 < d)
        *reinterpret_cast<W *>(p) = static_cast<W>(w[i]);
      else if (c + i * 64 < d)
        *p = static_cast<H>(w[i]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t before = __shfl_sync(
        0xFFFFFFFFu, lane == 31 ? w[i > 0 ? i - 1 : 0] : w[i], (lane + 31) & 31);
    H *p = row + c + i * 64;
    if (c + i * 64 < d) {
      if (i == 0 && lane == 0)
        *p = static_cast<H>(w[i]);
      else
        *reinterpret_cast<W *>(p - 1) = static_cast<W>((before >> B) | (w[i] << B));
    } else if (c + i * 64 == d && (i > 0 || lane > 0)) {
      p[-1] = static_cast<H>(before >> B);
    }
  }
  if (lane == 31 && base + 255 < d) row[base + 255] = static_cast<H>(w[3] >> B);
}

template <bool F32, int L>
__device__ __forceinline__ void load8(const void *row, int base, int lane, int d, Raw<F32> &r) {
  if (L == kWide) {
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
  } else if (L == kPairs) {  // d is even
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int c = column<L>(base, lane, e);
      r.w[e / 2] = c < d ? static_cast<const uint32_t *>(row)[c / 2] : 0u;
    }
  } else if (L == kShifted) {
    if constexpr (!F32) load_shifted(static_cast<const uint16_t *>(row), base, lane, d, r);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<L>(base, lane, e);
      if (F32) {
        r.w[F32 ? e : 0] = c < d ? static_cast<const uint32_t *>(row)[c] : 0u;
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
__device__ __forceinline__ V8 unpack8(const Raw<F32> &r) {
  V8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v.p[i] = F32 ? pair(__uint_as_float(r.w[F32 ? 2 * i : 0]),
                        __uint_as_float(r.w[F32 ? 2 * i + 1 : 0]))
                 : pair(bf16_lo(r.w[i]), bf16_hi(r.w[i]));
  return v;
}

template <bool F32, int L>
__device__ __forceinline__ void store8(void *row, int base, int lane, int d, const V8 &x) {
  float v[8];
  split8(x, v);
  if (L == kWide) {
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
  } else if (L == kPairs) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int c = column<L>(base, lane, e);
      if (c < d) static_cast<uint32_t *>(row)[c / 2] = pack_bf16(v[e], v[e + 1]);
    }
  } else if (L == kShifted) {
    const uint32_t w[4] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                           pack_bf16(v[6], v[7])};
    store_shifted<uint16_t, uint32_t>(static_cast<uint16_t *>(row), base, lane, d, w);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<L>(base, lane, e);
      if (c < d) {
        if (F32)
          static_cast<float *>(row)[c] = v[e];
        else
          static_cast<uint16_t *>(row)[c] = to_bf16(v[e]);
      }
    }
  }
}

__device__ __forceinline__ uint32_t pick(bool c, uint32_t a, uint32_t b) { return c ? a : b; }

// The Philox words of a lane's eight columns, two 16-bit lanes each.
template <int L>
__device__ __forceinline__ Philox4 drop8_words(const DropArgs &dr, int base, int lane, int row) {
  const Philox4 p = drop_words(dr, base / 8 + lane, row);
  if (L == kWide) return p;
  // Lane g drew the four words of columns 8g .. 8g+7.
  const int t = lane >> 3;
  uint32_t a[4], b[4], q[4];
  if constexpr (L != kSingle) {
    // Pair i of lane l wants word l % 4 of lane 8i + l / 4.  In step s, lane l
    // asks for its pair (s + l) % 4, so that lane g is asked for one word only,
    // (g / 8 - s) % 4: four shuffles between a rotation before and one after.
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = pick(t & 2, p.w[(j + 2) & 3], p.w[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = pick(t & 1, a[(j + 1) & 3], a[j]);  // word (j + t) % 4
#pragma unroll
    for (int s = 0; s < 4; ++s)
      a[s] = __shfl_sync(0xFFFFFFFFu, b[(4 - s) & 3], ((s + lane) & 3) * 8 + (lane >> 2));
    // a[s] is pair (s + lane) % 4
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = pick(lane & 2, a[(j + 2) & 3], a[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = pick(lane & 1, b[(j + 3) & 3], b[j]);
  } else {
    // column e of lane l wants the 16 bits l % 8 of lane 4e + l / 8
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int src = 4 * e + (lane >> 3);
      const uint32_t w0 = __shfl_sync(0xFFFFFFFFu, p.w[0], src);
      const uint32_t w1 = __shfl_sync(0xFFFFFFFFu, p.w[1], src);
      const uint32_t w2 = __shfl_sync(0xFFFFFFFFu, p.w[2], src);
      const uint32_t w3 = __shfl_sync(0xFFFFFFFFu, p.w[3], src);
      const uint32_t w = pick(lane & 4, pick(lane & 2, w3, w2), pick(lane & 2, w1, w0));
      const uint32_t half = lane & 1 ? w >> 16 : w & 0xFFFFu;
      if (e & 1)
        q[e / 2] |= half << 16;
      else
        q[e / 2] = half;
    }
  }
  return {{q[0], q[1], q[2], q[3]}};
}

// dropout(x); a select, so that what a dropped element holds (NaN, infinity)
// is gone.  A 16-bit lane is kept iff it is below T: the upper half of a word
// compares with T in the upper half, the lower one once shifted there.
__device__ __forceinline__ V8 drop8(const DropArgs &dr, const Philox4 &p, const V8 &x) {
  const uint64_t s = pair(dr.scale, dr.scale);
  V8 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y.p[i] = mul2(x.p[i], s);
  float v[8];
  split8(y, v);
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    v[e] = (p.w[e >> 1] << 16) < dr.keep_hi ? v[e] : 0.0f;
    v[e + 1] = p.w[e >> 1] < dr.keep_hi ? v[e + 1] : 0.0f;
  }
  return join8(v);
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

// A row's warps share values through `slots` (as many as warps).  They meet at
// the CTA's barrier, or (OWN) at one of the row's own, so that the CTA's rows do
// not wait for one another; that takes all 16 barriers of a CTA, and few CTAs
// then fit an SM.
template <bool OWN = false>
__device__ __forceinline__ void row_barrier(int group, int warps) {
  if (OWN)
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
  else
    __syncthreads();
}
template <bool OWN = false>
__device__ __forceinline__ float row_sum(float v, float *slots, int group, int w, int warps,
                                         int lane) {
  v = warp_sum(v);
  if (warps == 1) return v;
  if (lane == 0) slots[group * warps + w] = v;
  row_barrier<OWN>(group, warps);
  return warp_sum(lane < warps ? slots[group * warps + lane] : 0.0f);
}
__device__ __forceinline__ float row_max_nan(float v, float *slots, int group, int w, int warps,
                                             int lane) {
  v = warp_max_nan(v);
  if (warps == 1) return v;
  if (lane == 0) slots[group * warps + w] = v;
  row_barrier(group, warps);
  return warp_max_nan(lane < warps ? slots[group * warps + lane] : 0.0f);
}

// two e4m3 numbers
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

constexpr float kE4m3Max = 448.0f;

__device__ __forceinline__ float scale_of(float top) {
  const float s = top / kE4m3Max;
  return s == 0.0f ? 1.0f : s;  // also where it underflows
}

// The bytes of y / scale, the quotient that fp32 division gives.  Rounding is
// monotone: where products with a little less and a little more than 1 / scale give
// the same byte, the quotient between them has it too (each is off by three
// roundings of 2^-24, the quotient by one; 2^-21 is put between).  Where they differ,
// next to a tie, or where the reciprocal would overflow, it is divided.  15360 x 2048
// with a scale for 128 columns take 39.0 us, 45.2 if all is divided, and 37.5 with
// the reciprocal alone, whose bytes next to a tie are a step off.
struct Quotients {
  float scale;
  uint64_t less, more;
  bool divide;
};

__device__ __forceinline__ Quotients by_scale(float scale) {
  Quotients q;
  const float inv = 1.0f / scale;
  const float less = inv * (1.0f - 0x1p-21f), more = inv * (1.0f + 0x1p-21f);
  q.scale = scale;
  q.less = pair(less, less);
  q.more = pair(more, more);
  q.divide = scale <= 1e-35f;
  return q;
}

// pairs FIRST .. FIRST + N - 1 of the eight
template <int FIRST, int N>
__device__ __forceinline__ void e4m3_of(const V8 &y, const Quotients &q, uint32_t (&w)[4]) {
  uint32_t differ = q.divide;
#pragma unroll
  for (int i = FIRST; i < FIRST + N; ++i) {
    float a, b;
    halves(mul2(y.p[i], q.less), a, b);
    w[i] = e4m3x2(a, b);
    halves(mul2(y.p[i], q.more), a, b);
    differ |= w[i] ^ e4m3x2(a, b);
  }
  if (differ) {
#pragma unroll
    for (int i = FIRST; i < FIRST + N; ++i) {
      float a, b;
      halves(y.p[i], a, b);
      w[i] = e4m3x2(a / q.scale, b / q.scale);
    }
  }
}

template <int L>
__device__ __forceinline__ void store8_e4m3(uint8_t *row, int base, int lane, int d,
                                            const uint32_t (&w)[4]) {
  if (L == kWide) {
    const int c = base + lane * 8;
    if (c >= d) return;
    *reinterpret_cast<uint2 *>(row + c) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  } else if (L == kPairs) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int c = column<L>(base, lane, e);
      if (c < d) *reinterpret_cast<uint16_t *>(row + c) = static_cast<uint16_t>(w[e / 2]);
    }
  } else if (L == kShifted) {
    store_shifted<uint8_t, uint16_t>(row, base, lane, d, w);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<L>(base, lane, e);
      if (c < d) row[c] = static_cast<uint8_t>(w[e / 2] >> (8 * (e & 1)));
    }
  }
}

// The bytes with a scale for 128 columns: 16 lanes if a lane's columns are
// neighbours, else the warp's first or last four
template <int L>
__device__ __forceinline__ void by_groups(const NormArgs &a, int64_t row, int base, int lane,
                                          const V8 &y, uint32_t (&w)[4]) {
  float v[8];
  split8(y, v);
  float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) t0 = fmax_nan(t0, fabsf(v[e]));
#pragma unroll
  for (int e = 4; e < 8; ++e) t1 = fmax_nan(t1, fabsf(v[e]));
  if (L == kWide) {
    t0 = fmax_nan(t0, t1);
#pragma unroll
    for (int o = 8; o; o >>= 1) t0 = fmax_nan(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, o));
    const float s = scale_of(t0);
    if ((lane & 15) == 0 && base + lane * 8 < a.d)
      a.scale[row * a.groups + (base + lane * 8) / 128] = s;
    e4m3_of<0, 4>(y, by_scale(s), w);
  } else {
    const float s0 = scale_of(warp_max_nan(t0)), s1 = scale_of(warp_max_nan(t1));
    if (lane == 0 && base < a.d) a.scale[row * a.groups + base / 128] = s0;
    if (lane == 0 && base + 128 < a.d) a.scale[row * a.groups + base / 128 + 1] = s1;
    e4m3_of<0, 2>(y, by_scale(s0), w);
    e4m3_of<2, 2>(y, by_scale(s1), w);
  }
}

__device__ __forceinline__ float top8(float top, const V8 &y) {
  float v[8];
  split8(y, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmax_nan(top, fabsf(v[e]));
  return top;
}

// sum of squares, two running sums
__device__ __forceinline__ void squares8(const V8 &r, uint64_t &sum) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = fma2(r.p[i], r.p[i], sum);
}

// r rstd gain
template <bool F32, int L>
__device__ __forceinline__ V8 times_gain(const void *gain, float rstd, int base, int lane, int d,
                                         const V8 &r) {
  Raw<F32> raw;
  load8<F32, L>(gain, base, lane, d, raw);
  settle<L>(raw, lane);
  const V8 g = unpack8<F32>(raw);
  const uint64_t s = pair(rstd, rstd);
  V8 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y.p[i] = mul2(mul2(r.p[i], s), g.p[i]);
  return y;
}

// ---------------------------------------------------------------- forward
// `warps` warps hold a row, NV x 256 columns each (chunk i of a warp starts at
// column 256 (i warps + w)); a CTA has as many rows as fit.  Up to four chunks a
// warp: one row's loads are all in flight before its sum, and most rows need one
// or two warps and a barrier of few.  At 15360 x 2048 bf16 39 us in 16 bits (95%
// of measured HBM), 39 in 8 bits with a scale for 128 columns (84%: the scales'
// maxima and conversions), 45 with dropout as well (72%: a chunk's Philox words are
// drawn after its load has been waited for, not under it; dropout_kernel draws as
// many at 94%).  Few rows: the latency of a load, a sum and a store, 3.9 us for 56
// rows.
template <bool F32, int L, int NV>
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

  V8 r[NV];
  uint64_t sum2 = 0;
  if (live) {
    Raw<F32> rx[NV], rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) load8<F32, L>(x, (i * warps + w) * 256, lane, a.d, rx[i]);
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < NV; ++i) load8<F32, L>(res, (i * warps + w) * 256, lane, a.d, rr[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      settle<L>(rx[i], lane);
      r[i] = unpack8<F32>(rx[i]);
      if (a.drop.on)
        r[i] = drop8(
            a.drop, drop8_words<L>(a.drop, (i * warps + w) * 256, lane, static_cast<int>(row)),
            r[i]);
      if (a.residual) {
        settle<L>(rr[i], lane);
        const V8 t = unpack8<F32>(rr[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) r[i].p[e] = add2(r[i].p[e], t.p[e]);
      }
      squares8(r[i], sum2);
    }
  }
  float lo, hi;
  halves(sum2, lo, hi);
  const float sum = row_sum(lo + hi, slots[0], group, w, warps, lane);
  const float rstd = rsqrtf(fmaf(sum, a.inv_d, a.eps));
  float top = 0.0f;
  if (live) {
    if (a.rstd && w == 0 && lane == 0) a.rstd[row] = rstd;
    uint8_t *ro = static_cast<uint8_t *>(a.r) + row * a.r_stride * E;
    uint8_t *yo = static_cast<uint8_t *>(a.y) + row * a.y_stride * (a.e4m3 ? 1 : E);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int base = (i * warps + w) * 256;
      if (a.r) store8<F32, L>(ro, base, lane, a.d, r[i]);
      r[i] = times_gain<F32, L>(a.gain, rstd, base, lane, a.d, r[i]);
      if (!a.e4m3) {
        store8<F32, L>(yo, base, lane, a.d, r[i]);
      } else if (a.group == 0) {
        top = top8(top, r[i]);
      } else {
        uint32_t bytes[4];
        by_groups<L>(a, row, base, lane, r[i], bytes);
        store8_e4m3<L>(yo, base, lane, a.d, bytes);
      }
    }
  }
  if (a.e4m3 && a.group == 0) {
    const float s = scale_of(row_max_nan(top, slots[1], group, w, warps, lane));
    if (live) {
      if (w == 0 && lane == 0) a.scale[row] = s;
      uint8_t *yo = static_cast<uint8_t *>(a.y) + row * a.y_stride;
      const Quotients q = by_scale(s);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        uint32_t bytes[4];
        e4m3_of<0, 4>(r[i], q, bytes);
        store8_e4m3<L>(yo, (i * warps + w) * 256, lane, a.d, bytes);
      }
    }
  }
}

// Rows too wide to hold: a CTA to a row, which is read again (from L2) for
// every use of it.
constexpr int WIDE_WARPS = 16;

template <bool F32, int L>
__device__ __forceinline__ V8 stream8(const NormArgs &a, const uint8_t *x, const uint8_t *res,
                                      int64_t row, int base, int lane) {
  Raw<F32> rx, rr;
  load8<F32, L>(x, base, lane, a.d, rx);
  if (a.residual) load8<F32, L>(res, base, lane, a.d, rr);
  settle<L>(rx, lane);
  V8 r = unpack8<F32>(rx);
  if (a.drop.on) r = drop8(a.drop, drop8_words<L>(a.drop, base, lane, static_cast<int>(row)), r);
  if (a.residual) {
    settle<L>(rr, lane);
    const V8 t = unpack8<F32>(rr);
#pragma unroll
    for (int e = 0; e < 4; ++e) r.p[e] = add2(r.p[e], t.p[e]);
  }
  return r;
}

template <bool F32, int L>
__global__ void __launch_bounds__(WIDE_WARPS * 32) norm_wide_kernel(const NormArgs a) {
  allow_next_kernel();
  wait_for_earlier_kernel();
  __shared__ float slots[2][32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  constexpr int E = F32 ? 4 : 2;
  const uint8_t *x = static_cast<const uint8_t *>(a.x) + row * a.x_stride * E;
  const uint8_t *res = static_cast<const uint8_t *>(a.residual) + row * a.residual_stride * E;
  uint64_t sum2 = 0;
  for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256)
    squares8(stream8<F32, L>(a, x, res, row, base, lane), sum2);
  float lo, hi;
  halves(sum2, lo, hi);
  const float sum = row_sum(lo + hi, slots[0], 0, w, WIDE_WARPS, lane);
  const float rstd = rsqrtf(fmaf(sum, a.inv_d, a.eps));
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  float s = 1.0f;
  if (a.e4m3 && a.group == 0) {
    float top = 0.0f;
    for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256) {
      const V8 r = stream8<F32, L>(a, x, res, row, base, lane);
      top = top8(top, times_gain<F32, L>(a.gain, rstd, base, lane, a.d, r));
    }
    s = scale_of(row_max_nan(top, slots[1], 0, w, WIDE_WARPS, lane));
    if (threadIdx.x == 0) a.scale[row] = s;
  }
  uint8_t *ro = static_cast<uint8_t *>(a.r) + row * a.r_stride * E;
  uint8_t *yo = static_cast<uint8_t *>(a.y) + row * a.y_stride * (a.e4m3 ? 1 : E);
  for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256) {
    const V8 r = stream8<F32, L>(a, x, res, row, base, lane);
    if (a.r) store8<F32, L>(ro, base, lane, a.d, r);
    const V8 y = times_gain<F32, L>(a.gain, rstd, base, lane, a.d, r);
    if (!a.e4m3) {
      store8<F32, L>(yo, base, lane, a.d, y);
      continue;
    }
    uint32_t bytes[4];
    if (a.group == 0)
      e4m3_of<0, 4>(y, by_scale(s), bytes);
    else
      by_groups<L>(a, row, base, lane, y, bytes);
    store8_e4m3<L>(yo, base, lane, a.d, bytes);
  }
}

// --------------------------------------------------------------- backward
// A row as in the forward kernel.  A CTA goes over rows and keeps dgain's sums of
// its columns in registers, joins its row groups in order and writes one fp32
// line of partial sums.  dgain_kernel adds the lines up in order.  HBM bounds it:
// at 15360 x 2048 bf16 with dropout 58 us for both kernels, 80% of measured HBM
// (the first one 50 to 53 us; the rest is the second one's launch and latency).
template <bool F32>
struct GradRow {
  Raw<F32> dy, r, dr;
  float rstd;
};

template <bool F32, int L>
__device__ __forceinline__ void load_row(const NormGradArgs &a, int64_t row, int base, int lane,
                                         GradRow<F32> &x) {
  constexpr int E = F32 ? 4 : 2;
  load8<F32, L>(static_cast<const uint8_t *>(a.dy) + row * a.dy_stride * E, base, lane, a.d, x.dy);
  load8<F32, L>(static_cast<const uint8_t *>(a.r) + row * a.r_stride * E, base, lane, a.d, x.r);
  if (a.dr)
    load8<F32, L>(static_cast<const uint8_t *>(a.dr) + row * a.dr_stride * E, base, lane, a.d,
                    x.dr);
  x.rstd = a.rstd[row];
}

// a row's lines on their way to L2
template <bool F32>
__device__ __forceinline__ void row_to_l2(const NormGradArgs &a, int64_t row, int base, int lane) {
  constexpr int E = F32 ? 4 : 2;
  const int c = base + lane * (128 / E);
  if (row >= a.M || lane >= 2 * E || c >= a.d) return;
  asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t *>(a.dy) +
                                                (row * a.dy_stride + c) * E));
  asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t *>(a.r) +
                                                (row * a.r_stride + c) * E));
  if (a.dr)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t *>(a.dr) +
                                                  (row * a.dr_stride + c) * E));
}

// What a row keeps between its sum and its use: xh = r rstd and a = dy gain.
struct GradHalf {
  V8 xh, a;
};

// dg += dy xh, dot += a xh
template <bool F32>
__device__ __forceinline__ GradHalf grad_dot(const GradRow<F32> &x, const Raw<F32> &gain, V8 &dg,
                                             uint64_t &dot) {
  const V8 y = unpack8<F32>(x.dy), r = unpack8<F32>(x.r), g = unpack8<F32>(gain);
  const uint64_t rs = pair(x.rstd, x.rstd);
  GradHalf h;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h.xh.p[e] = mul2(r.p[e], rs);
    h.a.p[e] = mul2(y.p[e], g.p[e]);
    dg.p[e] = fma2(y.p[e], h.xh.p[e], dg.p[e]);
    dot = fma2(h.a.p[e], h.xh.p[e], dot);
  }
  return h;
}

// dr' = rstd (a - xh mean) + dr
template <bool F32>
__device__ __forceinline__ V8 grad_sum(const Raw<F32> *dr, const GradHalf &h, float rstd,
                                       float mean) {
  const uint64_t rs = pair(rstd, rstd), m = pair(-mean, -mean);
  V8 o = {};
  if (dr) o = unpack8<F32>(*dr);
#pragma unroll
  for (int e = 0; e < 4; ++e) o.p[e] = fma2(fma2(h.xh.p[e], m, h.a.p[e]), rs, o.p[e]);
  return o;
}

template <bool F32, int L>
__device__ __forceinline__ void grad_out(const NormGradArgs &a, int64_t row, int base, int lane,
                                         const GradRow<F32> &x, const GradHalf &h, float mean,
                                         const Philox4 &words) {
  constexpr int E = F32 ? 4 : 2;
  V8 o = grad_sum<F32>(a.dr ? &x.dr : nullptr, h, x.rstd, mean);
  if (a.dresidual)
    store8<F32, L>(static_cast<uint8_t *>(a.dresidual) + row * a.dresidual_stride * E, base, lane,
                     a.d, o);
  if (a.dx) {
    if (a.drop.on) o = drop8(a.drop, words, o);
    store8<F32, L>(static_cast<uint8_t *>(a.dx) + row * a.dx_stride * E, base, lane, a.d, o);
  }
}

// a CTA's line of dgain: the row groups' sums, joined in order
template <int L>
__device__ __forceinline__ void write_line(const NormGradArgs &a, float *lines, int group,
                                           int groups, int base, int lane, const V8 &dg) {
  float *line = a.partial + static_cast<int64_t>(blockIdx.x) * a.d;
  float sums[8];
  split8(dg, sums);
  for (int k = 0; k < groups; ++k) {
    if (group == k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<L>(base, lane, e);
        if (c < a.d) {
          if (groups == 1)
            line[c] = sums[e];
          else if (k == 0)
            lines[c] = sums[e];
          else if (k < groups - 1)
            lines[c] += sums[e];
          else
            line[c] = lines[c] + sums[e];
        }
      }
    }
    __syncthreads();
  }
}

// Aligned bf16 rows, NV chunks a warp.  Every thread copies its own columns of the
// next rows into shared memory, two rows before it reads them, and no other
// thread's: the copies need no barrier and hold no registers.
constexpr int kAhead = 2;

template <int NV>
__global__ void __launch_bounds__(512)
    norm_grad_kernel(const NormGradArgs a, int warps) {
  __shared__ float slots[2][32];
  extern __shared__ __align__(16) uint8_t dyn[];
  constexpr bool F32 = false;
  constexpr int E = 2;
  wait_for_earlier_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / warps, w = warp - group * warps;
  const int groups = (blockDim.x >> 5) / warps;
  const int c = w * 256 + lane * 8, chunk = warps * 256;  // chunk i: c + i * chunk
  V8 dg[NV] = {};

  const int step = gridDim.x * groups;
  int row = blockIdx.x * groups + group;
  const int rounds = (a.M - static_cast<int>(blockIdx.x) * groups + step - 1) / step;
  auto at = [&](const void *p, int64_t stride) {
    return static_cast<const uint8_t *>(p) + (row * stride + c) * E;
  };
  const uint8_t *dy = at(a.dy, a.dy_stride), *r = at(a.r, a.r_stride), *dr = at(a.dr, a.dr_stride);
  const int64_t dy_step = step * a.dy_stride * E, r_step = step * a.r_stride * E,
                dr_step = step * a.dr_stride * E;
  uint8_t *dx = const_cast<uint8_t *>(at(a.dx, a.dx_stride)),
          *ds = const_cast<uint8_t *>(at(a.dresidual, a.dresidual_stride));
  const int64_t dx_step = step * a.dx_stride * E, ds_step = step * a.dresidual_stride * E;

  // a stage: dy, r and dr, each NV parts of 16 bytes a thread, and rstd
  const uint32_t part = blockDim.x * 16, tensor = NV * part;
  const uint32_t stage = 3 * tensor + part / 4;
  const uint32_t mine = smem_u32(dyn) + threadIdx.x * 16;
  const uint32_t rstd_at = 3 * tensor - threadIdx.x * 12;
  uint32_t fill = mine, use = mine;
  const uint32_t end = mine + (kAhead + 1) * stage;
  int fill_row = row;
  // the gain's columns, behind the stages
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (c + i * chunk < a.d)
      cp_async_16(end + i * part,
                  static_cast<const uint8_t *>(a.gain) + static_cast<size_t>(c + i * chunk) * E);
  }
  auto copy_row = [&] {
    if (fill_row < a.M) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (c + i * chunk < a.d) {
          const uint32_t to = fill + i * part;
          const int from = i * chunk * E;
          cp_async_16(to, dy + from);
          cp_async_16(to + tensor, r + from);
          if (a.dr) cp_async_16(to + 2 * tensor, dr + from);
        }
      }
      cp_async_4(fill + rstd_at, a.rstd + fill_row);
    }
    cp_async_commit();
    dy += dy_step;
    r += r_step;
    dr += dr_step;
    fill_row += step;
    fill += stage;
    if (fill == end) fill = mine;
  };
  auto get = [&](uint32_t from, Raw<F32> &x) {
    const uint4 v = ld_shared_v4(from);
    x.w[0] = v.x;
    x.w[1] = v.y;
    x.w[2] = v.z;
    x.w[3] = v.w;
  };
  for (int i = 0; i < kAhead; ++i) copy_row();

  for (int k = 0; k < rounds; ++k, row += step) {
    copy_row();
    cp_async_wait<kAhead>();
    const bool live = row < a.M;
    uint64_t dot2 = 0;
    float rstd = 0.0f;
    GradHalf h[NV];
    if (live) {
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(rstd) : "r"(use + rstd_at));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (c + i * chunk < a.d) {
          GradRow<F32> x;
          Raw<F32> g;
          x.rstd = rstd;
          get(use + i * part, x.dy);
          get(use + tensor + i * part, x.r);
          get(end + i * part, g);
          h[i] = grad_dot<F32>(x, g, dg[i], dot2);
        }
      }
    }
    float lo, hi;
    halves(dot2, lo, hi);
    // the mask needs none of the data: drawn before the sum is waited for
    Philox4 words[NV];
    if (a.drop.on && a.dx) {
#pragma unroll
      for (int i = 0; i < NV; ++i) words[i] = drop_words(a.drop, (c + i * chunk) / 8, row);
    }
    // two sets of slots: a row's sums are read while the next row's are written
    const float mean = row_sum<true>(lo + hi, slots[k & 1], group, w, warps, lane) * a.inv_d;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (c + i * chunk < a.d) {
          Raw<F32> t;
          if (a.dr) get(use + 2 * tensor + i * part, t);
          V8 o = grad_sum<F32>(a.dr ? &t : nullptr, h[i], rstd, mean);
          // (column 0 of a row that begins at these columns)
          if (a.dresidual) store8<F32, kWide>(ds + i * chunk * E, -lane * 8, lane, 1, o);
          if (a.dx) {
            if (a.drop.on) o = drop8(a.drop, words[i], o);
            store8<F32, kWide>(dx + i * chunk * E, -lane * 8, lane, 1, o);
          }
        }
      }
    }
    dx += dx_step;
    ds += ds_step;
    use += stage;
    if (use == end) use = mine;
  }
  // not before: CTAs that wait here for the rows' end take the place of ones
  // that work (70 us instead of 59 at 15360 x 2048)
  allow_next_kernel();
  if (!a.dgain) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i)
    write_line<kWide>(a, reinterpret_cast<float *>(dyn), group, groups, w * 256 + i * chunk, lane,
                     dg[i]);
}

// Other rows: the next row's lines are sent to L2 instead.  (fp32 rows too: copied
// ahead, with two chunks a warp, 7680 x 2048 of them took 102 us instead of 57.)  The
// launch bound, 1024 threads for the widest rows, leaves 64 registers: aligned and
// single-column fp32 rows spill 24 to 28 bytes, bf16 ones 8.
template <bool F32, int L>
__global__ void __launch_bounds__(1024) norm_grad_direct_kernel(const NormGradArgs a, int warps) {
  __shared__ float slots[2][32];
  extern __shared__ __align__(16) uint8_t dyn[];
  allow_next_kernel();
  wait_for_earlier_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / warps, w = warp - group * warps;
  const int groups = (blockDim.x >> 5) / warps;
  const int base = w * 256;
  V8 dg = {};
  Raw<F32> g;
  load8<F32, L>(a.gain, base, lane, a.d, g);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int turn = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * groups; r0 < a.M; r0 += step, turn ^= 1) {
    const int64_t row = r0 + group;
    const bool live = row < a.M;
    uint64_t dot2 = 0;
    GradHalf h;
    GradRow<F32> x;
    if (live) {
      load_row<F32, L>(a, row, base, lane, x);
      row_to_l2<F32>(a, row + step, base, lane);
      h = grad_dot<F32>(x, g, dg, dot2);
    }
    float lo, hi;
    halves(dot2, lo, hi);
    Philox4 words = {};
    if (a.drop.on && a.dx) words = drop8_words<L>(a.drop, base, lane, static_cast<int>(row));
    const float mean = row_sum(lo + hi, slots[turn], group, w, warps, lane) * a.inv_d;
    if (live) grad_out<F32, L>(a, row, base, lane, x, h, mean, words);
  }
  if (!a.dgain) return;
  write_line<L>(a, reinterpret_cast<float *>(dyn), group, groups, base, lane, dg);
}

// Rows too wide to hold: a CTA to a row, read twice; dgain's sums stay in
// shared memory, every column with one thread.
template <bool F32, int L>
__global__ void __launch_bounds__(WIDE_WARPS * 32) norm_grad_wide_kernel(const NormGradArgs a) {
  __shared__ float slots[2][32];
  extern __shared__ float line[];
  allow_next_kernel();
  wait_for_earlier_kernel();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (a.dgain)
    for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<L>(base, lane, e);
        if (c < a.d) line[c] = 0.0f;
      }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
    uint64_t dot2 = 0;
    for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256) {
      GradRow<F32> x;
      Raw<F32> g;
      load8<F32, L>(a.gain, base, lane, a.d, g);
      load_row<F32, L>(a, row, base, lane, x);
      V8 dg = {};
      grad_dot<F32>(x, g, dg, dot2);
      float s[8];
      split8(dg, s);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<L>(base, lane, e);
        if (a.dgain && c < a.d) line[c] += s[e];
      }
    }
    float lo, hi;
    halves(dot2, lo, hi);
    const float mean = row_sum(lo + hi, slots[turn], 0, w, WIDE_WARPS, lane) * a.inv_d;
    for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256) {
      GradRow<F32> x;
      Raw<F32> g;
      load8<F32, L>(a.gain, base, lane, a.d, g);
      load_row<F32, L>(a, row, base, lane, x);
      V8 dg = {};
      const GradHalf h = grad_dot<F32>(x, g, dg, dot2);
      Philox4 words = {};
      if (a.drop.on && a.dx) words = drop8_words<L>(a.drop, base, lane, static_cast<int>(row));
      grad_out<F32, L>(a, row, base, lane, x, h, mean, words);
    }
  }
  if (!a.dgain) return;
  float *out = a.partial + static_cast<int64_t>(blockIdx.x) * a.d;
  for (int base = w * 256; base < a.d; base += WIDE_WARPS * 256)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<L>(base, lane, e);
      if (c < a.d) out[c] = line[c];
    }
}

// Eight columns (a sector) of 64 lines at a time; the order is fixed.  152 lines
// of 2048 columns are 1.2 MB from L2: 4 us, all of it latency.  With 16 warps
// four CTAs fit an SM (32 warps: 777 x 5001 fp32 23.7 us instead of 22.8 for both
// kernels).
constexpr int DGAIN_COLS = 8;
constexpr int DGAIN_WARPS = 16;

template <bool F32>
__global__ void __launch_bounds__(DGAIN_WARPS * 32)
    dgain_kernel(const float *partial, int lines, int d, void *dgain) {
  __shared__ float part[DGAIN_WARPS][DGAIN_COLS];
  allow_next_kernel();
  wait_for_earlier_kernel();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * DGAIN_COLS + (lane & 7);
  float s = 0.0f;
  if (c < d) {
#pragma unroll 8
    for (int i = w * 4 + (lane >> 3); i < lines; i += DGAIN_WARPS * 4)
      s += partial[static_cast<int64_t>(i) * d + c];
  }
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
  if (lane < DGAIN_COLS) part[w][lane] = s;
  __syncthreads();
  if (w > 0) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < DGAIN_WARPS / 4; ++i)
    s += part[(lane >> 3) * (DGAIN_WARPS / 4) + i][lane & 7];
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
  if (lane < DGAIN_COLS && c < d) {
    if (F32)
      static_cast<float *>(dgain)[c] = s;
    else
      static_cast<uint16_t *>(dgain)[c] = to_bf16(s);
  }
}

// ------------------------------------------------- dropout by itself
// A CTA takes `rows_per_cta` rows of `chunks` 256-column chunks; warps go over
// them in order.  HBM: at 15360 x 2048 bf16 29.5 us, 94% of measured.
template <bool F32, int L>
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
    load8<F32, L>(static_cast<const uint8_t *>(a.x) + row * a.x_stride * E, base, lane, a.d, rx);
    if (a.residual)
      load8<F32, L>(static_cast<const uint8_t *>(a.residual) + row * a.residual_stride * E, base,
                      lane, a.d, rs);
    settle<L>(rx, lane);
    V8 v = unpack8<F32>(rx);
    if (a.drop.on) v = drop8(a.drop, drop8_words<L>(a.drop, base, lane, static_cast<int>(row)), v);
    if (a.residual) {
      settle<L>(rs, lane);
      const V8 t = unpack8<F32>(rs);
#pragma unroll
      for (int e = 0; e < 4; ++e) v.p[e] = add2(v.p[e], t.p[e]);
    }
    store8<F32, L>(static_cast<uint8_t *>(a.y) + row * a.y_stride * E, base, lane, a.d, v);
  }
}

// ------------------------------------------------------------------ host
// Whether every row of a tensor (or none: NULL) begins at a multiple of `bytes`.
bool rows_at(const void *p, int64_t stride, int esz, int bytes) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0 &&
                          (stride * esz) % bytes == 0);
}

// How a row is spread: chunks of 256 columns, nv of them a warp; nv = 0: rows
// too wide to hold, a CTA to a row.
struct RowPlan {
  int nv, warps, rows_per_cta, threads;
};

constexpr int kHeldColumns = 8192;
constexpr int kSms = 152;  // a GB300's
constexpr int kGradShared = 226 * 1024;

RowPlan row_plan(int d, int nv, int warps) {
  if (d > kHeldColumns) return {0, WIDE_WARPS, 1, WIDE_WARPS * 32};
  RowPlan p;
  const int chunks = (d + 255) / 256;
  p.nv = std::min(nv, chunks >= 4 ? 4 : chunks >= 2 ? 2 : 1);
  p.warps = (chunks + p.nv - 1) / p.nv;
  p.rows_per_cta = std::max(1, warps / p.warps);
  p.threads = p.rows_per_cta * p.warps * 32;
  return p;
}

RowPlan norm_plan(int d) { return row_plan(d, 4, 4); }

// Gradient.  Aligned bf16 rows: two chunks a warp, as what a warp does once for
// a row (its sum, pointers, branches) costs a third of what it does for a chunk,
// and one CTA of 16 warps an SM, as each CTA writes a line of dgain's sums (608
// lines of four smaller CTAs an SM: 59.1 us instead of 57.6 at 15360 x 2048); few
// rows are spread over the SMs first.  Others: one chunk, so that 64 registers
// hold it.
RowPlan norm_grad_plan(int32_t M, int d, bool copied) {
  if (!copied) return row_plan(d, 1, 4);
  RowPlan p = row_plan(d, 2, 16);
  if (p.nv) {
    p.rows_per_cta = std::min({p.rows_per_cta, (M + kSms - 1) / kSms, 15});
    p.threads = p.rows_per_cta * p.warps * 32;
  }
  return p;
}

// CTAs go over the rows: as many as a GB300 holds.
int grad_grid(int32_t M, const RowPlan &p, bool copied) {
  const int64_t most = kSms * (p.nv == 0 ? 2 : copied ? 1 : std::max(1, 1024 / p.threads));
  return static_cast<int>(
      std::min<int64_t>((static_cast<int64_t>(M) + p.rows_per_cta - 1) / p.rows_per_cta, most));
}

template <bool F32, int L>
cudaError_t norm_launch_t(const NormArgs &a, cudaStream_t st) {
  const RowPlan p = norm_plan(a.d);
  const unsigned grid = (static_cast<int64_t>(a.M) + p.rows_per_cta - 1) / p.rows_per_cta;
  switch (p.nv) {
    case 0: return launch_overlapped(norm_wide_kernel<F32, L>, grid, p.threads, 0, st, a);
    case 1: return launch_overlapped(norm_kernel<F32, L, 1>, grid, p.threads, 0, st, a, p.warps);
    case 2: return launch_overlapped(norm_kernel<F32, L, 2>, grid, p.threads, 0, st, a, p.warps);
    default: return launch_overlapped(norm_kernel<F32, L, 4>, grid, p.threads, 0, st, a, p.warps);
  }
}

template <bool F32, int L>
cudaError_t norm_grad_launch_t(const NormGradArgs &a, cudaStream_t st) {
  constexpr bool COPIED = !F32 && L == kWide;
  const RowPlan p = norm_grad_plan(a.M, a.d, COPIED);
  const int grid = grad_grid(a.M, p, COPIED);
  const size_t line = static_cast<size_t>(a.d) * 4;
  const size_t sm = p.rows_per_cta > 1 ? line : 0;
  const auto most = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e;
  if (p.nv == 0) {
    const auto kernel = norm_grad_wide_kernel<F32, L>;
    e = cudaFuncSetAttribute(kernel, most, kMaxNormColumns * 4);
    if (e == cudaSuccess)
      e = launch_overlapped(kernel, grid, p.threads, a.dgain ? line : 0, st, a);
  } else if constexpr (COPIED) {
    const size_t part = static_cast<size_t>(p.threads) * 16 * p.nv;
    const size_t stage = 3 * part + static_cast<size_t>(p.threads) * 4;
    const auto kernel = p.nv == 1 ? norm_grad_kernel<1> : norm_grad_kernel<2>;
    e = cudaFuncSetAttribute(kernel, most, kGradShared);
    if (e == cudaSuccess)
      e = launch_overlapped(kernel, grid, p.threads, std::max((kAhead + 1) * stage + part, sm), st,
                            a, p.warps);
  } else {
    e = launch_overlapped(norm_grad_direct_kernel<F32, L>, grid, p.threads, sm, st, a, p.warps);
  }
  if (e != cudaSuccess || !a.dgain) return e;
  return launch_overlapped(dgain_kernel<F32>, (a.d + DGAIN_COLS - 1) / DGAIN_COLS,
                           DGAIN_WARPS * 32, 0, st,
                           static_cast<const float *>(a.partial), grid, a.d, a.dgain);
}

template <bool F32, int L>
cudaError_t dropout_launch_t(const DropoutArgs &a, cudaStream_t st) {
  const int chunks = (a.d + 255) / 256;
  const int rows = std::max(1, 16 / chunks);
  const unsigned grid = (static_cast<int64_t>(a.M) + rows - 1) / rows;
  return launch_overlapped(dropout_kernel<F32, L>, grid, 256, 0, st, a, rows, chunks);
}

dspark_status result(cudaError_t e) { return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA; }

}  // namespace

size_t norm_workspace_bytes(int32_t M, int32_t d) {
  // either kernel's lines
  const int lines =
      std::max(grad_grid(M, norm_grad_plan(M, d, true), true),
               grad_grid(M, norm_grad_plan(M, d, false), false));
  return kNormPartialOffset + static_cast<size_t>(lines) * d * 4;
}

template <class F>
Layout layout(int f32, int d, F rows_at_all) {
  if (d % 8 == 0 && rows_at_all(16)) return kWide;
  return !f32 && d % 2 == 0 && rows_at_all(4) ? kPairs : kSingle;
}

dspark_status norm_launch(const NormArgs &a, cudaStream_t st) {
  const int e = a.f32 ? 4 : 2;
  const Layout l = layout(a.f32, a.d, [&](int n) {
    return rows_at(a.x, a.x_stride, e, n) && rows_at(a.residual, a.residual_stride, e, n) &&
           rows_at(a.r, a.r_stride, e, n) && rows_at(a.gain, 0, e, n) &&
           (a.e4m3 ? rows_at(a.y, a.y_stride, 1, n / 2) : rows_at(a.y, a.y_stride, e, n));
  });
  if (a.f32)
    return result(l == kWide ? norm_launch_t<true, kWide>(a, st)
                             : norm_launch_t<true, kSingle>(a, st));
  return result(l == kWide    ? norm_launch_t<false, kWide>(a, st)
                : l == kPairs ? norm_launch_t<false, kPairs>(a, st)
                              : norm_launch_t<false, kShifted>(a, st));
}

dspark_status norm_grad_launch(const NormGradArgs &a, cudaStream_t st) {
  const int e = a.f32 ? 4 : 2;
  const Layout l = layout(a.f32, a.d, [&](int n) {
    return rows_at(a.dy, a.dy_stride, e, n) && rows_at(a.dr, a.dr_stride, e, n) &&
           rows_at(a.r, a.r_stride, e, n) && rows_at(a.gain, 0, e, n) &&
           rows_at(a.dx, a.dx_stride, e, n) && rows_at(a.dresidual, a.dresidual_stride, e, n);
  });
  if (a.f32)
    return result(l == kWide ? norm_grad_launch_t<true, kWide>(a, st)
                             : norm_grad_launch_t<true, kSingle>(a, st));
  return result(l == kWide    ? norm_grad_launch_t<false, kWide>(a, st)
                : l == kPairs ? norm_grad_launch_t<false, kPairs>(a, st)
                              : norm_grad_launch_t<false, kSingle>(a, st));
}

dspark_status dropout_launch(const DropoutArgs &a, cudaStream_t st) {
  const int e = a.f32 ? 4 : 2;
  const Layout l = layout(a.f32, a.d, [&](int n) {
    return rows_at(a.x, a.x_stride, e, n) && rows_at(a.residual, a.residual_stride, e, n) &&
           rows_at(a.y, a.y_stride, e, n);
  });
  if (a.f32)
    return result(l == kWide ? dropout_launch_t<true, kWide>(a, st)
                             : dropout_launch_t<true, kSingle>(a, st));
  return result(l == kWide    ? dropout_launch_t<false, kWide>(a, st)
                : l == kPairs ? dropout_launch_t<false, kPairs>(a, st)
                              : dropout_launch_t<false, kShifted>(a, st));
}

}  // namespace dspark
