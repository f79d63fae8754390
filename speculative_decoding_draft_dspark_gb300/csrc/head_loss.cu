// Softmax cross entropy of the Markov head's scores and its gradient.
//
//   A_i = [h_i, U[prev_i]]      B_v = [W_v, V_v]      z_iv = A_i . B_v
//   lse_i = log sum_v exp z_iv        loss_i = lse_i - z_{i, target_i}
//   G_iv = dloss_i (exp(z_iv - lse_i) - [v = target_i])
//   dA = G B      dB = G^T A      dU[t] = sum over prev_i = t of dA_i's tail
//
// The scores are never stored.  The loss keeps (maximum, sum) pairs for a row;
// the gradient computes z again for a piece of the vocabulary, writes that
// piece of G^T as bf16 and takes both products with it before the next piece.
// Only rows with a target are computed: they are gathered, in order, into a
// packed A first.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "chain_common.cuh"
#include "common.cuh"
#include "head_internal.h"
#include "launch.cuh"
#include "ptx_pair.cuh"

namespace dspark {

namespace {

constexpr int HT = 256;        // rows of a pair's tile, and its columns at most
constexpr int HU = 32;         // a tile's rows of A come in units of this
constexpr int HK = 64;         // reduction entries of a stage (128 bytes)
constexpr int H_STAGES = 6;
constexpr int H_BOX = 64 * 128;             // a 64 x 64 bf16 box
constexpr int H_OPERAND = 2 * H_BOX;        // a CTA's 128 rows of one operand
constexpr int H_STAGE = 2 * H_OPERAND;
constexpr int H_OUT_BOX = 32 * 128;         // a warp's 32 rows of 128 bytes at most
constexpr int H_OUT = 4 * 2 * H_OUT_BOX;    // four warps, two boxes each
constexpr int H_OUT_OFF = H_STAGES * H_STAGE;
constexpr int H_BAR_OFF = H_OUT_OFF + H_OUT;
constexpr int H_BARS = 2 * H_STAGES + 2 + 2 + 1;
constexpr int H_SMEM = H_BAR_OFF + H_BARS * 8 + 16 + 1024;
constexpr int H_THREADS = 256;
constexpr int kPairs = 76;                  // CTA pairs of a GB300: the layout is planned for it
constexpr uint32_t H_TMEM = 512;            // two accumulators of 256 columns
static_assert(H_SMEM <= 232448, "shared memory budget");

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// what a call keeps about its rows, at HeadLayout::rowinfo
struct RowInfo {
  int32_t *n_valid;   // rows that count
  float *scale;       // gradient: largest |dloss|
  int32_t *index;     // [rows_pad] the row's place in the caller's arrays
  int32_t *target;    // [rows_pad]
  int32_t *prev;      // [rows_pad]
  float *lse2;        // [rows_pad] gradient: lse log2 e
  float *weight;      // [rows_pad] gradient: dloss / scale
  float *z_target;    // [rows_pad] loss: z at the target
};

__host__ __device__ inline RowInfo row_info(uint8_t *at, int64_t rows_pad) {
  RowInfo r;
  r.n_valid = reinterpret_cast<int32_t *>(at);
  r.scale = reinterpret_cast<float *>(at + 4);
  int32_t *p = reinterpret_cast<int32_t *>(at + 256);
  r.index = p;
  r.target = p + rows_pad;
  r.prev = p + 2 * rows_pad;
  r.lse2 = reinterpret_cast<float *>(p + 3 * rows_pad);
  r.weight = reinterpret_cast<float *>(p + 4 * rows_pad);
  r.z_target = reinterpret_cast<float *>(p + 5 * rows_pad);
  return r;
}

// ------------------------------------------------------------------ pack
// Gathers the rows with a target into A = [h, U[prev]], zero-padded to whole
// 64-column blocks and 256-row tiles, and their row data.  A row that is
// ignored is never read, so what it holds (NaN, infinities) reaches nothing.
// Every CTA counts the targets before its rows itself: the target array is a
// few KB from L2, and a scan across CTAs would cost a second launch.
struct PackParams {
  const uint16_t *h;
  int64_t h_stride;
  const uint16_t *U;
  const int32_t *prev, *target;
  const float *lse, *dloss;
  float *loss_out, *lse_out;
  uint16_t *dh;       // gradient: rows without a target are zeroed here
  int64_t dh_stride;
  int32_t M, vocab, d, rank, cols_pad, d_pad, rows_per_cta;
  uint16_t *a;
  RowInfo rows;
  uint32_t *status;
};

constexpr int PACK_WARPS = 8;
constexpr int PACK_THREADS = PACK_WARPS * 32;
constexpr int PACK_ROWS = 256;  // at most, for one CTA

__device__ __forceinline__ bool counts(int32_t t, int32_t vocab) {
  return t >= 0 && t < vocab;
}

template <bool GRAD>
__global__ void __launch_bounds__(PACK_THREADS) head_pack_kernel(const PackParams p) {
  __shared__ int32_t s_before[PACK_WARPS], s_total[PACK_WARPS];
  __shared__ float s_max[PACK_WARPS];
  __shared__ uint32_t s_mask[PACK_ROWS / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = blockIdx.x * p.rows_per_cta;
  const int n = min(p.M - r0, p.rows_per_cta);
  allow_next_kernel();
  wait_for_earlier_kernel();

  // the CTA's own rows: which count (a bit each), and their first lines on
  // their way to L2 while the other targets are counted
  const int i = r0 + tid;
  const int32_t t = tid < n ? p.target[i] : -1;
  const bool ok = counts(t, p.vocab);
  const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok);
  if (lane == 0) s_mask[warp] = mask;
  for (int j = warp; j < n; j += PACK_WARPS) {
    const uint16_t *hr = p.h + static_cast<int64_t>(r0 + j) * p.h_stride;
    if (lane * 64 < p.d) asm volatile("prefetch.global.L2 [%0];" ::"l"(hr + lane * 64));
  }
  int before = 0, total = 0;
  float top = 0.0f;
#pragma unroll 4
  for (int k = tid; k < p.M; k += PACK_THREADS) {
    const bool c = counts(p.target[k], p.vocab);
    total += c;
    before += c && k < r0;
    if (GRAD && c) top = fmaxf(top, fabsf(p.dloss[k]));
  }
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  total = __reduce_add_sync(0xFFFFFFFFu, total);
  if (GRAD)
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (lane == 0) {
    s_before[warp] = before;
    s_total[warp] = total;
    s_max[warp] = top;
  }
  __syncthreads();
  before = total = 0;
  top = 0.0f;
#pragma unroll
  for (int w = 0; w < PACK_WARPS; ++w) {
    before += s_before[w];
    total += s_total[w];
    top = fmaxf(top, s_max[w]);
  }
  if (blockIdx.x == 0 && tid == 0) {
    *p.rows.n_valid = total;
    if (GRAD) *p.rows.scale = top;
  }

  const int chunks = p.cols_pad / 8;
  for (int j = warp; j < n; j += PACK_WARPS) {
    const int row = r0 + j;
    const uint32_t word = s_mask[j >> 5];
    if (!((word >> (j & 31)) & 1u)) {
      if (GRAD) {
        for (int c = lane * 8; c < p.d; c += 256)
          *reinterpret_cast<uint4 *>(p.dh + static_cast<int64_t>(row) * p.dh_stride + c) =
              make_uint4(0u, 0u, 0u, 0u);
      } else if (lane == 0) {
        p.loss_out[row] = 0.0f;
        p.lse_out[row] = 0.0f;
      }
      if (lane == 0 && p.target[row] >= p.vocab) raise_status(p.status, DSPARK_DEV_TOKEN_OOR);
      continue;
    }
    int at = before + __popc(word & ((1u << (j & 31)) - 1u));
    for (int w = 0; w < (j >> 5); ++w) at += __popc(s_mask[w]);
    int32_t pv = 0;
    if (p.rank > 0) {
      pv = p.prev[row];
      if (pv < 0 || pv >= p.vocab) {
        pv = 0;
        if (lane == 0) raise_status(p.status, DSPARK_DEV_TOKEN_OOR);
      }
    }
    if (lane == 0) {
      p.rows.index[at] = row;
      p.rows.target[at] = p.target[row];
      p.rows.prev[at] = pv;
      if (GRAD) {
        p.rows.lse2[at] = p.lse[row] * kLog2e;
        // equal weights (a mean) become exactly 1
        p.rows.weight[at] = top > 0.0f ? p.dloss[row] / top : p.dloss[row];
      }
    }
    const uint16_t *hr = p.h + static_cast<int64_t>(row) * p.h_stride;
    const uint16_t *ur = p.U + static_cast<int64_t>(pv) * p.rank;
    uint16_t *ar = p.a + static_cast<int64_t>(at) * p.cols_pad;
#pragma unroll 4
    for (int c = lane; c < chunks; c += 32) {
      const int col = c * 8;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (col < p.d)
        v = *reinterpret_cast<const uint4 *>(hr + col);
      else if (col >= p.d_pad && col - p.d_pad < p.rank)
        v = *reinterpret_cast<const uint4 *>(ur + (col - p.d_pad));
      *reinterpret_cast<uint4 *>(ar + col) = v;
    }
  }
  // the rows that fill up the last tile
  const int end = (total + HT - 1) / HT * HT;
  for (int j = total + blockIdx.x * PACK_WARPS + warp; j < end; j += gridDim.x * PACK_WARPS) {
    uint16_t *ar = p.a + static_cast<int64_t>(j) * p.cols_pad;
    for (int c = lane; c < chunks; c += 32)
      *reinterpret_cast<uint4 *>(ar + c * 8) = make_uint4(0u, 0u, 0u, 0u);
    if (lane == 0) {
      p.rows.target[j] = -1;
      p.rows.lse2[j] = 0.0f;
      p.rows.weight[j] = 0.0f;
    }
  }
}

// -------------------------------------------------------------- products
// Three kernels on one main loop.  A cluster of two CTAs computes a tile of
// 256 rows with tcgen05.mma.cta_group::2: each CTA stages 128 of them and half
// of the columns, 64 deep, and holds its 128 rows of the accumulator, so an
// operand byte is read from L2 once for 256 entries of the other one.
//
//   LSE    z^T tile, 256 vocabulary entries x up to 256 rows of A
//          -> per row of A (max, sum exp), and z at the target
//   PROB   z^T tile -> G^T, bf16
//   GRAD   dA^T tiles (256 columns of A x up to 256 rows; reduction over a
//          piece of the vocabulary, added up in fp32 by TMA) and dB tiles (256
//          vocabulary entries x 256 columns; reduction over the rows, bf16),
//          in one launch so that the ones fill the others' last wave
//
// The rows of A are always the tile's columns or the reduction: those come in
// steps of 32 and 16, where a tile's rows are always 256, so that 403 rows cost
// 416 and not 512.  Both operands of z^T and G^T in dB have the reduction index
// contiguous; for the others the 64 x 64 boxes are read as they lie, and the
// descriptors say that the other index is the contiguous one.
enum HeadKind { kLse = 0, kProb = 1, kGrad = 2 };

struct HeadMaps {
  CUtensorMap a;      // packed A, 64 x 64 boxes
  CUtensorMap w, v;   // W and V, 64 x 64 boxes
  CUtensorMap a_rows, w_rows, v_rows;  // the same, 128 rows x 64 boxes
  CUtensorMap g;      // G^T, 64 x 64 boxes
  CUtensorMap g_out;  // G^T, 32 x 32 boxes
  CUtensorMap dw, dv; // dW and dV, 32 rows x 64 boxes
  CUtensorMap acc;    // fp32 sums of dA^T, 32 x 32 boxes
};

struct HeadParams {
  RowInfo rows;
  int32_t rows_pad, cols_pad, vocab;
  int32_t kd, kr;       // 64-column blocks of d and of rank
  int32_t v0;           // first vocabulary entry of the piece
  int32_t v_tiles;      // 256-entry tiles of the piece
  int32_t d_tiles;      // 256-column tiles of A
  int32_t splits;
  int32_t first_piece;
  int32_t d, rank;
  float2 *partial;
  uint32_t *status;
};

struct HeadTile {
  int da;       // GRAD: a dA tile
  int m, n;     // first row and column of the output tile
  int cols;     // its columns
  int k0, nk;   // range of the reduction, in 64-entry blocks
  int split;
};

// The rows of A in tiles: units of 32, spread evenly over as few tiles of at
// most 256 as hold them.
__device__ __forceinline__ int row_tiles(int n_valid) { return (n_valid + HT - 1) / HT; }

__device__ __forceinline__ void row_tile(int n_valid, int i, int &first, int &count) {
  const int nt = row_tiles(n_valid), units = (n_valid + HU - 1) / HU;
  const int lo = static_cast<int>(static_cast<int64_t>(units) * i / nt);
  const int hi = static_cast<int>(static_cast<int64_t>(units) * (i + 1) / nt);
  first = lo * HU;
  count = (hi - lo) * HU;
}

template <int KIND>
__device__ __forceinline__ int head_tiles(const HeadParams &p, int n_valid) {
  const int nt = row_tiles(n_valid);
  if (KIND != kGrad) return nt * p.v_tiles;
  return nt * p.d_tiles * p.splits + p.v_tiles * p.d_tiles;
}

template <int KIND>
__device__ __forceinline__ HeadTile head_tile(const HeadParams &p, int n_valid, int t) {
  const int nt = row_tiles(n_valid);
  HeadTile x;
  x.da = 0;
  x.split = 0;
  if (KIND != kGrad) {
    x.m = (t / nt) * HT;
    row_tile(n_valid, t % nt, x.n, x.cols);
    x.k0 = 0;
    x.nk = p.kd + p.kr;
    return x;
  }
  const int n_da = nt * p.d_tiles * p.splits;
  if (t < n_da) {
    x.da = 1;
    x.m = (t % p.d_tiles) * HT;
    const int u = t / p.d_tiles;
    row_tile(n_valid, u % nt, x.n, x.cols);
    x.split = u / nt;
    const int kb = p.v_tiles * (HT / HK);
    x.k0 = static_cast<int>(static_cast<int64_t>(kb) * x.split / p.splits);
    x.nk = static_cast<int>(static_cast<int64_t>(kb) * (x.split + 1) / p.splits) - x.k0;
  } else {
    t -= n_da;
    x.n = (t % p.d_tiles) * HT;
    x.cols = HT;
    x.m = (t / p.d_tiles) * HT;
    x.k0 = 0;
    x.nk = (n_valid + HK - 1) / HK;
  }
  return x;
}

// K-major operand (the reduction index contiguous): common.cuh's descriptor.
// Otherwise the 128-byte rows run along the other index, 64 entries each; one
// row per reduction index, 8 rows (1024 bytes) an atom, atoms 1024 bytes apart
// along the reduction (bits 32-45) and a box apart along the other index
// (bits 16-29).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(H_BOX >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------- epilogues
// A warp has 32 rows of the accumulator, a lane one of them, 32 columns at a
// time.  What goes to memory is laid out in a box of shared memory (the
// swizzle of its tensor map) and stored by TMA; two boxes alternate.
__device__ __forceinline__ uint32_t next_box(uint32_t out, int &boxes, int lane) {
  if (lane == 0) bulk_wait_read<1>();  // the box's last store has read it
  __syncwarp();
  return out + (boxes++ & 1) * H_OUT_BOX;
}

// LSE: lanes are vocabulary entries, columns rows of A.  The 32 x 32 block is
// turned in shared memory, so that a lane has 32 entries of its own row of A
// and needs no other lane for their maximum and sum.
__device__ __forceinline__ void lse_tile(const HeadParams &p, const HeadTile &x, uint32_t acc_at,
                                         int v_first, float2 *slot, uint32_t out, int lane) {
  const bool beyond = v_first + lane >= p.vocab;
  for (int c0 = 0; c0 < x.cols; c0 += 32) {
    const int row = x.n + c0 + lane;
    const float2 old = slot[row];
    const int at = p.rows.target[row] - v_first;
    uint32_t acc[32];
    tmem_ld_32x32b_x32(acc_at + c0, acc);
    tmem_ld_wait(acc);
    if (beyond) {
#pragma unroll
      for (int e = 0; e < 32; ++e) acc[e] = 0xFF800000u;  // -infinity
    }
    const uint32_t box = out + ((c0 >> 5) & 1) * H_OUT_BOX;
#pragma unroll
    for (int c = 0; c < 8; ++c)
      st_shared_v4(box + lane * 128 + ((c ^ (lane & 7)) << 4),
                   make_uint4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]));
    __syncwarp();
    float z[32];
#pragma unroll
    for (int v = 0; v < 32; ++v) {
      uint32_t w;
      asm volatile("ld.shared.u32 %0, [%1];"
                   : "=r"(w)
                   : "r"(box + v * 128 + (((lane >> 2) ^ (v & 7)) << 4) + (lane & 3) * 4));
      z[v] = __uint_as_float(w);
    }
    if (static_cast<uint32_t>(at) < 32u) {
      float zt = 0.0f;
#pragma unroll
      for (int v = 0; v < 32; ++v) zt = v == at ? z[v] : zt;
      p.rows.z_target[row] = zt;
    }
    float top = old.x;
#pragma unroll
    for (int v = 0; v < 32; ++v) top = fmaxf(top, z[v]);
    // a row of -infinity keeps a finite reference: its sum is 0
    const float ref = top == -INFINITY ? 0.0f : top * kLog2e;
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < 32; ++v) part[v & 3] += ex2(fmaf(z[v], kLog2e, -ref));
    const float sum =
        fmaf(old.y, ex2(fmaf(old.x, kLog2e, -ref)), (part[0] + part[1]) + (part[2] + part[3]));
    slot[row] = make_float2(top, sum);
  }
}

// PROB: lanes are vocabulary entries, columns rows of A.
__device__ __forceinline__ void prob_tile(const HeadParams &p, const CUtensorMap &g_out,
                                          const HeadTile &x, uint32_t acc_at, int row0,
                                          uint32_t out, int &boxes, int lane) {
  const int v_first = p.v0 + row0;
  const bool beyond = v_first + lane >= p.vocab;
  for (int c0 = 0; c0 < x.cols; c0 += 32) {
    const float4 *lse2 = reinterpret_cast<const float4 *>(p.rows.lse2 + x.n + c0);
    const float4 *weight = reinterpret_cast<const float4 *>(p.rows.weight + x.n + c0);
    const int at = p.rows.target[x.n + c0 + lane] - v_first;
    uint32_t hits = __ballot_sync(0xFFFFFFFFu, static_cast<uint32_t>(at) < 32u);
    uint32_t acc[32];
    tmem_ld_32x32b_x32(acc_at + c0, acc);
    tmem_ld_wait(acc);
    float g[32];
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const float4 l = lse2[e / 4], w = weight[e / 4];
      g[e] = ex2(fmaf(__uint_as_float(acc[e]), kLog2e, -l.x)) * w.x;
      g[e + 1] = ex2(fmaf(__uint_as_float(acc[e + 1]), kLog2e, -l.y)) * w.y;
      g[e + 2] = ex2(fmaf(__uint_as_float(acc[e + 2]), kLog2e, -l.z)) * w.z;
      g[e + 3] = ex2(fmaf(__uint_as_float(acc[e + 3]), kLog2e, -l.w)) * w.w;
    }
    if (hits) {
      const float own = p.rows.weight[x.n + c0 + lane];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int v = __shfl_sync(0xFFFFFFFFu, at, e);
        const float w = __shfl_sync(0xFFFFFFFFu, own, e);
        if (v == lane) g[e] -= w;
      }
    }
    if (beyond) {
#pragma unroll
      for (int e = 0; e < 32; ++e) g[e] = 0.0f;
    }
    const uint32_t box = next_box(out, boxes, lane);
    // rows of 64 bytes, 64-byte swizzle
#pragma unroll
    for (int c = 0; c < 4; ++c)
      st_shared_v4(box + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4),
                   make_uint4(pack_bf16(g[8 * c], g[8 * c + 1]),
                              pack_bf16(g[8 * c + 2], g[8 * c + 3]),
                              pack_bf16(g[8 * c + 4], g[8 * c + 5]),
                              pack_bf16(g[8 * c + 6], g[8 * c + 7])));
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&g_out, box, x.n + c0, row0);
      bulk_commit();
    }
  }
}

// dA^T: lanes are columns of A, columns its rows; fp32, one addition a piece.
__device__ __forceinline__ void sum_tile(const HeadParams &p, const CUtensorMap &acc_map,
                                         const HeadTile &x, uint32_t acc_at, int row0,
                                         uint32_t out, int &boxes, int lane) {
  if (row0 >= p.cols_pad) return;
  for (int c0 = 0; c0 < x.cols; c0 += 32) {
    uint32_t acc[32];
    if (x.nk > 0) {
      tmem_ld_32x32b_x32(acc_at + c0, acc);
      tmem_ld_wait(acc);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) acc[e] = 0u;
    }
    const uint32_t box = next_box(out, boxes, lane);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      st_shared_v4(box + lane * 128 + ((c ^ (lane & 7)) << 4),
                   make_uint4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]));
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      const int y = x.split * p.cols_pad + row0;
      if (p.first_piece)
        tma_store_2d(&acc_map, box, x.n + c0, y);
      else
        tma_reduce_add_2d(&acc_map, box, x.n + c0, y);
      bulk_commit();
    }
  }
}

// dB: lanes are vocabulary entries, columns those of [W, V].
__device__ __forceinline__ void weight_tile(const HeadParams &p, const HeadMaps &maps,
                                            const HeadTile &x, uint32_t acc_at, int row0,
                                            uint32_t out, int &boxes, int lane) {
  if (p.v0 + row0 >= p.vocab) return;
  const float scale = *p.rows.scale;
  for (int c0 = 0; c0 < x.cols; c0 += 64) {
    const int col = x.n + c0;
    const bool in_d = col < p.kd * HK;
    const int left = in_d ? p.d - col : p.rank - (col - p.kd * HK);
    if (left <= 0) continue;
    const uint32_t box = next_box(out, boxes, lane);
#pragma unroll
    for (int half = 0; half < 64; half += 32) {
      uint32_t acc[32];
      if (x.nk > 0) {
        tmem_ld_32x32b_x32(acc_at + c0 + half, acc);
        tmem_ld_wait(acc);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] = 0u;
      }
      float g[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) g[e] = __uint_as_float(acc[e]) * scale;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        st_shared_v4(box + lane * 128 + (((half / 8 + c) ^ (lane & 7)) << 4),
                     make_uint4(pack_bf16(g[8 * c], g[8 * c + 1]),
                                pack_bf16(g[8 * c + 2], g[8 * c + 3]),
                                pack_bf16(g[8 * c + 4], g[8 * c + 5]),
                                pack_bf16(g[8 * c + 6], g[8 * c + 7])));
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (in_d)
        tma_store_2d(&maps.dw, box, col, p.v0 + row0);
      else
        tma_store_2d(&maps.dv, box, col - p.kd * HK, p.v0 + row0);
      bulk_commit();
    }
  }
}

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(H_THREADS, 1)
    head_gemm_kernel(const __grid_constant__ HeadMaps maps, const HeadParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t *smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + H_BAR_OFF);
  uint64_t *empty = full + H_STAGES;
  uint64_t *acc_full = empty + H_STAGES;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *mma_done = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(full + H_BARS);
  volatile uint32_t *abort_flag = tmem_slot + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < H_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8);  // four epilogue warps of either CTA
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0u;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, H_TMEM);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  allow_next_kernel();
  wait_for_earlier_kernel();
  const uint32_t tmem_base = *tmem_slot;
  const int n_valid = *p.rows.n_valid;
  const int tiles = head_tiles<KIND>(p, n_valid);

  if (warp == 0) {
    // ---------------------------------------------------------- loads
    if (lane == 0) {
      const uint32_t full0 = mapa_u32(smem_u32(full), 0);
      bool ok = true;
      int it = 0;
      for (int t = pair; t < tiles && ok; t += pairs) {
        const HeadTile x = head_tile<KIND>(p, n_valid, t);
        for (int kb = x.k0; kb < x.k0 + x.nk; ++kb, ++it) {
          const int s = it % H_STAGES;
          if (!(ok = wait_bounded(&empty[s], ((it / H_STAGES) & 1) ^ 1u, abort_flag, p.status)))
            break;
          const uint32_t bar = full0 + s * 8;
          uint8_t *sa = smem + s * H_STAGE, *sb = sa + H_OPERAND;
          if (KIND != kGrad) {
            // whole 64-row boxes, also for fewer rows: 16-row boxes, eight a
            // stage, took 1.6 times as long (2080 us against 1289 us at 1613 rows)
            const int slabs = (x.cols / 2 + 63) / 64;
            if (cta == 0) mbar_arrive_expect_tx(&full[s], 2 * (H_OPERAND + slabs * H_BOX));
            const bool in_d = kb < p.kd;
            tma_load_2d_pair(sa, in_d ? &maps.w_rows : &maps.v_rows, bar,
                             (in_d ? kb : kb - p.kd) * HK, p.v0 + x.m + cta * 128);
            tma_load_2d_pair(sb, slabs == 2 ? &maps.a_rows : &maps.a, bar, kb * HK,
                             x.n + cta * (x.cols / 2));
          } else if (x.da) {
            const int slabs = (x.cols / 2 + 63) / 64;
            if (cta == 0) mbar_arrive_expect_tx(&full[s], 2 * (H_OPERAND + slabs * H_BOX));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int cb = (x.m + cta * 128) / HK + j;
              const bool in_d = cb < p.kd || p.kr == 0;
              tma_load_2d_pair(sa + j * H_BOX, in_d ? &maps.w : &maps.v, bar,
                               (in_d ? cb : cb - p.kd) * HK, p.v0 + kb * HK);
            }
            for (int j = 0; j < slabs; ++j)
              tma_load_2d_pair(sb + j * H_BOX, &maps.g, bar, x.n + cta * (x.cols / 2) + j * 64,
                               kb * HK);
          } else {
            if (cta == 0) mbar_arrive_expect_tx(&full[s], 2 * H_STAGE);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int r = cta * 128 + j * 64;
              tma_load_2d_pair(sa + j * H_BOX, &maps.g, bar, kb * HK, x.m + r);
              tma_load_2d_pair(sb + j * H_BOX, &maps.a, bar, x.n + r, kb * HK);
            }
          }
        }
      }
      if (!ok) {
        // copies in flight land before the shared memory is given back
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 20000000ull) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (cta == 0 && lane == 0) {
      const uint32_t base = smem_u32(smem);
      bool ok = true;
      int it = 0, ig = 0;
      for (int t = pair; t < tiles && ok; t += pairs) {
        const HeadTile x = head_tile<KIND>(p, n_valid, t);
        if (x.nk == 0) continue;
        const bool a_mn = KIND == kGrad && x.da, b_mn = KIND == kGrad;
        const uint32_t idesc = umma_idesc_bf16_f32(HT, static_cast<uint32_t>(x.cols)) |
                               (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
        const int buf = ig & 1;
        if (!(ok = wait_bounded(&acc_empty[buf], ((ig >> 1) & 1) ^ 1u, abort_flag, p.status)))
          break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * HT);
        for (int kb = 0; kb < x.nk; ++kb, ++it) {
          const int s = it % H_STAGES;
          if (!(ok = wait_bounded(&full[s], (it / H_STAGES) & 1, abort_flag, p.status))) break;
          tc_fence_after();
          const uint32_t sa = base + s * H_STAGE, sb = sa + H_OPERAND;
          // dB's reduction ends with the rows: no 16 of them are multiplied
          // that hold none (nor were written)
          const int steps = KIND == kGrad && !x.da
                                ? min(HK / 16, (n_valid - kb * HK + 15) / 16)
                                : HK / 16;
#pragma unroll
          for (int kk = 0; kk < HK / 16; ++kk) {
            if (kk >= steps) break;
            const uint64_t ad = a_mn ? sw128_mnmajor_desc(sa + kk * 2048)
                                     : sw128_kmajor_desc(sa + kk * 32);
            const uint64_t bd = b_mn ? sw128_mnmajor_desc(sb + kk * 2048)
                                     : sw128_kmajor_desc(sb + kk * 32);
            umma_bf16_pair(d_tmem, ad, bd, idesc, (kb | kk) != 0 ? 1u : 0u);
          }
          umma_commit_pair(&empty[s]);
        }
        if (!ok) break;
        umma_commit_pair(&acc_full[buf]);
        ++ig;
      }
      umma_commit_pair(mma_done);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------- epilogue
    const int q = warp & 3;
    const uint32_t acc_empty0 = mapa_u32(smem_u32(acc_empty), 0);
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    uint8_t *out = smem + H_OUT_OFF + q * 2 * H_OUT_BOX;
    const uint32_t out_addr = smem_u32(out);
    int ig = 0, boxes = 0;
    bool ok = true;
    float2 *slot = nullptr;
    if (KIND == kLse) {
      // the warp's own running pairs, one for a row of A
      slot = p.partial + static_cast<int64_t>(blockIdx.x * 4 + q) * p.rows_pad;
      for (int i = lane; i < (n_valid + HU - 1) / HU * HU; i += 32)
        slot[i] = make_float2(-INFINITY, 0.0f);
    }
    for (int t = pair; t < tiles && ok; t += pairs) {
      const HeadTile x = head_tile<KIND>(p, n_valid, t);
      const int buf = ig & 1;
      if (x.nk > 0) {
        ok = __all_sync(0xFFFFFFFFu,
                        wait_bounded(&acc_full[buf], (ig >> 1) & 1, abort_flag, p.status));
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t acc_at = lane_base + static_cast<uint32_t>(buf * HT);
      const int row0 = x.m + cta * 128 + q * 32;  // the warp's first output row
      if (KIND == kLse) {
        lse_tile(p, x, acc_at, p.v0 + row0, slot, out_addr, lane);
      } else if (KIND == kProb) {
        prob_tile(p, maps.g_out, x, acc_at, row0, out_addr, boxes, lane);
      } else if (x.da) {
        sum_tile(p, maps.acc, x, acc_at, row0, out_addr, boxes, lane);
      } else {
        weight_tile(p, maps, x, acc_at, row0, out_addr, boxes, lane);
      }
      if (x.nk > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty0 + buf * 8);
        ++ig;
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  // the last commit's arrival has reached this CTA before either one leaves
  if (threadIdx.x == 32) drain_wait(mma_done, 0, p.status);
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, H_TMEM);
}

// --------------------------------------------------------------- joining
// Joins the (max, sum) pairs of a row: a warp reads 32 neighbouring rows of
// one slot, 32 warps share the slots.
constexpr int JOIN_WARPS = 32;

__global__ void __launch_bounds__(JOIN_WARPS * 32)
    head_join_kernel(const float2 *partial, int slots, int rows_pad, RowInfo rows,
                     float *loss, float *lse) {
  allow_next_kernel();
  wait_for_earlier_kernel();
  __shared__ float2 part[JOIN_WARPS][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * 32 + lane;
  const int n_valid = *rows.n_valid;
  if (blockIdx.x * 32 >= n_valid) return;
  float m = -INFINITY, s = 0.0f;
  constexpr int U = 8;
  for (int v = warp; v < slots; v += JOIN_WARPS * U) {
    float2 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = v + u * JOIN_WARPS;
      x[u] = at < slots && row < n_valid
                 ? partial[static_cast<int64_t>(at) * rows_pad + row]
                 : make_float2(-INFINITY, 0.0f);
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, x[u].x);
    const float ref = top == -INFINITY ? 0.0f : top * kLog2e;
    s *= ex2(fmaf(m, kLog2e, -ref));
#pragma unroll
    for (int u = 0; u < U; ++u) s += x[u].y * ex2(fmaf(x[u].x, kLog2e, -ref));
    m = top;
  }
  part[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp == 0) {
    float top = -INFINITY;
    for (int w = 0; w < JOIN_WARPS; ++w) top = fmaxf(top, part[w][lane].x);
    const float ref = top == -INFINITY ? 0.0f : top * kLog2e;
    float sum = 0.0f;
    for (int w = 0; w < JOIN_WARPS; ++w)
      sum += part[w][lane].y * ex2(fmaf(part[w][lane].x, kLog2e, -ref));
    if (row < n_valid) {
      const int i = rows.index[row];
      const float l = fmaf(log2f(sum), kLn2, top);
      lse[i] = l;
      loss[i] = l - rows.z_target[row];
    }
  }
}

// ------------------------------------------------------- dh and dU, at last
// The splits' sums of dA^T in order, times the scale, turned: d columns go to
// dh at the row's own place, the rank's to dE (fp32, packed rows) for dU.  A
// CTA turns 64 columns of 32 rows.
constexpr int TURN_COLS = 64;

__global__ void __launch_bounds__(256)
    head_turn_kernel(const float *acc, int splits, int rows_pad, int cols_pad, int d_pad, int d,
                     int rank, RowInfo rows, uint16_t *dh, int64_t dh_stride, float *de) {
  allow_next_kernel();
  wait_for_earlier_kernel();
  __shared__ float block[32][TURN_COLS + 1];
  const int n_valid = *rows.n_valid;
  const int r0 = blockIdx.y * 32, c0 = blockIdx.x * TURN_COLS;
  if (r0 >= n_valid) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float scale = *rows.scale;
#pragma unroll
  for (int c = warp; c < TURN_COLS; c += 8) {
    const float *x = acc + static_cast<int64_t>(c0 + c) * rows_pad + r0 + lane;
    float s = 0.0f;
    for (int k = 0; k < splits; ++k) s += x[static_cast<int64_t>(k) * cols_pad * rows_pad];
    block[lane][c] = s * scale;
  }
  __syncthreads();
  const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 8;
  if (r0 + r >= n_valid) return;
  const float *s = &block[r][c];
  if (c0 < d_pad) {
    if (c0 + c < d)
      *reinterpret_cast<uint4 *>(dh + static_cast<int64_t>(rows.index[r0 + r]) * dh_stride + c0 +
                                 c) = make_uint4(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]),
                                                 pack_bf16(s[4], s[5]), pack_bf16(s[6], s[7]));
  } else if (c0 - d_pad + c < rank) {
    float4 *o = reinterpret_cast<float4 *>(de + static_cast<int64_t>(r0 + r) * rank + c0 - d_pad +
                                           c);
    o[0] = make_float4(s[0], s[1], s[2], s[3]);
    o[1] = make_float4(s[4], s[5], s[6], s[7]);
  }
}

// dU: one CTA for a counted row.  The first row with a token sums that token's
// rows in a fixed order (eight warps take consecutive eighths of the rows, and
// their sums are joined in order), so the result does not depend on the order
// in which CTAs run.  Tokens that no row names were zeroed before.
constexpr int DU_WARPS = 8;

__global__ void __launch_bounds__(DU_WARPS * 32)
    head_du_kernel(const float *de, RowInfo rows, int rank, uint16_t *dU) {
  allow_next_kernel();
  wait_for_earlier_kernel();
  __shared__ float part[DU_WARPS][32][9];
  const int n_valid = *rows.n_valid;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j = blockIdx.x; j < n_valid; j += gridDim.x) {
    const int token = rows.prev[j];
    bool seen = false;
    for (int i = threadIdx.x; i < j && !seen; i += DU_WARPS * 32) seen = rows.prev[i] == token;
    if (__syncthreads_or(seen)) continue;
    const int n = n_valid - j;
    const int lo = j + static_cast<int>(static_cast<int64_t>(n) * warp / DU_WARPS);
    const int hi = j + static_cast<int>(static_cast<int64_t>(n) * (warp + 1) / DU_WARPS);
    float s[8] = {};
    for (int base = lo; base < hi; base += 32) {
      uint32_t hit = __ballot_sync(0xFFFFFFFFu,
                                   base + lane < hi && rows.prev[base + lane] == token);
      while (hit) {
        const int i = base + __ffs(hit) - 1;
        hit &= hit - 1;
        if (lane * 8 < rank) {
          const float *x = de + static_cast<int64_t>(i) * rank + lane * 8;
          const float4 a = *reinterpret_cast<const float4 *>(x);
          const float4 b = *reinterpret_cast<const float4 *>(x + 4);
          s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
          s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) part[warp][lane][e] = s[e];
    __syncthreads();
    if (warp == 0 && lane * 8 < rank) {
      float r[8] = {};
      for (int w = 0; w < DU_WARPS; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] += part[w][lane][e];
      *reinterpret_cast<uint4 *>(dU + static_cast<int64_t>(token) * rank + lane * 8) =
          make_uint4(pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3]), pack_bf16(r[4], r[5]),
                     pack_bf16(r[6], r[7]));
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host
int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

std::mutex g_head_mu;
bool g_head_attr[128];

bool encode_2d(CUtensorMap *m, CUtensorMapDataType type, int esz, const void *base, int64_t cols,
               int64_t rows, int64_t pitch, int box_cols, int box_rows) {
  // the swizzle is as wide as the box's rows
  const auto swizzle =
      box_cols * esz == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  EncodeTiledFn enc = encode_tiled_fn();
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * esz};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1, 1};
  return enc(m, type, 2, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct HeadPlan {
  HeadLayout lay;
  HeadMaps maps;
  HeadParams p;
  PackParams pack;
  int sms, pack_grid;
};

dspark_status head_plan(const HeadArgs &a, bool grad, HeadPlan &o) {
  if (!encode_tiled_fn()) return DSPARK_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return DSPARK_ERR_CUDA;
  o.sms = device_sm_count(dev);
  if (o.sms <= 0) return DSPARK_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lk(g_head_mu);
    if (!g_head_attr[dev]) {
      const auto at = cudaFuncAttributeMaxDynamicSharedMemorySize;
      if (cudaFuncSetAttribute(head_gemm_kernel<kLse>, at, H_SMEM) != cudaSuccess ||
          cudaFuncSetAttribute(head_gemm_kernel<kProb>, at, H_SMEM) != cudaSuccess ||
          cudaFuncSetAttribute(head_gemm_kernel<kGrad>, at, H_SMEM) != cudaSuccess)
        return DSPARK_ERR_CUDA;
      g_head_attr[dev] = true;
    }
  }
  const HeadLayout &l = o.lay = head_layout(a.M, a.vocab, a.d, a.rank, grad);
  uint8_t *ws = a.workspace;
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int64_t vr = a.rank ? a.rank : a.d;
  const void *V = a.rank ? a.V : a.W;
  const void *A = ws + l.a;
  bool ok = encode_2d(&o.maps.a, bf16, 2, A, l.cols_pad, l.rows_pad, l.cols_pad, 64, 64) &&
            encode_2d(&o.maps.w, bf16, 2, a.W, a.d, a.vocab, a.d, 64, 64) &&
            encode_2d(&o.maps.v, bf16, 2, V, vr, a.vocab, vr, 64, 64) &&
            encode_2d(&o.maps.a_rows, bf16, 2, A, l.cols_pad, l.rows_pad, l.cols_pad, 64, 128) &&
            encode_2d(&o.maps.w_rows, bf16, 2, a.W, a.d, a.vocab, a.d, 64, 128) &&
            encode_2d(&o.maps.v_rows, bf16, 2, V, vr, a.vocab, vr, 64, 128);
  if (grad) {
    ok = ok && encode_2d(&o.maps.g, bf16, 2, ws + l.g, l.rows_pad, l.piece, l.rows_pad, 64, 64) &&
         encode_2d(&o.maps.g_out, bf16, 2, ws + l.g, l.rows_pad, l.piece, l.rows_pad, 32, 32) &&
         encode_2d(&o.maps.dw, bf16, 2, a.dW, a.d, a.vocab, a.d, 64, 32) &&
         encode_2d(&o.maps.dv, bf16, 2, a.rank ? a.dV : a.dW, vr, a.vocab, vr, 64, 32) &&
         encode_2d(&o.maps.acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, ws + l.acc, l.rows_pad,
                   l.cols_pad * l.splits, l.rows_pad, 32, 32);
  }
  if (!ok) return DSPARK_ERR_INVALID_ARG;

  HeadParams &p = o.p;
  p.rows = row_info(ws + l.rowinfo, l.rows_pad);
  p.rows_pad = static_cast<int32_t>(l.rows_pad);
  p.cols_pad = static_cast<int32_t>(l.cols_pad);
  p.vocab = a.vocab;
  p.kd = (a.d + HK - 1) / HK;
  p.kr = (a.rank + HK - 1) / HK;
  p.d_tiles = static_cast<int32_t>((l.cols_pad + HT - 1) / HT);
  p.splits = l.splits;
  p.v0 = 0;
  p.v_tiles = (a.vocab + HT - 1) / HT;
  p.first_piece = 0;
  p.d = a.d;
  p.rank = a.rank;
  p.partial = reinterpret_cast<float2 *>(ws + l.partial);
  p.status = reinterpret_cast<uint32_t *>(ws + kStatusOffset);

  PackParams &k = o.pack;
  k.h = static_cast<const uint16_t *>(a.h);
  k.h_stride = a.h_stride;
  k.U = static_cast<const uint16_t *>(a.U);
  k.prev = a.prev;
  k.target = a.target;
  k.lse = a.lse;
  k.dloss = a.dloss;
  k.loss_out = a.loss;
  k.lse_out = a.lse;
  k.M = a.M;
  k.vocab = a.vocab;
  k.d = a.d;
  k.rank = a.rank;
  k.cols_pad = static_cast<int32_t>(l.cols_pad);
  k.d_pad = p.kd * HK;
  k.rows_per_cta = static_cast<int>(
      std::min<int64_t>(PACK_ROWS, up((a.M + o.sms * 8 - 1) / (o.sms * 8), PACK_WARPS)));
  k.dh = static_cast<uint16_t *>(a.dh);
  k.dh_stride = a.dh_stride;
  k.a = reinterpret_cast<uint16_t *>(ws + l.a);
  k.rows = p.rows;
  k.status = p.status;
  o.pack_grid = (a.M + k.rows_per_cta - 1) / k.rows_per_cta;
  return DSPARK_OK;
}

// no more pairs than there can be tiles
template <int KIND>
int head_pairs(const HeadPlan &o, const HeadParams &p) {
  const int64_t nt = o.lay.rows_pad / HT;
  const int64_t tiles = KIND == kGrad ? nt * p.d_tiles * p.splits + int64_t(p.v_tiles) * p.d_tiles
                                      : nt * p.v_tiles;
  return static_cast<int>(std::min<int64_t>(std::min(o.sms / 2, kPairs), tiles));
}

template <int KIND>
cudaError_t head_gemm(const HeadPlan &o, const HeadParams &p, cudaStream_t stream) {
  return launch_overlapped(head_gemm_kernel<KIND>, head_pairs<KIND>(o, p) * 2, H_THREADS, H_SMEM,
                           stream, o.maps, p);
}

}  // namespace

HeadLayout head_layout(int32_t M, int32_t vocab, int32_t d, int32_t rank, bool grad) {
  HeadLayout l = {};
  l.rows_pad = up(M, HT);
  l.cols_pad = up(d, HK) + up(rank, HK);
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = static_cast<size_t>(up(static_cast<int64_t>(at + bytes), 1024));
    return here;
  };
  at = 1024;
  l.rowinfo = take(256 + static_cast<size_t>(l.rows_pad) * 4 * 6);
  l.a = take(static_cast<size_t>(l.rows_pad) * l.cols_pad * 2);
  const int64_t v_pad = up(vocab, HT);
  l.splits = 1;
  if (!grad) {
    const int64_t pairs = std::min<int64_t>(kPairs, l.rows_pad / HT * (v_pad / HT));
    l.partial = take(static_cast<size_t>(pairs) * 8 * l.rows_pad * 8);
  } else {
    constexpr int64_t kPieceBytes = 192ll << 20;
    const int64_t most = std::max<int64_t>(4096, kPieceBytes / (2 * l.rows_pad) / HT * HT);
    const int64_t pieces = (v_pad + most - 1) / most;
    l.piece = up((v_pad + pieces - 1) / pieces, HT);
    const int64_t tiles = l.rows_pad / HT * ((l.cols_pad + HT - 1) / HT);
    const int64_t deep = l.piece / HK;  // 64-entry blocks of the reduction
    l.splits = static_cast<int32_t>(
        std::max<int64_t>(1, std::min<int64_t>({kPairs / tiles, deep / 8, 16})));
    l.g = take(static_cast<size_t>(l.rows_pad) * l.piece * 2);
    l.acc = take(static_cast<size_t>(l.splits) * l.rows_pad * l.cols_pad * 4);
    l.de = take(static_cast<size_t>(l.rows_pad) * rank * 4);
  }
  l.total = at;
  return l;
}

dspark_status head_loss_launch(const HeadArgs &a, cudaStream_t stream) {
  HeadPlan o;
  const dspark_status s = head_plan(a, false, o);
  if (s != DSPARK_OK) return s;
  cudaError_t e =
      launch_overlapped(head_pack_kernel<false>, o.pack_grid, PACK_THREADS, 0, stream, o.pack);
  if (e == cudaSuccess) e = head_gemm<kLse>(o, o.p, stream);
  if (e == cudaSuccess)
    e = launch_overlapped(head_join_kernel, (a.M + 31) / 32, JOIN_WARPS * 32, 0, stream,
                          static_cast<const float2 *>(o.p.partial), head_pairs<kLse>(o, o.p) * 8,
                          o.p.rows_pad, o.p.rows, a.loss, a.lse);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

dspark_status head_loss_grad_launch(const HeadArgs &a, cudaStream_t stream) {
  HeadPlan o;
  const dspark_status s = head_plan(a, true, o);
  if (s != DSPARK_OK) return s;
  const HeadLayout &l = o.lay;
  cudaError_t e = cudaSuccess;
  if (a.rank) e = cudaMemsetAsync(a.dU, 0, static_cast<size_t>(a.vocab) * a.rank * 2, stream);
  if (e == cudaSuccess)
    e = launch_overlapped(head_pack_kernel<true>, o.pack_grid, PACK_THREADS, 0, stream, o.pack);
  HeadParams p = o.p;
  for (int64_t v0 = 0; v0 < a.vocab && e == cudaSuccess; v0 += l.piece) {
    p.v0 = static_cast<int32_t>(v0);
    p.v_tiles = static_cast<int32_t>((std::min<int64_t>(l.piece, a.vocab - v0) + HT - 1) / HT);
    p.first_piece = v0 == 0;
    e = head_gemm<kProb>(o, p, stream);
    if (e == cudaSuccess) e = head_gemm<kGrad>(o, p, stream);
  }
  const float *acc = reinterpret_cast<const float *>(a.workspace + l.acc);
  float *de = reinterpret_cast<float *>(a.workspace + l.de);
  const dim3 turn(static_cast<unsigned>(l.cols_pad / TURN_COLS), (a.M + 31) / 32);
  if (e == cudaSuccess)
    e = launch_overlapped(head_turn_kernel, turn, 256, 0, stream, acc, l.splits, p.rows_pad,
                          p.cols_pad, o.pack.d_pad, a.d, a.rank, p.rows,
                          static_cast<uint16_t *>(a.dh), a.dh_stride, de);
  if (e == cudaSuccess && a.rank)
    e = launch_overlapped(head_du_kernel, std::min(a.M, o.sms * 32), DU_WARPS * 32, 0, stream,
                          static_cast<const float *>(de), p.rows, a.rank,
                          static_cast<uint16_t *>(a.dU));
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // namespace dspark
