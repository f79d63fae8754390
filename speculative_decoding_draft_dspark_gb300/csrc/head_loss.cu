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

constexpr int HT = 256;        // rows of a pair's tile
constexpr int HW = 512;        // its columns at most, in two halves
constexpr int HU = 32;         // a tile's rows of A come in units of this
constexpr int HK = 64;         // reduction entries of a stage (128 bytes)
constexpr int H_BOX = 64 * 128;             // a 64 x 64 bf16 box
constexpr int H_OPERAND = 2 * H_BOX;        // 128 rows of an operand
constexpr int H_RING = 12 * H_OPERAND;      // 8 stages of 24 KB, 6 of 32 or 4 of 48
constexpr int H_MAX_STAGES = 8;
constexpr int H_EPI_WARPS = 8;
constexpr int H_OUT_BOX = 32 * 128;         // a warp's 32 rows of 128 bytes at most
constexpr int H_BAR_OFF = H_RING + H_EPI_WARPS * H_OUT_BOX;
constexpr int H_BARS = 2 * H_MAX_STAGES + 2 + 2 + 1;
constexpr int H_SMEM = H_BAR_OFF + H_BARS * 8 + 16 + 1024;
constexpr int H_THREADS = (4 + H_EPI_WARPS) * 32;
constexpr int kPairs = 76;                  // CTA pairs of a GB300: the layout is planned for it
// LSE and PROB: registers of an epilogue thread and of the others.  What the ones
// gain the others have given up: no more in all than the launch's 168 a thread, which
// the host checks before the first launch.
constexpr int H_REGS = 168, H_Z_EPI_REGS = 216, H_Z_OTHER_REGS = 72;
static_assert(H_EPI_WARPS * H_Z_EPI_REGS + 4 * H_Z_OTHER_REGS <= (4 + H_EPI_WARPS) * H_REGS,
              "registers of a launch");
constexpr uint32_t H_TMEM = 512;            // two accumulators of 256 columns
static_assert(H_SMEM <= 232448, "shared memory limit");

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// what a call keeps about its rows, at HeadLayout::rowinfo
struct RowInfo {
  int32_t *n_valid;   // rows that count
  float *scale;       // gradient: largest |dloss|
  int32_t *index;     // [rows_pad] the row's place in the caller's arrays
  int32_t *target;    // [rows_pad]
  int32_t *prev;      // [rows_pad]
  float *lse;         // [rows_pad] gradient: as the caller gave it
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
  r.lse = reinterpret_cast<float *>(p + 3 * rows_pad);
  r.weight = reinterpret_cast<float *>(p + 4 * rows_pad);
  r.z_target = reinterpret_cast<float *>(p + 5 * rows_pad);
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// With the largest score goes the sum of e^(score - base(largest)).  An infinite
// one is not subtracted from itself: scores of -infinity alone sum to 0, one of
// +infinity makes the sum infinite.  The difference is taken first and then
// multiplied by log2 e: where nothing changes a sum's rescaling by e^(old - new)
// is exactly 1, and scores as large as fp32's largest (bf16's lowest value as a
// mask) do not overflow.
__device__ __forceinline__ float base(float top) {
  return fabsf(top) == INFINITY ? 0.0f : top;
}

// ------------------------------------------------------------------ pack
// Gathers the rows with a target into A = [h, U[prev]], zero-padded to whole
// 64-column blocks and to a multiple of 32 rows, and their row data.  What an ignored
// row holds (NaN, infinities, tokens out of range) reaches nothing: its first lines
// may be prefetched, no more.  Every CTA counts the targets before its rows itself:
// 4 bytes a row from L2 (8 for the gradient), where a scan across CTAs would cost a
// second launch.  It is quadratic, but with blocks of 256 rows: the largest M, 2^20,
// reads 34 GB, some milliseconds beside products of a second.  A warp takes
// a row, eight a CTA; where that leaves SMs idle the columns are spread over CTAs
// too, 1024 or more to each (300 rows of 8192: 6 us instead of 19; loss and
// gradient with 4000 entries 143 us instead of 171).
struct PackParams {
  const uint16_t *h;
  int64_t h_stride;
  const uint16_t *U;
  const int32_t *prev, *target;
  const float *lse, *dloss;
  float *loss_out, *lse_out;
  uint16_t *dh;       // gradient: rows without a target are zeroed here
  int64_t dh_stride;
  int32_t M, vocab, d, rank, cols_pad, d_pad, rows_per_cta, cols_per_cta;
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
  const int c0 = blockIdx.y * p.cols_per_cta, c1 = min(p.cols_pad, c0 + p.cols_per_cta);
  const int chunks = (c1 - c0) / 8;
  // what there is once for a row is written with the first columns
  const auto first = [] { return blockIdx.y == 0; };
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
    const int col = c0 + lane * 64;
    if (col < min(c1, p.d)) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(
          p.h + static_cast<int64_t>(r0 + j) * p.h_stride + col));
    }
    const int u = lane * 64;
    if (u < p.rank && p.d_pad + u >= c0 && p.d_pad + u < c1) {
      const int32_t pv = p.prev[r0 + j];
      if (counts(pv, p.vocab))
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.U + static_cast<int64_t>(pv) * p.rank + u));
    }
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
  if (!(top < INFINITY)) top = 1.0f;  // an infinite one is its own row's alone in dh
  if (first() && blockIdx.x == 0 && tid == 0) {
    *p.rows.n_valid = total;
    if (GRAD) *p.rows.scale = top;
  }

  for (int j = warp; j < n; j += PACK_WARPS) {
    const int row = r0 + j;
    const uint32_t word = s_mask[j >> 5];
    if (!((word >> (j & 31)) & 1u)) {
      if (GRAD) {
        for (int c = c0 + lane * 8; c < min(c1, p.d); c += 256)
          *reinterpret_cast<uint4 *>(p.dh + static_cast<int64_t>(row) * p.dh_stride + c) =
              make_uint4(0u, 0u, 0u, 0u);
      } else if (first() && lane == 0) {
        p.loss_out[row] = 0.0f;
        p.lse_out[row] = 0.0f;
      }
      if (first() && lane == 0 && p.target[row] >= p.vocab)
        raise_status(p.status, DSPARK_DEV_TOKEN_OOR);
      continue;
    }
    int at = before + __popc(word & ((1u << (j & 31)) - 1u));
    for (int w = 0; w < (j >> 5); ++w) at += __popc(s_mask[w]);
    int32_t pv = 0;
    if (p.rank > 0) {
      pv = p.prev[row];
      if (pv < 0 || pv >= p.vocab) {
        pv = 0;
        if (first() && lane == 0) raise_status(p.status, DSPARK_DEV_TOKEN_OOR);
      }
    }
    if (first() && lane == 0) {
      p.rows.index[at] = row;
      p.rows.target[at] = p.target[row];
      p.rows.prev[at] = pv;
      if (GRAD) {
        p.rows.lse[at] = p.lse[row];
        // equal weights (a mean) become exactly 1
        p.rows.weight[at] = top > 0.0f ? p.dloss[row] / top : p.dloss[row];
      }
    }
    const uint16_t *hr = p.h + static_cast<int64_t>(row) * p.h_stride;
    const uint16_t *ur = p.U + static_cast<int64_t>(pv) * p.rank;
    uint16_t *ar = p.a + static_cast<int64_t>(at) * p.cols_pad;
#pragma unroll 4
    for (int c = lane; c < chunks; c += 32) {
      const int col = c0 + c * 8;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (col < p.d)
        v = *reinterpret_cast<const uint4 *>(hr + col);
      else if (col >= p.d_pad && col - p.d_pad < p.rank)
        v = *reinterpret_cast<const uint4 *>(ur + (col - p.d_pad));
      *reinterpret_cast<uint4 *>(ar + col) = v;
    }
  }
  // the rows that fill up the last tile's columns; what its boxes read beyond
  // them is not multiplied
  const int end = (total + HU - 1) / HU * HU;
  for (int j = total + blockIdx.x * PACK_WARPS + warp; j < end; j += gridDim.x * PACK_WARPS) {
    uint16_t *ar = p.a + static_cast<int64_t>(j) * p.cols_pad;
    for (int c = c0 + lane * 8; c < c1; c += 256)
      *reinterpret_cast<uint4 *>(ar + c) = make_uint4(0u, 0u, 0u, 0u);
    if (first() && lane == 0) {
      p.rows.target[j] = -1;
      p.rows.lse[j] = 0.0f;
      p.rows.weight[j] = 0.0f;
    }
  }
}

// -------------------------------------------------------------- products
// Three kernels on one main loop.  A cluster of two CTAs computes a tile of
// 256 rows and up to 512 columns with tcgen05.mma.cta_group::2: each CTA stages
// 128 of the rows and half of the columns, 64 deep, and holds its 128 rows of
// the accumulators.
//
//   LSE    z^T tile, 256 vocabulary entries x up to 256 rows of A
//          -> per row of A (max, sum exp), and z at the target
//   PROB   z^T tile -> G^T, bf16
//   GRAD   dA^T tiles (256 columns of A x up to 512 rows; reduction over a
//          piece of the vocabulary, added up in fp32 by TMA) and dB tiles (256
//          vocabulary entries x up to 512 columns; reduction over the rows,
//          bf16), in one launch so that the ones fill the others' last wave
//
// 512 columns are two halves, both accumulators, for one read of the rows'
// operand.  The epilogue of a half runs while the other one is still
// multiplied, and at a tile's start the first half gets ahead as far as the ring
// holds.  z^T tiles have up to 256 columns, and the accumulators take turns: a chunk of
// the reduction each, of one tile after the other.
//
// What bounds them.  Many rows: the tensor cores and, after a tenth of a second
// of them, the 1400 W limit.  1632 columns x 262144 x 2304 (LSE) take 1.20 to
// 1.25 ms, 1.58 to 1.64 PFLOP/s, 0.83 to 0.86 of cuBLAS's measured burst and as
// much as its 1.71 PFLOP/s of seconds allows for the added weight stream; by
// themselves, cool, LSE reaches 2.04, PROB 1.89 and GRAD 1.85 PFLOP/s at 6464
// columns.  Few rows: HBM; LSE for 64 columns takes 180 us, 6.7 TB/s of W and V,
// GRAD for 16 rows x 65536 x 2560 138 us, 5.1 TB/s of them read and written and of
// dU's zeros.  In between a tile's operands: each SM takes in at most some 50 bytes a
// cycle, which a 256 x 256 tile needs for 0.8 of the tensor cores' rate.  Short
// reductions (some 600 entries and below): the epilogues of z^T.
//
// The rows of A are always the tile's columns or the reduction: those come in
// steps of 32 and 16, where a tile's rows are always 256, so that 403 rows cost
// 416 and not 512.  Both operands of z^T and G^T in dB have the reduction index
// contiguous; for the others the 64 x 64 boxes are read as they lie, and the
// descriptors say that the other index is the contiguous one.
enum HeadKind { kLse = 0, kProb = 1, kGrad = 2 };

// The tensor maps.  Boxes are 64 entries (128 bytes) wide.  "rows": many rows,
// for an operand whose reduction index is contiguous.  "wide": two neighbouring
// 64 x 64 blocks as one copy (a third dimension over the blocks), for the
// others: a copy costs some 30 to 50 cycles of the TMA unit beside its bytes.
struct HeadMaps {
  CUtensorMap a_rows;        // packed A, 128 rows
  CUtensorMap w_rows, v_rows;  // W and V, 128 rows
  CUtensorMap a, a_wide;
  CUtensorMap w, v, w_wide, v_wide;
  CUtensorMap g;             // G^T
  CUtensorMap g_rows;        // 128 rows
  CUtensorMap g_out;         // 32 x 32
  CUtensorMap dw, dv;        // dW and dV, 64 x 32
  CUtensorMap acc;           // fp32 sums of dA^T, 32 x 32
};

struct HeadParams {
  RowInfo rows;
  int32_t rows_pad, cols_pad, vocab;
  int32_t kd, kr;       // 64-column blocks of d and of rank
  int32_t v0;           // first vocabulary entry of the piece
  int32_t v_tiles;      // 256-entry tiles of the piece
  int32_t splits;
  int32_t first_piece;
  int32_t d, rank;
  int32_t w_whole, v_whole;  // d and rank are multiples of 64: the wide maps hold
  int32_t chunk;        // z^T: steps of 16 products that an accumulator adds up, even
  float2 *partial;
  uint4 *zeroed;             // GRAD: what it sets to zero (dU), and how many
  int64_t n_zeroed;
  uint32_t *status;
};

struct HeadTile {
  int da;       // GRAD: a dA tile
  int m, n;     // first row and column of the output tile
  int cols[2];  // columns of its halves; the second may have none
  int k0, nk;   // range of the reduction, in 64-entry blocks
  int split;
};

// `units` of `unit` columns, spread evenly over as few tiles of at most `width`
// as hold them: tile i of them, the first half as wide as it can be.
__device__ __forceinline__ void spread(int units, int unit, int width, int tiles, int i,
                                       HeadTile &x) {
  // below 2^28: no more than 2^15 units and 2^12 tiles
  const int lo = static_cast<int>(static_cast<uint32_t>(units * i) / static_cast<uint32_t>(tiles));
  const int n = static_cast<int>(static_cast<uint32_t>(units * (i + 1)) /
                                 static_cast<uint32_t>(tiles)) - lo;
  x.n = lo * unit;
  x.cols[0] = min(n * unit, HT);
  x.cols[1] = n * unit - x.cols[0];
}

__device__ __forceinline__ int row_tiles(int n_valid, int width) {
  return (n_valid + width - 1) / width;
}

__device__ __forceinline__ void row_tile(int n_valid, int width, int i, HeadTile &x) {
  spread((n_valid + HU - 1) / HU, HU, width, row_tiles(n_valid, width), i, x);
}

// Width of the tiles whose columns are rows of A.  z^T tiles leave an accumulator
// to the chunk that follows: their epilogues (an exponential for each entry) take a
// fifth of a tile's time and hide only behind other products (512 columns: 1280 us
// instead of 1190 at 1613 rows x 262144 x 2304).  dA^T tiles have a long reduction
// and a short epilogue (256 columns: 19.8 ms instead of 18.9 for 6452 rows, loss and
// gradient).
template <int KIND>
__device__ __forceinline__ int row_width(int n_valid) {
  return KIND == kGrad && n_valid > HT ? HW : HT;
}

// dB tiles: 512 columns where the reduction over the rows is as long (256: 20.0
// ms instead of 18.9 for 6452 rows); for few rows 256, whose epilogue hides
// behind the next tile (512: 835 us instead of 790 for 403 rows).
__device__ __forceinline__ int weight_width(int n_valid) { return n_valid > 1024 ? HW : HT; }

// What a pair does.  z^T tiles, and dA tiles before dB tiles, go round over the
// pairs; each pair then gets a run of dB tiles, shorter where it has one dA tile
// more, so that all have the same to do.
struct HeadWork {
  int width;             // of tiles whose columns are rows of A
  int nt;                // and how many there are side by side
  int round;             // z^T or dA tiles
  int db_lo, db_hi;      // the pair's dB tiles
};

template <int KIND>
__device__ __forceinline__ HeadWork head_work(const HeadParams &p, int n_valid, int pair,
                                              int pairs) {
  HeadWork w;
  w.width = row_width<KIND>(n_valid);
  const int nt = w.nt = row_tiles(n_valid, w.width);
  if (KIND != kGrad) {
    w.round = nt * p.v_tiles;
    w.db_lo = w.db_hi = 0;
    return w;
  }
  const int d_tiles = (p.cols_pad + HT - 1) / HT;
  w.round = nt * d_tiles * p.splits;
  const int width = weight_width(n_valid);
  const int n_db = p.v_tiles * ((p.cols_pad + width - 1) / width);
  // times in 64-entry blocks of 256 columns; with fewer columns a block of dA
  // takes as long, for W streams through it (2 rows x 89769 x 1152: 0.28 us a
  // block); a dB tile takes as long as its reduction and about three more for
  // the stores, but no less than seven (four: 1062 us instead of 965 for 16 rows
  // x 262144 x 2560, loss and gradient)
  const float t_da = static_cast<float>(p.v_tiles) * (HT / HK) / p.splits *
                     fmaxf(1.0f, static_cast<float>(n_valid) / (HT * (nt > 0 ? nt : 1)));
  const float t_db = max((n_valid + HK - 1) / HK + 3, 7) * static_cast<float>(p.cols_pad) *
                     p.v_tiles / (static_cast<float>(HT) * n_db);
  const int more = w.round % pairs;  // pairs with one dA tile more
  const float gap = t_da / t_db;
  float x = (n_db - (pairs - more) * gap) / pairs, y = x + gap;
  if (x < 0.0f) {
    x = 0.0f;
    y = static_cast<float>(n_db) / (pairs - more);
  }
  if (more == 0) y = static_cast<float>(n_db) / pairs;
  auto start = [&](int q) {
    if (q >= pairs) return n_db;
    // unfused, so that neighbours agree on where the one ends and the other begins
    const float at = __fadd_rn(__fmul_rn(x, static_cast<float>(min(q, more))),
                               __fmul_rn(y, static_cast<float>(max(q - more, 0))));
    return min(n_db, static_cast<int>(at));
  };
  w.db_lo = start(pair);
  w.db_hi = start(pair + 1);
  return w;
}

// The i-th tile of a pair; false after the last.
template <int KIND>
__device__ __forceinline__ bool head_tile(const HeadParams &p, const HeadWork &w, int n_valid,
                                          int pair, int pairs, int i, HeadTile &x) {
  const int nt = w.nt;
  int t = pair + i * pairs;
  x.da = 0;
  x.split = 0;
  if (t < w.round) {
    if (KIND != kGrad) {
      x.m = (t / nt) * HT;
      row_tile(n_valid, w.width, t % nt, x);
      x.k0 = 0;
      x.nk = p.kd + p.kr;
      return true;
    }
    const int d_tiles = (p.cols_pad + HT - 1) / HT;
    x.da = 1;
    x.m = (t % d_tiles) * HT;
    const int u = t / d_tiles;
    row_tile(n_valid, w.width, u % nt, x);
    x.split = u / nt;
    const int kb = p.v_tiles * (HT / HK);
    x.k0 = kb * x.split / p.splits;
    x.nk = kb * (x.split + 1) / p.splits - x.k0;
    return true;
  }
  if (KIND != kGrad) return false;
  const int da = w.round > pair ? (w.round - pair + pairs - 1) / pairs : 0;
  t = w.db_lo + i - da;
  if (t >= w.db_hi) return false;
  const int width = weight_width(n_valid), tiles = (p.cols_pad + width - 1) / width;
  spread(p.cols_pad / 64, 64, width, tiles, t % tiles, x);
  x.m = (t / tiles) * HT;
  x.k0 = 0;
  x.nk = (n_valid + HK - 1) / HK;
  return true;
}

// Operand descriptors, as in common.cuh, in halves.  K-major operand (the
// reduction index contiguous): 8-row atoms of 1024 bytes.  Otherwise the
// 128-byte rows run along the other index, 64 entries each; one row per
// reduction index, 8 rows (1024 bytes) an atom, atoms 1024 bytes apart along
// the reduction (bits 32-45) and a box apart along the other index (bits
// 16-29).  The upper half is the same; 16 reduction entries on, the address is
// 32 bytes further in the one, two atoms in the other (in units of 16 bytes).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr, bool mn_major) {
  return ((smem_addr & 0x3FFFFu) >> 4) | (mn_major ? static_cast<uint32_t>(H_BOX >> 4) << 16
                                                   : 1u << 16);
}
__device__ __forceinline__ uint32_t desc_step(bool mn_major) { return mn_major ? 128u : 2u; }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ------------------------------------------------------------- epilogues
// A warp has 32 rows of the accumulator, a lane one of them; two warps share
// the rows and take every second block of a half's columns (`part` 0 or 1; the
// half begins at column n and has `cols`).  The next 32 columns are on their
// way from tensor memory while the ones before are used, and the accumulator
// is given back as soon as its last are in registers.  What goes to memory is
// laid out in the warp's box of shared memory (the swizzle of its tensor map)
// and stored by TMA.
struct HalfTile {
  int n, cols, part;
  bool empty;         // no reduction: all zero, and no accumulator
  uint32_t acc, box;  // tensor memory, shared memory
  uint32_t acc_empty; // barrier, in the cluster's window
  int lane;
  int *stores;        // the warp's stores so far: which half of its box is next
};

__device__ __forceinline__ void give_back(const HalfTile &t) {
  if (t.empty) return;
  tc_fence_before();
  __syncwarp();
  if (t.lane == 0) mbar_arrive_cluster(t.acc_empty);
}

// use(b, column, values) for each block b of 32 columns; the two warps take every
// second one, or with BY64 every second two
template <bool BY64 = false, class F>
__device__ __forceinline__ void each_block(const HalfTile &t, F use) {
  auto column = [&](int b) {
    return BY64 ? t.part * 64 + (b >> 1) * 128 + (b & 1) * 32 : t.part * 32 + b * 64;
  };
  uint32_t v[2][32];
  if (t.empty) {
#pragma unroll
    for (int e = 0; e < 32; ++e) v[0][e] = 0u;
    for (int b = 0; b < 4; ++b)
      if (column(b) < t.cols) use(b, column(b), v[0]);
    return;
  }
  if (column(0) >= t.cols) {
    give_back(t);
    return;
  }
  tmem_ld_32x32b_x32(t.acc + column(0), v[0]);
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (column(b) >= t.cols) break;
    tmem_ld_wait(v[b & 1]);
    if (b < 3 && column(b + 1) < t.cols)
      tmem_ld_32x32b_x32(t.acc + column(b + 1), v[(b + 1) & 1]);
    else
      give_back(t);
    use(b, column(b), v[b & 1]);
  }
}

// z^T: the warp's columns of a tile, 32 of each block.  The tensor cores truncate
// their running sum each time they add 16 products to it, which takes up to an ulp
// of that sum towards zero; over a whole reduction of 2304 scores that grow evenly
// come out 2.1e-6 of themselves too small, others not at all.  So an accumulator
// adds up a chunk of the reduction only (HeadParams::chunk), and the chunks are added
// here, rounded to nearest, while the next ones are multiplied.  In five chunks
// 1613 rows x 262144 x 2304 take 2 to 3 % longer than in one, 601 x 50003 x 1000 a
// tenth; short reductions, whose epilogues are as long as their products, a quarter
// to two fifths (256 and 576 entries).
struct Scores {
  float z[4][32];
};

// two blocks are on their way at once
__device__ __forceinline__ void add_chunk(const HalfTile &t, Scores &s) {
  auto column = [&](int b) { return t.part * 32 + b * 64; };
#pragma unroll
  for (int b = 0; b < 4; b += 2) {
    if (column(b) >= t.cols) break;
    uint32_t v[2][32];
    const bool two = column(b + 1) < t.cols;
    tmem_ld_32x32b_x32(t.acc + column(b), v[0]);
    if (two) tmem_ld_32x32b_x32(t.acc + column(b + 1), v[1]);
    tmem_ld_wait(v[0]);
    if (b == 2 || column(2) >= t.cols) give_back(t);
#pragma unroll
    for (int e = 0; e < 32; ++e) s.z[b][e] += __uint_as_float(v[0][e]);
    if (two) {
      tmem_ld_wait(v[1]);
#pragma unroll
      for (int e = 0; e < 32; ++e) s.z[b + 1][e] += __uint_as_float(v[1][e]);
    }
  }
  if (column(0) >= t.cols) give_back(t);
}

// use(b, column, scores) for each block of 32 columns
template <class F>
__device__ __forceinline__ void each_scores(const HalfTile &t, Scores &s, F use) {
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int c = t.part * 32 + b * 64;
    if (c >= t.cols) break;
    use(b, c, s.z[b]);
  }
}

__device__ __forceinline__ void box_is_free(int lane) {
  if (lane == 0) bulk_wait_read<0>();  // the last store has read it
  __syncwarp();
}

// 32 x 32 values as bf16 into one of the warp's two boxes of 2 KB (rows of 64
// bytes, 64-byte swizzle).  They take turns store by store, over tiles too
// (which may have an odd number of blocks, or skip some): the only store that
// may still be reading is then the other box's.
__device__ __forceinline__ uint32_t put_32x32(const HalfTile &t, const float (&g)[32]) {
  const uint32_t box = t.box + (*t.stores & 1) * (H_OUT_BOX / 2);
  ++*t.stores;
  if (t.lane == 0) bulk_wait_read<1>();
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    st_shared_v4(box + t.lane * 64 + ((c ^ ((t.lane >> 1) & 3)) << 4),
                 make_uint4(pack_bf16(g[8 * c], g[8 * c + 1]),
                            pack_bf16(g[8 * c + 2], g[8 * c + 3]),
                            pack_bf16(g[8 * c + 4], g[8 * c + 5]),
                            pack_bf16(g[8 * c + 6], g[8 * c + 7])));
  fence_proxy_async_smem();
  __syncwarp();
  return box;
}

// LSE: lanes are vocabulary entries, columns rows of A.  A 32 x 32 block is
// turned in shared memory, so that a lane has 32 entries of its own row of A
// and needs no other lane for their maximum and sum.  A row's running pair and
// target are read before the accumulator is waited for.
struct LseRows {
  float2 run[4];
  int target[4];
};

__device__ __forceinline__ LseRows lse_rows(const HeadParams &p, const float2 *slot, bool first,
                                            int n, int cols, int part, int lane) {
  LseRows r;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int c = part * 32 + b * 64;
    if (c < cols) {
      r.run[b] = first ? make_float2(-INFINITY, 0.0f) : slot[n + c + lane];
      r.target[b] = p.rows.target[n + c + lane];
    }
  }
  return r;
}

__device__ __forceinline__ void lse_tile(const HeadParams &p, const HalfTile &t, Scores &scores,
                                         int v_first, const LseRows &rows, float2 *slot) {
  const int lane = t.lane;
  const bool beyond = v_first + lane >= p.vocab;
  each_scores(t, scores, [&](int b, int c0, float (&own)[32]) {
    const int row = t.n + c0 + lane;
    if (beyond) {
#pragma unroll
      for (int e = 0; e < 32; ++e) own[e] = -INFINITY;
    }
    __syncwarp();  // the block before has been read
#pragma unroll
    for (int c = 0; c < 8; ++c)
      st_shared_v4(t.box + lane * 128 + ((c ^ (lane & 7)) << 4),
                   make_uint4(__float_as_uint(own[4 * c]), __float_as_uint(own[4 * c + 1]),
                              __float_as_uint(own[4 * c + 2]), __float_as_uint(own[4 * c + 3])));
    __syncwarp();
    float z[32];
#pragma unroll
    for (int v = 0; v < 32; ++v) {
      uint32_t w;
      asm volatile("ld.shared.u32 %0, [%1];"
                   : "=r"(w)
                   : "r"(t.box + v * 128 + (((lane >> 2) ^ (v & 7)) << 4) + (lane & 3) * 4));
      z[v] = __uint_as_float(w);
    }
    const int at = rows.target[b] - v_first;
    if (static_cast<uint32_t>(at) < 32u) {
      float zt = 0.0f;
#pragma unroll
      for (int v = 0; v < 32; ++v) zt = v == at ? z[v] : zt;
      p.rows.z_target[row] = zt;
    }
    const float2 old = rows.run[b];
    float m[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
    for (int v = 4; v < 32; ++v) m[v & 3] = fmaxf(m[v & 3], z[v]);
    const float top = fmaxf(old.x, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
    const float ref = base(top);
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < 32; ++v) part[v & 3] += ex2((z[v] - ref) * kLog2e);
    const float sum =
        fmaf(old.y, ex2((old.x - ref) * kLog2e), (part[0] + part[1]) + (part[2] + part[3]));
    slot[row] = make_float2(top, sum);
  });
}

__device__ __forceinline__ float prob(float z, float lse) { return ex2((z - lse) * kLog2e); }

// PROB: lanes are vocabulary entries, columns rows of A.  G^T is rounded to bf16:
// as an operand it has to be, for bf16 products; at most 2^-8 of an entry, and
// the entries' roundings are independent in the sums.  dloss enters as a share of
// the largest one, so that a mean's small weights lose nothing.
__device__ __forceinline__ void prob_tile(const HeadParams &p, const CUtensorMap &g_out,
                                          const HalfTile &t, Scores &scores, int row0,
                                          int n_valid) {
  const int lane = t.lane, v_first = p.v0 + row0;
  const bool beyond = v_first + lane >= p.vocab;
  each_scores(t, scores, [&](int, int c0, float (&z)[32]) {
    const float4 *lse = reinterpret_cast<const float4 *>(p.rows.lse + t.n + c0);
    const float4 *weight = reinterpret_cast<const float4 *>(p.rows.weight + t.n + c0);
    const int at = p.rows.target[t.n + c0 + lane] - v_first;
    const uint32_t hits = __ballot_sync(0xFFFFFFFFu, static_cast<uint32_t>(at) < 32u);
    float g[32];
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const float4 l = lse[e / 4], w = weight[e / 4];
      g[e] = prob(z[e], l.x) * w.x;
      g[e + 1] = prob(z[e + 1], l.y) * w.y;
      g[e + 2] = prob(z[e + 2], l.z) * w.z;
      g[e + 3] = prob(z[e + 3], l.w) * w.w;
    }
    if (hits) {
      const float own = p.rows.weight[t.n + c0 + lane];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int v = __shfl_sync(0xFFFFFFFFu, at, e);
        const float w = __shfl_sync(0xFFFFFFFFu, own, e);
        if (v == lane) g[e] -= w;
      }
    }
    // Zero by choice, not by a product with 0, for entries and rows that there are
    // not: the rows that fill up a 16 of dB's reduction score NaN at an entry that
    // holds an infinity (a mask in V, say).
    const int live = beyond ? 0 : n_valid - (t.n + c0);
    if (live < 32) {
#pragma unroll
      for (int e = 0; e < 32; ++e) g[e] = e < live ? g[e] : 0.0f;
    }
    const uint32_t box = put_32x32(t, g);
    if (lane == 0) {
      tma_store_2d(&g_out, box, t.n + c0, row0);
      bulk_commit();
    }
  });
}

// dA^T: lanes are columns of A, columns its rows; fp32, one addition a piece.
// What its truncated additions lose (at most 393216 / 16 of them, 2^-26 of the
// sum each) is below 2^-11 of it, and dB's (2^20 rows at most) below 2^-10; the
// results' rounding to bf16 is up to 2^-8.
__device__ __forceinline__ void sum_tile(const HeadParams &p, const CUtensorMap &acc_map,
                                         const HalfTile &t, int split, int row0) {
  const int lane = t.lane;
  each_block(t, [&](int, int c0, uint32_t (&acc)[32]) {
    if (row0 >= p.cols_pad) return;
    box_is_free(lane);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      st_shared_v4(t.box + lane * 128 + ((c ^ (lane & 7)) << 4),
                   make_uint4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]));
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      const int y = split * p.cols_pad + row0;
      if (p.first_piece)
        tma_store_2d(&acc_map, t.box, t.n + c0, y);
      else
        tma_reduce_add_2d(&acc_map, t.box, t.n + c0, y);
      bulk_commit();
    }
  });
}

// dB: lanes are vocabulary entries, columns those of [W, V].  Stored 64 columns
// at a time, whole lines of 128 bytes.
__device__ __forceinline__ void weight_tile(const HeadParams &p, const HeadMaps &maps,
                                            const HalfTile &t, int row0, float scale) {
  const int lane = t.lane;
  if (p.v0 + row0 >= p.vocab) {
    give_back(t);
    return;
  }
  each_block<true>(t, [&](int b, int c0, uint32_t (&acc)[32]) {
    const int odd = b & 1;
    if (!odd) box_is_free(lane);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float g[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = __uint_as_float(acc[8 * c + e]) * scale;
      st_shared_v4(t.box + lane * 128 + (((odd * 4 + c) ^ (lane & 7)) << 4),
                   make_uint4(pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]),
                              pack_bf16(g[4], g[5]), pack_bf16(g[6], g[7])));
    }
    if (!odd) return;
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      const int col = t.n + c0 - 32;
      if (col < p.kd * HK)
        tma_store_2d(&maps.dw, t.box, col, p.v0 + row0);
      else
        tma_store_2d(&maps.dv, t.box, col - p.kd * HK, p.v0 + row0);
      bulk_commit();
    }
  });
}

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(H_THREADS, 1)
    head_gemm_kernel(const __grid_constant__ HeadMaps maps, const HeadParams p) {
  constexpr int HALVES = KIND == kGrad ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t *smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + H_BAR_OFF);
  uint64_t *empty = full + H_MAX_STAGES;
  uint64_t *acc_full = empty + H_MAX_STAGES;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *mma_done = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(full + H_BARS);
  volatile uint32_t *abort_flag = tmem_slot + 1;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int cta = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < H_MAX_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * H_EPI_WARPS);  // of either CTA
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
  const int n_valid = __shfl_sync(0xFFFFFFFFu, *p.rows.n_valid, 0);
  const HeadWork work = head_work<KIND>(p, n_valid, pair, pairs);
  // a stage holds 128 rows and up to 128 columns of one half or of two, or 64
  const bool wide = work.width == HW || (KIND == kGrad && weight_width(n_valid) == HW);
  const bool few = KIND != kGrad && n_valid <= 128;
  const int stages = wide ? 4 : few ? 8 : 6;
  const int stage_bytes = H_RING / stages;
  HeadTile x;

  if (warp < 4) {
    if (KIND != kGrad) registers_down<H_Z_OTHER_REGS>();
    if (warp == 0) {
      // ---------------------------------------------------------- loads
      const uint32_t one = elect_one();
      const uint32_t full0 = mapa_u32(smem_u32(full), 0), ring = smem_u32(smem);
      bool ok = true;
      int s = 0;
      uint32_t phase = 1u;
      for (int i = 0; ok && head_tile<KIND>(p, work, n_valid, pair, pairs, i, x); ++i) {
        // this CTA's half of each half's columns, in whole blocks of 64
        const int mine[2] = {x.cols[0] / 2, x.cols[1] / 2};
        const int col0[2] = {x.n + cta * mine[0], x.n + x.cols[0] + cta * mine[1]};
        const int blocks[2] = {(mine[0] + 63) / 64, (mine[1] + 63) / 64};
        const uint32_t bytes = 2 * (H_OPERAND + (blocks[0] + blocks[1]) * H_BOX);
        for (int kb = x.k0; kb < x.k0 + x.nk; ++kb) {
          ok = __all_sync(0xFFFFFFFFu, wait_bounded(&empty[s], phase, abort_flag, p.status));
          if (!ok) break;
          if (cta == 0 && one) mbar_arrive_expect_tx(&full[s], bytes);
          __syncwarp();
          const uint32_t bar = full0 + s * 8;
          const uint32_t sa = ring + s * stage_bytes, sb = sa + H_OPERAND;
          if (KIND != kGrad) {
            const bool in_d = kb < p.kd;
            tma_load_2d_pair(one, sa, in_d ? &maps.w_rows : &maps.v_rows, bar,
                             (in_d ? kb : kb - p.kd) * HK, p.v0 + x.m + cta * 128);
            // few and large copies, also of fewer rows: exact ones of 64, 32 and
            // 16 rows instead took up to 1.3 times as long
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
              if (blocks[h])
                tma_load_2d_pair(one, sb + h * H_OPERAND, blocks[h] == 2 ? &maps.a_rows : &maps.a,
                                 bar, kb * HK, col0[h]);
          } else if (x.da) {
            const int cb = (x.m + cta * 128) / HK;
            const bool in_d = cb < p.kd || p.kr == 0, both = in_d == (cb + 1 < p.kd || p.kr == 0);
            if (both && (in_d ? p.w_whole : p.v_whole)) {
              tma_load_3d_pair(one, sa, in_d ? &maps.w_wide : &maps.v_wide, bar, 0, p.v0 + kb * HK,
                               in_d ? cb : cb - p.kd);
            } else {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const bool d = cb + j < p.kd || p.kr == 0;
                tma_load_2d_pair(one, sa + j * H_BOX, d ? &maps.w : &maps.v, bar,
                                 (d ? cb + j : cb + j - p.kd) * HK, p.v0 + kb * HK);
              }
            }
            // G^T's columns: any 16 of them begin a block
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if (j < blocks[h])
                  tma_load_2d_pair(one, sb + h * H_OPERAND + j * H_BOX, &maps.g, bar,
                                   col0[h] + j * 64, kb * HK);
          } else {
            tma_load_2d_pair(one, sa, &maps.g_rows, bar, kb * HK, x.m + cta * 128);
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
              if (mine[h] == 128) {
                tma_load_3d_pair(one, sb + h * H_OPERAND, &maps.a_wide, bar, 0, kb * HK,
                                 col0[h] / 64);
              } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  if (j < blocks[h])
                    tma_load_2d_pair(one, sb + h * H_OPERAND + j * H_BOX, &maps.a, bar,
                                     col0[h] + j * 64, kb * HK);
              }
            }
          }
          if (++s == stages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // copies in flight land before the shared memory is given back
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 20000000ull) __nanosleep(1000);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA
      if (cta == 0) {
        const uint32_t one = elect_one();
        const uint32_t base = smem_u32(smem);
        const uint32_t empty0 = smem_u32(empty), acc_full0 = smem_u32(acc_full);
        bool ok = true;
        int s = 0, ig = 0;
        uint32_t phase = 0u;
        for (int i = 0; ok && head_tile<KIND>(p, work, n_valid, pair, pairs, i, x); ++i) {
          if (x.nk == 0) continue;
          const bool a_mn = KIND == kGrad && x.da, b_mn = KIND == kGrad;
          const uint32_t a_step = desc_step(a_mn), b_step = desc_step(b_mn);
          const uint32_t a_lo = desc_lo(base, a_mn);
          const uint32_t majors = (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
          const uint32_t idesc[2] = {
              umma_idesc_bf16_f32(HT, static_cast<uint32_t>(x.cols[0])) | majors,
              umma_idesc_bf16_f32(HT, static_cast<uint32_t>(x.cols[1])) | majors};
          const uint32_t d_tmem[2] = {tmem_base + static_cast<uint32_t>((ig & 1) * HT),
                                      tmem_base + static_cast<uint32_t>((~ig & 1) * HT)};
          const uint32_t b_lo[2] = {desc_lo(base + H_OPERAND, b_mn),
                                    desc_lo(base + 2 * H_OPERAND, b_mn)};
          auto multiply = [&](int half, int stage, int kb) {
            const uint32_t at = static_cast<uint32_t>(stage * stage_bytes) >> 4;
            const uint32_t a = a_lo + at, b = b_lo[half] + at;
            // dB's reduction ends with the rows: no 16 of them are multiplied
            // that hold none (nor were written)
            const int left = KIND == kGrad && !x.da ? n_valid - kb * HK : HK;
#pragma unroll
            for (int kk = 0; kk < HK / 16; ++kk)
              umma_bf16_pair(left > kk * 16 ? one : 0u, d_tmem[half], a + kk * a_step,
                             b + kk * b_step, kDescHi, idesc[half], kb | kk);
          };
          auto acc_free = [&](int g) {
            ok = __all_sync(0xFFFFFFFFu, wait_bounded(&acc_empty[g & 1], ((g >> 1) & 1) ^ 1u,
                                                      abort_flag, p.status));
            tc_fence_after();
            return ok;
          };
          auto arrived = [&] {
            ok = __all_sync(0xFFFFFFFFu, wait_bounded(&full[s], phase, abort_flag, p.status));
            tc_fence_after();
            return ok;
          };
          auto advance = [&] {
            if (++s == stages) {
              s = 0;
              phase ^= 1u;
            }
          };
          if (KIND != kGrad) {
            // an accumulator for each chunk of the reduction, in turn
            int step = 0;
            for (int kb = 0; kb < x.nk; ++kb) {
              if (!arrived()) break;
              const uint32_t at = static_cast<uint32_t>(s * stage_bytes) >> 4;
#pragma unroll
              for (int kk = 0; kk < HK / 16; ++kk) {
                if (step == 0 && !acc_free(ig)) break;
                umma_bf16_pair(one, tmem_base + static_cast<uint32_t>((ig & 1) * HT),
                               a_lo + at + kk * a_step, b_lo[0] + at + kk * b_step, kDescHi,
                               idesc[0], step);
                if (++step == p.chunk || (kb == x.nk - 1 && kk == HK / 16 - 1)) {
                  umma_commit_pair(one, acc_full0 + (ig & 1) * 8);
                  ++ig;
                  step = 0;
                }
              }
              if (!ok) break;
              umma_commit_pair(one, empty0 + s * 8);
              advance();
            }
            if (!ok) break;
            continue;
          }
          const bool two = HALVES == 2 && x.cols[1] > 0;
          if (!acc_free(ig)) break;
          int kb = 0;
          if (two) {
            // the first half alone, until the second one's accumulator is free
            const int s0 = s;
            const int ahead = min(stages - 1, x.nk);
            for (; kb < ahead; ++kb) {
              if (!arrived()) break;
              multiply(0, s, kb);
              advance();
            }
            if (!ok) break;
            if (ahead == x.nk) umma_commit_pair(one, acc_full0 + (ig & 1) * 8);
            if (!acc_free(ig + 1)) break;
            for (int k = 0, t = s0; k < ahead; ++k) {
              multiply(1, t, k);
              umma_commit_pair(one, empty0 + t * 8);
              t = t + 1 == stages ? 0 : t + 1;
            }
          }
          for (; kb < x.nk; ++kb) {
            if (!arrived()) break;
            multiply(0, s, kb);
            if (kb == x.nk - 1) umma_commit_pair(one, acc_full0 + (ig & 1) * 8);
            if (two) multiply(1, s, kb);
            umma_commit_pair(one, empty0 + s * 8);
            advance();
          }
          if (!ok) break;
          if (two) umma_commit_pair(one, acc_full0 + ((ig + 1) & 1) * 8);
          ig += two ? 2 : 1;
        }
        umma_commit_pair(one, smem_u32(mma_done));
      }
      __syncwarp();
    } else if (KIND == kGrad) {
      // dU, of which the last kernel writes the rows with a token.  Beside the
      // products and without a launch of its own: loss and gradient of 64 rows x
      // 32000 x (1024 + 256) 100 us instead of 106, 250 x 262144 x (2048 + 256) 964
      // instead of 972; by PROB's warps the z tiles took longer.
      const int64_t step = static_cast<int64_t>(gridDim.x) * 64;
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x - 64; i < p.n_zeroed;
           i += step)
        p.zeroed[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  } else {
    // ------------------------------------------------------- epilogue
    // the scores of a z^T tile take 128 registers of a thread
    if (KIND != kGrad) registers_up<H_Z_EPI_REGS>();
    const int q = warp & 3, part = (warp - 4) >> 2;
    const uint32_t acc_empty0 = mapa_u32(smem_u32(acc_empty), 0);
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t box = smem_u32(smem + H_RING + (warp - 4) * H_OUT_BOX);
    const float scale = KIND == kGrad ? *p.rows.scale : 0.0f;
    int ig = 0, stores = 0;
    bool ok = true;
    float2 *slot = nullptr;
    int period = 0;  // the pair's tiles after which the same rows come again
    if (KIND == kLse) {
      int g = pairs, r = work.nt;
      while (r) {
        const int m = g % r;
        g = r;
        r = m;
      }
      period = work.nt / g;
      // the running pairs of these 32 lanes' entries, one for a row of A; each
      // of the two warps has the rows that it will meet
      slot = p.partial + static_cast<int64_t>(blockIdx.x * 4 + q) * p.rows_pad;
      for (int i = 0; i < work.nt; ++i) {
        row_tile(n_valid, work.width, i, x);
        for (int h = 0; h < HALVES; ++h)
          for (int c0 = part * 32; c0 < x.cols[h]; c0 += 64)
            slot[x.n + h * x.cols[0] + c0 + lane] = make_float2(-INFINITY, 0.0f);
      }
    }
    for (int i = 0; ok && head_tile<KIND>(p, work, n_valid, pair, pairs, i, x); ++i) {
      const int row0 = x.m + cta * 128 + q * 32;  // the warp's first output row
      if constexpr (KIND != kGrad) {
        LseRows rows;
        if (KIND == kLse) rows = lse_rows(p, slot, i < period, x.n, x.cols[0], part, lane);
        HalfTile t;
        t.n = x.n;
        t.cols = x.cols[0];
        t.part = part;
        t.empty = false;
        t.box = box;
        t.lane = lane;
        t.stores = &stores;
        Scores scores;
        auto arrived = [&] {
          const int buf = ig & 1;
          ok = __all_sync(0xFFFFFFFFu,
                          wait_bounded(&acc_full[buf], (ig >> 1) & 1, abort_flag, p.status));
          tc_fence_after();
          t.acc = lane_base + static_cast<uint32_t>(buf * HT);
          t.acc_empty = acc_empty0 + buf * 8;
          ++ig;
          return ok;
        };
        const int chunks = (x.nk * (HK / 16) + p.chunk - 1) / p.chunk;
        scores = {};
#pragma unroll 1
        for (int c = 0; c < chunks && arrived(); ++c) add_chunk(t, scores);
        if (!ok) break;
        if (KIND == kLse)
          lse_tile(p, t, scores, p.v0 + row0, rows, slot);
        else
          prob_tile(p, maps.g_out, t, scores, row0, n_valid);
      } else {
#pragma unroll 1
        for (int h = 0; h < HALVES; ++h) {
          if (x.cols[h] == 0) break;
          const int buf = ig & 1;
          if (x.nk > 0) {
            ok = __all_sync(0xFFFFFFFFu,
                            wait_bounded(&acc_full[buf], (ig >> 1) & 1, abort_flag, p.status));
            if (!ok) break;
            tc_fence_after();
            ++ig;
          }
          HalfTile t;
          t.n = x.n + h * x.cols[0];
          t.cols = x.cols[h];
          t.part = part;
          t.empty = x.nk == 0;
          t.acc = lane_base + static_cast<uint32_t>(buf * HT);
          t.box = box;
          t.acc_empty = acc_empty0 + buf * 8;
          t.lane = lane;
          t.stores = &stores;
          if (x.da)
            sum_tile(p, maps.acc, t, x.split, row0);
          else
            weight_tile(p, maps, t, row0, scale);
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
    if (KIND != kGrad) {
      // all alike again; the warpgroup meets between two changes
      if (part == 0)
        warpgroup_sync<1>();
      else
        warpgroup_sync<2>();
      registers_down<H_Z_OTHER_REGS>();
    }
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
// Joins the (max, sum) pairs of a row.  A CTA takes eight neighbouring rows (64
// bytes of a slot), 128 slots at a time, in a fixed order.  Up to 608 slots: for
// few rows latency, 5 us; for 7053 rows their 34 MB, 14 us.
constexpr int JOIN_ROWS = 8;
constexpr int JOIN_THREADS = 1024;

__device__ __forceinline__ float2 join_pairs(float2 a, float2 b) {
  const float top = fmaxf(a.x, b.x);
  const float ref = base(top);
  return make_float2(top, a.y * ex2((a.x - ref) * kLog2e) + b.y * ex2((b.x - ref) * kLog2e));
}
__device__ __forceinline__ float2 join_across(float2 a, int lanes) {
  return join_pairs(a, make_float2(__shfl_xor_sync(0xFFFFFFFFu, a.x, lanes),
                                   __shfl_xor_sync(0xFFFFFFFFu, a.y, lanes)));
}

__global__ void __launch_bounds__(JOIN_THREADS)
    head_join_kernel(const float2 *partial, int slots, int rows_pad, RowInfo rows,
                     float *loss, float *lse) {
  __shared__ float2 part[JOIN_THREADS / 32][JOIN_ROWS];
  allow_next_kernel();
  wait_for_earlier_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * JOIN_ROWS + (lane & 7);
  const int n_valid = *rows.n_valid;
  if (blockIdx.x * JOIN_ROWS >= n_valid) return;
  constexpr int U = 5;  // 608 slots at once
  float2 run = make_float2(-INFINITY, 0.0f);
  for (int v = warp * 4 + (lane >> 3); v < slots; v += 128 * U) {
    float2 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = v + u * 128;
      x[u] = at < slots && row < n_valid ? partial[static_cast<int64_t>(at) * rows_pad + row]
                                         : make_float2(-INFINITY, 0.0f);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) run = join_pairs(run, x[u]);
  }
  run = join_across(join_across(run, 8), 16);
  if (lane < JOIN_ROWS) part[warp][lane] = run;
  __syncthreads();
  if (warp > 0) return;
  run = part[(lane >> 3) * 8][lane & 7];
#pragma unroll
  for (int w = 1; w < 8; ++w) run = join_pairs(run, part[(lane >> 3) * 8 + w][lane & 7]);
  run = join_across(join_across(run, 8), 16);
  if (lane < JOIN_ROWS && row < n_valid) {
    const int i = rows.index[row];
    // the loss by the distance to the largest score, which keeps what the largest
    // one's own rounding would take from lse
    const float log_sum = log2f(run.y) * kLn2;
    lse[i] = run.x + log_sum;
    loss[i] = (run.x - rows.z_target[row]) + log_sum;
  }
}

// ------------------------------------------------------- dh and dU, at last
// The splits' sums of dA^T in order, times the scale, turned: d columns go to
// dh at the row's own place, the rank's to dE (fp32, packed rows) for dU.  A
// CTA turns 64 columns of 32 rows.  Latency for few rows: 4 to 6 us for up to 8
// splits, 8 for 403 rows x 2304.
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
  {
    const float *x = acc + static_cast<int64_t>(c0 + warp) * rows_pad + r0 + lane;
    float s[TURN_COLS / 8] = {};
    // eight splits' values in flight at a time; added in the splits' order
    for (int k = 0; k < splits; k += 8) {
      float v[8][TURN_COLS / 8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int j = 0; j < TURN_COLS / 8; ++j)
          v[u][j] = k + u < splits
                        ? x[(static_cast<int64_t>(k + u) * cols_pad + j * 8) * rows_pad]
                        : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int j = 0; j < TURN_COLS / 8; ++j) s[j] += v[u][j];
    }
#pragma unroll
    for (int j = 0; j < TURN_COLS / 8; ++j) block[lane][warp + j * 8] = s[j] * scale;
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
// in which CTAs run.  Tokens that no row names were zeroed by GRAD.  Each CTA looks
// through all rows' tokens, from L2: 5 us for 403 rows, 23 for 7053, and some 6 ms for
// 131072 rows of different tokens (beside 53 ms of the narrowest products).
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
  EncodeTiledFn enc = encode_tiled_fn();
  // the swizzle is as wide as the box's rows
  const auto swizzle =
      box_cols * esz == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * esz};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1, 1};
  return enc(m, type, 2, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_bf16(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int box_rows) {
  return encode_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, cols, rows, cols, 64, box_rows);
}

// [rows, cols] of bf16 as 64-column blocks: boxes of 64 rows in two neighbouring
// blocks.  cols is a multiple of 64.
bool encode_wide(CUtensorMap *m, const void *base, int64_t cols, int64_t rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols / 64)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, 128};
  cuuint32_t box[3] = {64, 64, 2};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct HeadPlan {
  HeadLayout lay;
  HeadMaps maps;
  HeadParams p;
  PackParams pack;
  int sms;
  dim3 pack_grid;
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
      // an increase of registers beyond the launch's own would wait for ever
      cudaFuncAttributes lse = {}, prob = {};
      if (cudaFuncGetAttributes(&lse, head_gemm_kernel<kLse>) != cudaSuccess ||
          cudaFuncGetAttributes(&prob, head_gemm_kernel<kProb>) != cudaSuccess ||
          lse.numRegs < H_REGS || prob.numRegs < H_REGS)
        return DSPARK_ERR_CUDA;
      g_head_attr[dev] = true;
    }
  }
  const HeadLayout &l = o.lay = head_layout(a.M, a.vocab, a.d, a.rank, grad);
  uint8_t *ws = a.workspace;
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int64_t vr = a.rank ? a.rank : a.d;
  const void *V = a.rank ? a.V : a.W;
  const void *A = ws + l.a, *G = ws + l.g;
  o.p.w_whole = a.d % 64 == 0;
  o.p.v_whole = vr % 64 == 0;
  HeadMaps &m = o.maps;
  bool ok = encode_bf16(&m.w_rows, a.W, a.d, a.vocab, 128) &&
            encode_bf16(&m.v_rows, V, vr, a.vocab, 128) &&
            encode_bf16(&m.a_rows, A, l.cols_pad, l.rows_pad, 128) &&
            encode_bf16(&m.a, A, l.cols_pad, l.rows_pad, 64);
  if (grad) {
    ok = ok && encode_wide(&m.a_wide, A, l.cols_pad, l.rows_pad) &&
         encode_bf16(&m.w, a.W, a.d, a.vocab, 64) && encode_bf16(&m.v, V, vr, a.vocab, 64) &&
         (!o.p.w_whole || encode_wide(&m.w_wide, a.W, a.d, a.vocab)) &&
         (!o.p.v_whole || encode_wide(&m.v_wide, V, vr, a.vocab)) &&
         encode_bf16(&m.g, G, l.rows_pad, l.piece, 64) &&
         encode_bf16(&m.g_rows, G, l.rows_pad, l.piece, 128) &&
         encode_2d(&m.g_out, bf16, 2, G, l.rows_pad, l.piece,
                   l.rows_pad, 32, 32) &&
         encode_2d(&m.dw, bf16, 2, a.dW, a.d, a.vocab, a.d, 64, 32) &&
         encode_2d(&m.dv, bf16, 2, a.rank ? a.dV : a.dW, vr, a.vocab, vr, 64, 32) &&
         encode_2d(&m.acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, ws + l.acc, l.rows_pad,
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
  p.splits = l.splits;
  p.v0 = 0;
  p.v_tiles = (a.vocab + HT - 1) / HT;
  p.first_piece = 0;
  p.zeroed = nullptr;
  p.n_zeroed = 0;
  const int adds = (a.d + 15) / 16 + (a.rank + 15) / 16;
  // A chunk is a bit more than a fifth of the reduction, 2 additions at least and 64
  // at most: a score that grows evenly loses n + 1 of 2^-26 of itself for n additions
  // to a chunk (measured for 16 to 256 of them), a quarter or so of what one
  // accumulator would take, and one whose sums are exact loses nothing.
  p.chunk = std::max(2, std::min(64, adds * 2 / 9 / 2 * 2));
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
  // some CTAs also for the rows that fill up
  o.pack_grid = dim3(std::max(4, (a.M + k.rows_per_cta - 1) / k.rows_per_cta));
  const int64_t most = (l.cols_pad + 1023) / 1024;
  const int64_t parts =
      std::max<int64_t>(1, std::min<int64_t>(most, 2 * o.sms / int64_t{o.pack_grid.x}));
  k.cols_per_cta = static_cast<int32_t>(up((l.cols_pad + parts - 1) / parts, HK));
  o.pack_grid.y = static_cast<unsigned>((l.cols_pad + k.cols_per_cta - 1) / k.cols_per_cta);
  return DSPARK_OK;
}

// no more pairs than there can be tiles
template <int KIND>
int head_pairs(const HeadPlan &o, const HeadParams &p) {
  const int64_t rows = o.lay.rows_pad, dt = (o.lay.cols_pad + HT - 1) / HT;
  const int64_t tiles = KIND == kGrad ? dt * ((rows + HW - 1) / HW * p.splits + p.v_tiles)
                                      : rows / HT * p.v_tiles;
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
    // dA's reduction over the piece is split where a tile of it would take longer
    // than a pair's share of all tiles (as in head_work, in 64-entry blocks of 256
    // columns).  2 rows x 89769 x 1152 take 127 us in 10 splits, and 387 in one,
    // whose five pairs alone read all of W.
    const int64_t nt = (l.rows_pad + HW - 1) / HW, dt = (l.cols_pad + HT - 1) / HT;
    const double deep = static_cast<double>(l.piece) / HK;
    const double t_da = deep * std::max(1.0, M / (static_cast<double>(HT) * nt));
    const double t_db = std::max(static_cast<double>(M) / HK + 3.0, 7.0) * l.cols_pad / HT *
                        l.piece / HT;
    const double share = (static_cast<double>(nt * dt) * t_da + t_db) / kPairs;
    l.splits = static_cast<int32_t>(
        std::max(1.0, std::min({std::ceil(t_da / (0.9 * share)), deep / 8.0, 32.0})));
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
    e = launch_overlapped(head_join_kernel, (a.M + JOIN_ROWS - 1) / JOIN_ROWS, JOIN_THREADS, 0,
                          stream, static_cast<const float2 *>(o.p.partial),
                          head_pairs<kLse>(o, o.p) * 8, o.p.rows_pad, o.p.rows, a.loss, a.lse);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

dspark_status head_loss_grad_launch(const HeadArgs &a, cudaStream_t stream) {
  HeadPlan o;
  const dspark_status s = head_plan(a, true, o);
  if (s != DSPARK_OK) return s;
  const HeadLayout &l = o.lay;
  cudaError_t e =
      launch_overlapped(head_pack_kernel<true>, o.pack_grid, PACK_THREADS, 0, stream, o.pack);
  HeadParams p = o.p;
  for (int64_t v0 = 0; v0 < a.vocab && e == cudaSuccess; v0 += l.piece) {
    p.v0 = static_cast<int32_t>(v0);
    p.v_tiles = static_cast<int32_t>((std::min<int64_t>(l.piece, a.vocab - v0) + HT - 1) / HT);
    p.first_piece = v0 == 0;
    p.zeroed = reinterpret_cast<uint4 *>(a.dU);
    p.n_zeroed = v0 == 0 ? static_cast<int64_t>(a.vocab) * a.rank / 8 : 0;
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
