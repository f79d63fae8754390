// Softmax cross entropy of the Markov head's scores and its gradient.
//
//   A_i = [h_i, U[prev_i]]      B_v = [W_v, V_v]      z_iv = A_i . B_v
//   lse_i = log sum_v exp z_iv        loss_i = lse_i - z_{i, target_i}
//   G_iv = dloss_i (exp(z_iv - lse_i) - [v = target_i])
//   dA = G B      dB = G^T A      dU[t] = sum over prev_i = t of dA_i's tail
//
// The scores are never stored.  The loss keeps one (maximum, sum) pair for a
// row and 256 vocabulary entries; the gradient computes z again for a piece of
// the vocabulary, writes that piece of G as bf16 and takes both products with
// it before the next piece.  Only rows with a target are computed: they are
// gathered, in order, into a packed A first.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "chain_common.cuh"
#include "common.cuh"
#include "head_internal.h"
#include "ptx_pair.cuh"

namespace dspark {

namespace {

constexpr int HT = 256;        // rows and columns of a pair's tile
constexpr int HK = 64;         // reduction entries of a stage (128 bytes)
constexpr int H_STAGES = 6;
constexpr int H_BOX = 64 * 128;             // a 64 x 64 bf16 box
constexpr int H_OPERAND = 2 * H_BOX;        // a CTA's 128 rows of one operand
constexpr int H_STAGE = 2 * H_OPERAND;
constexpr int H_OUT_BOX = 32 * 128;         // a warp's 32 rows of 128 bytes
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
  int32_t M, vocab, d, rank, cols_pad, d_pad, rows_per_cta;
  int32_t *position;
  uint16_t *a;
  RowInfo rows;
  uint32_t *status;
};

constexpr int PACK_THREADS = 256;

__device__ __forceinline__ bool counts(int32_t t, int32_t vocab) {
  return t >= 0 && t < vocab;
}

template <bool GRAD>
__global__ void __launch_bounds__(PACK_THREADS) head_pack_kernel(const PackParams p) {
  __shared__ int32_t s_before[PACK_THREADS / 32], s_total[PACK_THREADS / 32];
  __shared__ float s_max[PACK_THREADS / 32];
  __shared__ int32_t s_pos[PACK_THREADS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = blockIdx.x * p.rows_per_cta;
  const int r1 = min(p.M, r0 + p.rows_per_cta);

  int before = 0, total = 0;
  float top = 0.0f;
  for (int i = tid; i < p.M; i += PACK_THREADS) {
    const bool ok = counts(p.target[i], p.vocab);
    total += ok;
    before += ok && i < r0;
    if (GRAD && ok) top = fmaxf(top, fabsf(p.dloss[i]));
  }
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    if (GRAD) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  }
  if (lane == 0) {
    s_before[warp] = before;
    s_total[warp] = total;
    s_max[warp] = top;
  }
  __syncthreads();
  before = total = 0;
  top = 0.0f;
  for (int w = 0; w < PACK_THREADS / 32; ++w) {
    before += s_before[w];
    total += s_total[w];
    top = fmaxf(top, s_max[w]);
  }
  if (blockIdx.x == 0 && tid == 0) {
    *p.rows.n_valid = total;
    if (GRAD) *p.rows.scale = top;
  }

  const int chunks = p.cols_pad / 8;
  for (int base = r0; base < r1; base += PACK_THREADS) {
    // places of up to 256 rows
    const int i = base + tid;
    const int32_t t = i < r1 ? p.target[i] : -1;
    const bool ok = counts(t, p.vocab);
    if (t >= p.vocab) raise_status(p.status, DSPARK_DEV_TOKEN_OOR);
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok);
    __syncthreads();
    if (lane == 0) s_before[warp] = __popc(mask);
    __syncthreads();
    int pos = before + __popc(mask & ((1u << lane) - 1u));
    int here = 0;
    for (int w = 0; w < PACK_THREADS / 32; ++w) {
      pos += w < warp ? s_before[w] : 0;
      here += s_before[w];
    }
    before += here;
    s_pos[tid] = ok ? pos : -1;
    if (i < r1) {
      p.position[i] = ok ? pos : -1;
      if (!GRAD && !ok) {
        p.loss_out[i] = 0.0f;
        p.lse_out[i] = 0.0f;
      }
    }
    if (ok) {
      int32_t pv = 0;
      if (p.rank > 0) {
        pv = p.prev[i];
        if (pv < 0 || pv >= p.vocab) {
          pv = 0;
          raise_status(p.status, DSPARK_DEV_TOKEN_OOR);
        }
      }
      p.rows.index[pos] = i;
      p.rows.target[pos] = t;
      p.rows.prev[pos] = pv;
      if (GRAD) {
        p.rows.lse2[pos] = p.lse[i] * kLog2e;
        // equal weights (a mean) become exactly 1
        p.rows.weight[pos] = top > 0.0f ? p.dloss[i] / top : p.dloss[i];
      }
    }
    __syncthreads();
    const int n = min(PACK_THREADS, r1 - base);
    for (int j = warp; j < n; j += PACK_THREADS / 32) {
      const int at = s_pos[j];
      if (at < 0) continue;
      int32_t pv = 0;
      if (p.rank > 0) {
        pv = p.prev[base + j];
        if (pv < 0 || pv >= p.vocab) pv = 0;
      }
      const uint16_t *hr = p.h + static_cast<int64_t>(base + j) * p.h_stride;
      const uint16_t *ur = p.U + static_cast<int64_t>(pv) * p.rank;
      uint16_t *ar = p.a + static_cast<int64_t>(at) * p.cols_pad;
      for (int c = lane; c < chunks; c += 32) {
        const int col = c * 8;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (col < p.d)
          v = ld_global_nc_v4(hr + col);
        else if (col >= p.d_pad && col - p.d_pad < p.rank)
          v = ld_global_nc_v4(ur + (col - p.d_pad));
        *reinterpret_cast<uint4 *>(ar + col) = v;
      }
    }
  }
  // the rows that fill up the last tile
  const int end = (total + HT - 1) / HT * HT;
  for (int j = total + blockIdx.x; j < end; j += gridDim.x) {
    uint16_t *ar = p.a + static_cast<int64_t>(j) * p.cols_pad;
    for (int c = tid; c < chunks; c += PACK_THREADS)
      *reinterpret_cast<uint4 *>(ar + c * 8) = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) {
      p.rows.target[j] = -1;
      p.rows.lse2[j] = 0.0f;
      p.rows.weight[j] = 0.0f;
    }
  }
}

// -------------------------------------------------------------- products
// Three kernels on one main loop.  A cluster of two CTAs computes a 256 x 256
// tile with tcgen05.mma.cta_group::2: each CTA stages 128 rows of either
// operand, 64 deep, and holds 128 rows of the accumulator, so an operand byte
// is read from L2 once for 256 rows of the other one.
//
//   LSE    z tile -> per row (max, sum exp) of 256 entries, and z at the target
//   PROB   z tile -> 256 x 256 of G, bf16
//   GRAD   dA tiles (G . B over a piece of the vocabulary, added up in fp32 by
//          TMA) and dB tiles (G^T . A over the rows, bf16), in one launch so
//          that the ones fill the others' last wave
//
// Both operands of z have the reduction index contiguous.  For dB neither
// has, for dA only G: there the 64 x 64 boxes are read as they lie, and the
// descriptors say that the other index is the contiguous one.
enum HeadKind { kLse = 0, kProb = 1, kGrad = 2 };

struct HeadMaps {
  CUtensorMap a;      // packed A, 64 x 64 boxes
  CUtensorMap w, v;   // W and V, 64 x 64 boxes
  CUtensorMap g;      // G, 64 x 64 boxes
  CUtensorMap g_out;  // G, 32 x 64 boxes
  CUtensorMap dw, dv; // dW and dV, 32 x 64 boxes
  CUtensorMap acc;    // fp32 sums of dA, 32 x 32 boxes
};

struct HeadParams {
  RowInfo rows;
  int32_t rows_pad, vocab;
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
  int k0, nk;   // range of the reduction, in 64-entry blocks
  int split;
};

template <int KIND>
__device__ __forceinline__ int head_tiles(const HeadParams &p, int n_valid) {
  const int mt = (n_valid + HT - 1) / HT;
  if (KIND != kGrad) return mt * p.v_tiles;
  return mt * p.d_tiles * p.splits + p.v_tiles * p.d_tiles;
}

template <int KIND>
__device__ __forceinline__ HeadTile head_tile(const HeadParams &p, int n_valid, int t) {
  const int mt = (n_valid + HT - 1) / HT;
  HeadTile x;
  x.da = 0;
  x.split = 0;
  if (KIND != kGrad) {
    x.m = (t % mt) * HT;
    x.n = (t / mt) * HT;
    x.k0 = 0;
    x.nk = p.kd + p.kr;
    return x;
  }
  const int n_da = mt * p.d_tiles * p.splits;
  if (t < n_da) {
    x.da = 1;
    x.n = (t % p.d_tiles) * HT;
    const int u = t / p.d_tiles;
    x.m = (u % mt) * HT;
    x.split = u / mt;
    const int kb = p.v_tiles * (HT / HK);
    x.k0 = static_cast<int>(static_cast<int64_t>(kb) * x.split / p.splits);
    x.nk = static_cast<int>(static_cast<int64_t>(kb) * (x.split + 1) / p.splits) - x.k0;
  } else {
    t -= n_da;
    x.n = (t % p.d_tiles) * HT;
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
          if (cta == 0) mbar_arrive_expect_tx(&full[s], 2 * H_STAGE);
          const uint32_t bar = full0 + s * 8;
          uint8_t *sa = smem + s * H_STAGE, *sb = sa + H_OPERAND;
          if (KIND != kGrad) {
            const CUtensorMap *mb = kb < p.kd ? &maps.w : &maps.v;
            const int xb = (kb < p.kd ? kb : kb - p.kd) * HK;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int r = cta * 128 + j * 64;
              tma_load_2d_pair(sa + j * H_BOX, &maps.a, bar, kb * HK, x.m + r);
              tma_load_2d_pair(sb + j * H_BOX, mb, bar, xb, p.v0 + x.n + r);
            }
          } else if (x.da) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int r = cta * 128 + j * 64;
              const int cb = (x.n + r) / HK;
              const bool in_d = cb < p.kd || p.kr == 0;
              tma_load_2d_pair(sa + j * H_BOX, &maps.g, bar, kb * HK, x.m + r);
              tma_load_2d_pair(sb + j * H_BOX, in_d ? &maps.w : &maps.v, bar,
                               (in_d ? cb : cb - p.kd) * HK, p.v0 + kb * HK);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int r = cta * 128 + j * 64;
              tma_load_2d_pair(sa + j * H_BOX, &maps.g, bar, x.m + r, kb * HK);
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
        const bool a_mn = KIND == kGrad && !x.da, b_mn = KIND == kGrad;
        const uint32_t idesc = umma_idesc_bf16_f32(HT, HT) | (a_mn ? 1u << 15 : 0u) |
                               (b_mn ? 1u << 16 : 0u);
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
#pragma unroll
          for (int kk = 0; kk < HK / 16; ++kk) {
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
      const int row = row0 + lane;
      if (KIND == kLse) {
        const int tcol = p.rows.target[row] - (p.v0 + x.n);
        const int left = p.vocab - (p.v0 + x.n);
        float m = -INFINITY, sum = 0.0f;
        for (int c0 = 0; c0 < HT; c0 += 32) {
          if (c0 >= left) break;
          uint32_t acc[32];
          tmem_ld_32x32b_x32(acc_at + c0, acc);
          tmem_ld_wait(acc);
          float z[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) z[e] = __uint_as_float(acc[e]);
          if (c0 + 32 > left) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c0 + e >= left) z[e] = -INFINITY;
          }
          if (static_cast<uint32_t>(tcol - c0) < 32u) {
            float zt = 0.0f;
#pragma unroll
            for (int e = 0; e < 32; ++e) zt = e == tcol - c0 ? z[e] : zt;
            p.rows.z_target[row] = zt;
          }
          float top = z[0];
#pragma unroll
          for (int e = 1; e < 32; ++e) top = fmaxf(top, z[e]);
          top = fmaxf(top, m);
          // a row of -infinity keeps a finite reference: its sum is 0
          const float ref = top == -INFINITY ? 0.0f : top * kLog2e;
          float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int e = 0; e < 32; ++e) part[e & 3] += ex2(fmaf(z[e], kLog2e, -ref));
          sum = fmaf(sum, ex2(fmaf(m, kLog2e, -ref)),
                     (part[0] + part[1]) + (part[2] + part[3]));
          m = top;
        }
        p.partial[static_cast<int64_t>((p.v0 + x.n) / HT) * p.rows_pad + row] =
            make_float2(m, sum);
      } else {
        const bool prob = KIND == kProb;
        const bool f32_out = KIND == kGrad && x.da;
        const int step = f32_out ? 32 : 64;   // columns of a box
        float lse2 = 0.0f, weight = 0.0f, scale = 0.0f;
        int tcol = -1, left = HT;
        if (prob) {
          lse2 = p.rows.lse2[row];
          weight = p.rows.weight[row];
          tcol = p.rows.target[row] - (p.v0 + x.n);
          left = p.vocab - (p.v0 + x.n);
        } else if (!x.da) {
          scale = *p.rows.scale;
        }
        for (int c0 = 0; c0 < HT; c0 += step, ++boxes) {
          const uint32_t box = out_addr + (boxes & 1) * H_OUT_BOX;
          if (lane == 0) bulk_wait_read<1>();  // the box's last store has read it
          __syncwarp();
          for (int half = 0; half < step; half += 32) {
            uint32_t acc[32];
            if (x.nk > 0) {
              tmem_ld_32x32b_x32(acc_at + c0 + half, acc);
              tmem_ld_wait(acc);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) acc[e] = 0u;
            }
            if (f32_out) {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                st_shared_v4(box + lane * 128 + ((c ^ (lane & 7)) << 4),
                             make_uint4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]));
              continue;
            }
            float g[32];
            if (prob) {
              const int c1 = c0 + half;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float pr = ex2(fmaf(__uint_as_float(acc[e]), kLog2e, -lse2));
                g[e] = pr * weight;
              }
              if (static_cast<uint32_t>(tcol - c1) < 32u) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (e == tcol - c1) g[e] -= weight;
              }
              if (c1 + 32 > left) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (c1 + e >= left) g[e] = 0.0f;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) g[e] = __uint_as_float(acc[e]) * scale;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint4 v = make_uint4(pack_bf16(g[8 * c], g[8 * c + 1]),
                                         pack_bf16(g[8 * c + 2], g[8 * c + 3]),
                                         pack_bf16(g[8 * c + 4], g[8 * c + 5]),
                                         pack_bf16(g[8 * c + 6], g[8 * c + 7]));
              st_shared_v4(box + lane * 128 + (((half / 8 + c) ^ (lane & 7)) << 4), v);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (prob) {
              tma_store_2d(&maps.g_out, box, x.n + c0, row0);
            } else if (x.da) {
              const int y = x.split * p.rows_pad + row0;
              if (x.n + c0 < (p.kd + p.kr) * HK) {
                if (p.first_piece)
                  tma_store_2d(&maps.acc, box, x.n + c0, y);
                else
                  tma_reduce_add_2d(&maps.acc, box, x.n + c0, y);
              }
            } else if (p.v0 + row0 < p.vocab) {
              const int col = x.n + c0;
              if (col < p.kd * HK) {
                if (col < p.d) tma_store_2d(&maps.dw, box, col, p.v0 + row0);
              } else if (col - p.kd * HK < p.rank) {
                tma_store_2d(&maps.dv, box, col - p.kd * HK, p.v0 + row0);
              }
            }
            bulk_commit();
          }
        }
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
// one vocabulary tile, 32 warps share the tiles.
constexpr int JOIN_WARPS = 32;

__global__ void __launch_bounds__(JOIN_WARPS * 32)
    head_join_kernel(const float2 *partial, int v_tiles, int rows_pad, RowInfo rows,
                     float *loss, float *lse) {
  __shared__ float2 part[JOIN_WARPS][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * 32 + lane;
  const int n_valid = *rows.n_valid;
  if (blockIdx.x * 32 >= n_valid) return;
  float m = -INFINITY, s = 0.0f;
  constexpr int U = 8;
  for (int v = warp; v < v_tiles; v += JOIN_WARPS * U) {
    float2 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = v + u * JOIN_WARPS;
      x[u] = at < v_tiles ? partial[static_cast<int64_t>(at) * rows_pad + row]
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
// dh: the splits' sums in order, times the scale, back at the row's own place;
// zero for rows without a target.
__global__ void __launch_bounds__(128)
    head_dh_kernel(const float *acc, int splits, int64_t split_stride, int cols_pad,
                   RowInfo rows, const int32_t *position, int M, int d, uint16_t *dh,
                   int64_t dh_stride) {
  const float scale = *rows.scale;
  for (int i = blockIdx.x; i < M; i += gridDim.x) {
    const int at = position[i];
    for (int c = threadIdx.x * 8; c < d; c += 128 * 8) {
      float s[8] = {};
      if (at >= 0) {
        for (int k = 0; k < splits; ++k) {
          const float *x = acc + k * split_stride + static_cast<int64_t>(at) * cols_pad + c;
          const float4 lo = *reinterpret_cast<const float4 *>(x);
          const float4 hi = *reinterpret_cast<const float4 *>(x + 4);
          s[0] += lo.x; s[1] += lo.y; s[2] += lo.z; s[3] += lo.w;
          s[4] += hi.x; s[5] += hi.y; s[6] += hi.z; s[7] += hi.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] *= scale;
      }
      *reinterpret_cast<uint4 *>(dh + static_cast<int64_t>(i) * dh_stride + c) =
          make_uint4(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]),
                     pack_bf16(s[6], s[7]));
    }
  }
}

// dU: one CTA for a counted row.  The first row with a token sums that token's
// rows in a fixed order (eight warps take consecutive eighths of the rows, and
// their sums are joined in order), so the result does not depend on the order
// in which CTAs run.  Tokens that no row names were zeroed before.
constexpr int DU_WARPS = 8;

__global__ void __launch_bounds__(DU_WARPS * 32)
    head_du_kernel(const float *acc, int splits, int64_t split_stride, int cols_pad, int d_pad,
                   RowInfo rows, int rank, uint16_t *dU) {
  __shared__ float part[DU_WARPS][32][9];
  const int n_valid = *rows.n_valid;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float scale = *rows.scale;
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
          for (int k = 0; k < splits; ++k) {
            const float *x = acc + k * split_stride + static_cast<int64_t>(i) * cols_pad + d_pad +
                             lane * 8;
            const float4 a = *reinterpret_cast<const float4 *>(x);
            const float4 b = *reinterpret_cast<const float4 *>(x + 4);
            s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
            s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
          }
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
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] *= scale;
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
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * esz};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1, 1};
  return enc(m, type, 2, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
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
  bool ok = encode_2d(&o.maps.a, bf16, 2, ws + l.a, l.cols_pad, l.rows_pad, l.cols_pad, 64, 64) &&
            encode_2d(&o.maps.w, bf16, 2, a.W, a.d, a.vocab, a.d, 64, 64) &&
            encode_2d(&o.maps.v, bf16, 2, V, vr, a.vocab, vr, 64, 64);
  if (grad) {
    ok = ok &&
         encode_2d(&o.maps.g, bf16, 2, ws + l.g, l.piece, l.rows_pad, l.piece, 64, 64) &&
         encode_2d(&o.maps.g_out, bf16, 2, ws + l.g, l.piece, l.rows_pad, l.piece, 64, 32) &&
         encode_2d(&o.maps.dw, bf16, 2, a.dW, a.d, a.vocab, a.d, 64, 32) &&
         encode_2d(&o.maps.dv, bf16, 2, a.rank ? a.dV : a.dW, vr, a.vocab, vr, 64, 32) &&
         encode_2d(&o.maps.acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, ws + l.acc, l.cols_pad,
                   l.rows_pad * l.splits, l.cols_pad, 32, 32);
  }
  if (!ok) return DSPARK_ERR_INVALID_ARG;

  HeadParams &p = o.p;
  p.rows = row_info(ws + l.rowinfo, l.rows_pad);
  p.rows_pad = static_cast<int32_t>(l.rows_pad);
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
  k.rows_per_cta = std::max<int>(8, static_cast<int>(up(a.M, o.sms * 4) / (o.sms * 4)));
  k.position = reinterpret_cast<int32_t *>(ws + l.position);
  k.a = reinterpret_cast<uint16_t *>(ws + l.a);
  k.rows = p.rows;
  k.status = p.status;
  o.pack_grid = (a.M + k.rows_per_cta - 1) / k.rows_per_cta;
  return DSPARK_OK;
}

template <int KIND>
void head_gemm(const HeadPlan &o, const HeadParams &p, cudaStream_t stream) {
  // no more pairs than tiles there can be
  const int64_t mt = o.lay.rows_pad / HT;
  const int64_t tiles = KIND == kGrad ? mt * p.d_tiles * p.splits + int64_t(p.v_tiles) * p.d_tiles
                                      : mt * p.v_tiles;
  const int pairs = static_cast<int>(std::min<int64_t>(o.sms / 2, tiles));
  head_gemm_kernel<KIND><<<pairs * 2, H_THREADS, H_SMEM, stream>>>(o.maps, p);
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
  l.position = take(static_cast<size_t>(M) * 4);
  l.a = take(static_cast<size_t>(l.rows_pad) * l.cols_pad * 2);
  const int64_t v_pad = up(vocab, HT);
  l.splits = 1;
  if (!grad) {
    l.partial = take(static_cast<size_t>(v_pad / HT) * l.rows_pad * 8);
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
  }
  l.total = at;
  return l;
}

dspark_status head_loss_launch(const HeadArgs &a, cudaStream_t stream) {
  HeadPlan o;
  const dspark_status s = head_plan(a, false, o);
  if (s != DSPARK_OK) return s;
  head_pack_kernel<false><<<o.pack_grid, PACK_THREADS, 0, stream>>>(o.pack);
  head_gemm<kLse>(o, o.p, stream);
  head_join_kernel<<<(a.M + 31) / 32, JOIN_WARPS * 32, 0, stream>>>(
      o.p.partial, o.p.v_tiles, o.p.rows_pad, o.p.rows, a.loss, a.lse);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

dspark_status head_loss_grad_launch(const HeadArgs &a, cudaStream_t stream) {
  HeadPlan o;
  const dspark_status s = head_plan(a, true, o);
  if (s != DSPARK_OK) return s;
  const HeadLayout &l = o.lay;
  if (a.rank && cudaMemsetAsync(a.dU, 0, static_cast<size_t>(a.vocab) * a.rank * 2, stream) !=
                    cudaSuccess)
    return DSPARK_ERR_CUDA;
  head_pack_kernel<true><<<o.pack_grid, PACK_THREADS, 0, stream>>>(o.pack);
  HeadParams p = o.p;
  for (int64_t v0 = 0; v0 < a.vocab; v0 += l.piece) {
    p.v0 = static_cast<int32_t>(v0);
    p.v_tiles = static_cast<int32_t>(
        (std::min<int64_t>(l.piece, a.vocab - v0) + HT - 1) / HT);
    p.first_piece = v0 == 0;
    head_gemm<kProb>(o, p, stream);
    head_gemm<kGrad>(o, p, stream);
  }
  const float *acc = reinterpret_cast<const float *>(a.workspace + l.acc);
  const int64_t stride = l.rows_pad * l.cols_pad;
  head_dh_kernel<<<std::min(a.M, 1 << 20), 128, 0, stream>>>(
      acc, l.splits, stride, static_cast<int>(l.cols_pad), p.rows, o.pack.position, a.M, a.d,
      static_cast<uint16_t *>(a.dh), a.dh_stride);
  if (a.rank)
    head_du_kernel<<<std::min(a.M, o.sms * 32), DU_WARPS * 32, 0, stream>>>(
        acc, l.splits, stride, static_cast<int>(l.cols_pad), o.pack.d_pad, p.rows, a.rank,
        static_cast<uint16_t *>(a.dU));
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // namespace dspark
