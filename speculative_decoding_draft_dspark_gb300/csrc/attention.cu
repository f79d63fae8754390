// Attention of a step's rows over the paged cache, on sm_103a.
//
// For one request, key head and block of 128 packed rows (row m = j * G + g: token j,
// query head g of the group of G that shares the key head) and the request's tokens,
// 64 at a time:
//     S = Q K^T                     tcgen05, 128 x 64, fp32 in tensor memory
//     P = exp2((S - m) c)           m: running maximum, c = scale log2 e
//     O = O + P V,  l = l + sum P   tcgen05, P in bf16 from tensor memory
// and out = O / l at the end.  O is scaled only where the maximum grew by more than
// 2^8 (P is then at most 2^8 in bf16, which has fp32's range; l is summed in fp32).
//
// Packing the group's heads into the tile's rows reads each key and value once for
// all of them.  With few rows the time is the cache's bytes: K and V tiles come by TMA
// through the block table into a ring, several tiles ahead, and two CTAs an SM hide
// each other's chain of dependent steps.
//
// Work is split by tiles of tokens, not by rows: all (request, head, block) items
// laid end to end are cut into equal runs, one a CTA, so that one long context
// occupies the whole GPU and short ones leave no tail.  A cut item leaves its O, m and
// l in the workspace and a second kernel joins them, in order.
#include <cuda_bf16.h>
#include <mutex>

#include "chain_common.cuh"
#include "launch.cuh"
#include "target_internal.h"

namespace dspark {

constexpr int AT_ROWS = 128;       // packed rows of a tile
constexpr int AT_TOKENS = 64;      // tokens of a tile
constexpr int AT_THREADS = 192;    // 4 softmax warps, TMA, MMA
constexpr int AT_MAX_CTAS = 320;   // that leave partial results
constexpr int AT_SEGS = 4;         // segments told ahead
constexpr int AT_INFOS = 8;        // tiles told ahead
constexpr float kRescale = 8.0f;   // log2 of what the maximum may grow by
// Up to this a maximum is taken off as fma(s, c, -round(m c)): whatever m c was rounded
// to is in lse too, so nothing is lost.  A larger m is taken off first, (s - m) c: at
// 2^24 and more m c would round by whole units.  Where a row passes from one form to
// the other they differ by 2^-17.
constexpr float kLarge = 256.0f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

template <int HD>
struct AtShape {
  static constexpr int kBoxes = HD / 64;                        // 64 columns each
  static constexpr int kStages = HD == 64 ? 8 : 4;
  static constexpr int kStage = kBoxes * AT_TOKENS * 128;        // bytes of a K or V tile
  static constexpr int kQ = kBoxes * AT_ROWS * 128;
  static constexpr int kCtas = HD == 256 ? 1 : 2;                // an SM
  static constexpr int kTmem = HD == 256 ? 512 : 256;            // columns: S, S, O
  static constexpr int kBytes = 1024 + kQ + kStages * kStage;    // aligned here to 1024
};

// What the joining kernel needs about an item that begins in a CTA and is cut.
struct AtMeta {
  int32_t last;    // CTA that holds its end; 0: nothing is cut here
  int32_t request, first, count, head, block;
};

struct AtParams {
  HeadRows q, out;
  const int32_t *block_table;
  int64_t table_stride;
  const int32_t *ctx_len, *cu_rows;
  const uint64_t *tree;
  const __nv_bfloat16 *v_cache;
  int64_t page_stride, token_stride, head_stride;
  int32_t tree_width, N, R, max_len, Hk, group, d;
  int32_t page_shift, num_pages, max_pages, least_tiles, tile_rows;
  float scale_log2;
  float *lse;
  uint32_t *status;
  AtMeta *meta;
  float2 *part_ml;  // [2 AT_MAX_CTAS][tile_rows]: maximum, sum
  float *part_o;    // [2 AT_MAX_CTAS][tile_rows][HD]
};

// A run of an item's tiles that one CTA computes.
struct AtSeg {
  int32_t request, first, count, ctx, head, block;  // request < 0: the end
  int32_t t0, t1, tiles;                            // of the item's tiles
  int32_t tree, end;                                // tokens [0, end)
  int32_t part;                                     // slot of its partial result, or -1
};

// ------------------------------------------------------------ instructions
__device__ __forceinline__ uint32_t at_elect() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one;
}

// a box of 64 columns of one head: tokens of one page
__device__ __forceinline__ void tma_load_page(uint32_t one, uint32_t dst, const CUtensorMap *m,
                                              uint64_t *bar, int32_t column, int32_t head,
                                              int32_t token, int32_t page) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %7, 0;\n\t"
      "@p cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(column), "r"(head), "r"(token),
      "r"(page), "r"(one)
      : "memory");
}

// D (+)= A B^T, A and B in shared memory; the descriptors' upper halves are alike
__device__ __forceinline__ void umma_ss(uint32_t one, uint32_t d_tmem, uint32_t a_lo,
                                        uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
// the same with A in tensor memory: a lane a row, two bf16 a column
__device__ __forceinline__ void umma_ts(uint32_t one, uint32_t d_tmem, uint32_t a_tmem,
                                        uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void umma_commit_one(uint32_t one, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(one)
      : "memory");
}

// 32 registers a lane to 32 columns of the warp's lanes of tensor memory
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, "
      "%31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2 of what a sum's terms carry for a maximum, and its difference for two of them
__device__ __forceinline__ float at_base(float m, float c) {
  return m == -INFINITY ? 0.0f : __fmul_rn(m, c);
}
__device__ __forceinline__ float at_difference(float m, float above, float c) {
  const float a = __fmul_rn(m, c), b = __fmul_rn(above, c);
  return fabsf(a) > kLarge || fabsf(b) > kLarge ? (m - above) * c : a - b;
}

// Matrix descriptors with 128-byte swizzle, in halves (see common.cuh): K-major rows
// of 64 columns; for V, whose rows run along the product's columns, boxes of 64 x 64.
constexpr uint32_t kAtDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t at_desc_k(uint32_t addr) {
  return ((addr & 0x3FFFFu) >> 4) | 1u << 16;
}
__device__ __forceinline__ uint32_t at_desc_mn(uint32_t addr) {
  return ((addr & 0x3FFFFu) >> 4) | static_cast<uint32_t>(AT_TOKENS * 128 >> 4) << 16;
}

// ----------------------------------------------------------------- planning
__device__ __forceinline__ int at_blocks(const AtParams &p, int count) {
  return (count * p.group + AT_ROWS - 1) / AT_ROWS;
}
// Tokens that some row of a block attends, as an end: those in the cache and the
// step's, up to the block's last row where the request is a chain.
__device__ __forceinline__ int at_end(const AtParams &p, int ctx, int count, bool tree, int b) {
  const int last = tree ? count : min(count, ((b + 1) * AT_ROWS - 1) / p.group + 1);
  const int64_t end = static_cast<int64_t>(ctx) + last;
  return static_cast<int>(min(end, static_cast<int64_t>(p.max_pages) << p.page_shift));
}
__device__ __forceinline__ int at_tiles(int end) { return (end + AT_TOKENS - 1) / AT_TOKENS; }

struct AtRequest {
  int first, count, ctx;
  bool tree;
};
__device__ __forceinline__ AtRequest at_request(const AtParams &p, int n) {
  AtRequest r;
  const RowSpan rows = row_span(p.cu_rows, n, p.R);
  r.first = rows.first;
  r.count = min(rows.count, p.max_len);
  r.ctx = max(p.ctx_len[n], 0);
  r.tree = is_tree(p.tree, p.tree_width, n, rows.count);
  return r;
}
__device__ __forceinline__ int64_t at_units(const AtParams &p, const AtRequest &r) {
  int64_t sum = 0;
  const int blocks = at_blocks(p, r.count);
  for (int b = 0; b < blocks; ++b) sum += at_tiles(at_end(p, r.ctx, r.count, r.tree, b));
  return sum * p.Hk;
}

// The CTAs' shares of U units: every CTA has at least `least_tiles` or the rest.
struct AtShares {
  int64_t units;
  int ctas;
  __device__ __forceinline__ int64_t begin(int c) const { return units * c / ctas; }
};

// Shared state besides the tiles
template <int HD>
struct AtShared {
  uint64_t full[AtShape<HD>::kStages], empty[AtShape<HD>::kStages];
  uint64_t s_full[2], p_full[2], pv_done[2], q_full, scanned;  // pairs: by tile, in turn
  uint64_t seg_full[AT_SEGS], seg_empty[AT_SEGS];
  uint64_t info_full[AT_INFOS];
  uint64_t valid[AT_INFOS];        // a tile's tokens that are there
  uint64_t poison[2][4][3];        // tokens whose values are not finite: warp, tile
  AtSeg seg[AT_SEGS];
  int64_t scan[AT_THREADS / 32];
  int64_t start_rest;
  int32_t start_request;
  uint32_t tmem, abort;
};

template <int HD>
__global__ void __launch_bounds__(AT_THREADS, AtShape<HD>::kCtas)
    attention_kernel(const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const AtParams p) {
  using Sh = AtShape<HD>;
  extern __shared__ uint8_t at_raw[];
  __shared__ AtShared<HD> sh;
  uint8_t *smem = at_raw + ((1024u - (smem_u32(at_raw) & 1023u)) & 1023u);
  uint8_t *ring = smem + Sh::kQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile uint32_t *abort_flag = &sh.abort;

  if (tid == 0) {
    for (int i = 0; i < Sh::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.pv_done[i], 1);
    }
    mbar_init(&sh.q_full, 4);
    mbar_init(&sh.scanned, 4);
    for (int i = 0; i < AT_SEGS; ++i) {
      mbar_init(&sh.seg_full[i], 1);
      mbar_init(&sh.seg_empty[i], 5);
    }
    for (int i = 0; i < AT_INFOS; ++i) mbar_init(&sh.info_full[i], 1);
    sh.abort = 0u;
    sh.start_request = -1;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 5) {
    tmem_alloc(&sh.tmem, Sh::kTmem);
    tmem_relinquish();
  }
  if (tid == 128) {
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  wait_for_earlier_kernel();
  allow_next_kernel();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int cta = static_cast<int>(blockIdx.x);

  // ---- plan: this CTA's run of units, and the request that it begins in
  AtShares shares;
  {
    const int C = (p.N + AT_THREADS - 1) / AT_THREADS;
    const int n0 = min(p.N, tid * C), n1 = min(p.N, n0 + C);
    int64_t mine = 0;
    for (int n = n0; n < n1; ++n) {
      const AtRequest r = at_request(p, n);
      if (cta == 0) {
        if (row_span(p.cu_rows, n, p.R).count > p.max_len)
          raise_status(p.status, DSPARK_DEV_LEN_OOR);
        if (r.count > 0 && static_cast<int64_t>(r.ctx) + r.count >
                               static_cast<int64_t>(p.max_pages) << p.page_shift)
          raise_status(p.status, DSPARK_DEV_PAGE_OOR);
      }
      mine += at_units(p, r);
    }
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh.scan[warp] = x;
    __syncthreads();
    int64_t before = x - mine, total = 0;
    for (int w = 0; w < AT_THREADS / 32; ++w) {
      if (w < warp) before += sh.scan[w];
      total += sh.scan[w];
    }
    shares.units = total;
    shares.ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x),
                                       (total + p.least_tiles - 1) / p.least_tiles));
    if (cta < shares.ctas) {
      int64_t rest = shares.begin(cta) - before;
      if (rest >= 0 && rest < mine) {
        for (int n = n0; n < n1; ++n) {
          const int64_t units = at_units(p, at_request(p, n));
          if (rest < units) {
            sh.start_request = n;
            sh.start_rest = rest;
            break;
          }
          rest -= units;
        }
      }
    }
    __syncthreads();
  }

  if (warp == 4) {
    // ------------------------------------------------------------ K and V
    const uint32_t one = at_elect();
    const int rows_box = min(1 << p.page_shift, AT_TOKENS);
    const int boxes = AT_TOKENS / rows_box;
    bool ok = true;
    int it = 0, infos = 0, segs = 0;
    AtMeta meta = {};
    auto place = [&](const AtSeg &s) {
      const int i = segs % AT_SEGS;
      ok = __all_sync(0xFFFFFFFFu, wait_bounded(&sh.seg_empty[i], ((segs / AT_SEGS) & 1) ^ 1u,
                                                abort_flag, p.status));
      if (ok && one) {
        sh.seg[i] = s;
        mbar_arrive(&sh.seg_full[i]);
      }
      ++segs;
    };
    if (cta < shares.ctas) {
      const int64_t end_unit = shares.begin(cta + 1);
      int64_t unit = shares.begin(cta);
      int n = sh.start_request;
      int64_t rest = sh.start_rest;
      while (ok && unit < end_unit && n < p.N) {
        const AtRequest r = at_request(p, n);
        const int blocks = at_blocks(p, r.count);
        // the items before the first one of this run
        int64_t a_head = 0;
        for (int b = 0; b < blocks; ++b) a_head += at_tiles(at_end(p, r.ctx, r.count, r.tree, b));
        int h = a_head > 0 ? static_cast<int>(rest / a_head) : p.Hk;
        rest -= h * a_head;
        int b = 0;
        while (b < blocks && h < p.Hk) {
          const int t = at_tiles(at_end(p, r.ctx, r.count, r.tree, b));
          if (rest < t) break;
          rest -= t;
          ++b;
        }
        for (; ok && h < p.Hk && unit < end_unit; ++h, b = 0) {
          for (; ok && b < blocks && unit < end_unit; ++b) {
            AtSeg s;
            s.request = n;
            s.first = r.first;
            s.count = r.count;
            s.ctx = r.ctx;
            s.head = h;
            s.block = b;
            s.tree = r.tree;
            s.end = at_end(p, r.ctx, r.count, r.tree, b);
            s.tiles = at_tiles(s.end);
            s.t0 = static_cast<int>(rest);
            s.t1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), rest + (end_unit - unit)));
            rest = 0;
            unit += s.t1 - s.t0;
            s.part = -1;
            if (s.t0 > 0) {
              s.part = 2 * cta;
            } else if (s.t1 < s.tiles) {
              s.part = 2 * cta + 1;
              const int64_t last_unit = unit + (s.tiles - s.t1) - 1;
              int c = static_cast<int>(last_unit * shares.ctas / shares.units);
              while (c + 1 < shares.ctas && shares.begin(c + 1) <= last_unit) ++c;
              while (shares.begin(c) > last_unit) --c;
              meta = {c, n, s.first, s.count, h, b};
            }
            place(s);
            if (!ok) break;
            // its tiles: K 0, K 1, V 0, K 2, V 1, ... as the products take them
            const int64_t table = static_cast<int64_t>(n) * p.table_stride;
            int base[2] = {-1, -1}, ids[2];
            const int T = s.t1 - s.t0;
            for (int x = 0; ok && x < 2 * T; ++x) {
              const bool is_v = x == 2 * T - 1 || (x > 1 && (x & 1) == 0);
              const int tile = s.t0 + (is_v ? (x == 2 * T - 1 ? T - 1 : x / 2 - 1) : (x + 1) / 2);
              const int token = tile * AT_TOKENS;
              const int stage = it % Sh::kStages;
              // pages of this and the following tiles, a lane each
              const int page0 = token >> p.page_shift, want = page0 & ~31;
              if (base[is_v] != want) {
                base[is_v] = want;
                const int k = want + lane;
                ids[is_v] = k < p.max_pages ? p.block_table[table + k] : -1;
              }
              ok = __all_sync(0xFFFFFFFFu,
                              wait_bounded(&sh.empty[stage], ((it / Sh::kStages) & 1) ^ 1u,
                                           abort_flag, p.status));
              if (!ok) break;
              uint64_t there = 0ull;
              int here[4], n_here = 0;
              for (int k = 0; k < boxes; ++k) {
                const int id = __shfl_sync(0xFFFFFFFFu, ids[is_v],
                                           ((token + k * rows_box) >> p.page_shift) & 31);
                const bool good = id >= 0 && id < p.num_pages && token + k * rows_box < s.end;
                here[k] = good ? id : -1;
                n_here += good;
                if (good) there |= low_bits(rows_box) << (k * rows_box);
                if (!good && token + k * rows_box < s.end && one)
                  raise_status(p.status, DSPARK_DEV_PAGE_OOR);
              }
              if (!is_v) {
                if (one) {
                  sh.valid[infos % AT_INFOS] = there & low_bits(s.end - token);
                  mbar_arrive(&sh.info_full[infos % AT_INFOS]);
                }
                ++infos;
              }
              if (one)
                mbar_arrive_expect_tx(&sh.full[stage],
                                      static_cast<uint32_t>(n_here * Sh::kBoxes * rows_box * 128));
              __syncwarp();
              const uint32_t dst = smem_u32(ring + stage * Sh::kStage);
              for (int k = 0; k < boxes; ++k) {
                if (here[k] < 0) continue;
#pragma unroll
                for (int c = 0; c < Sh::kBoxes; ++c)
                  tma_load_page(one, dst + c * (AT_TOKENS * 128) + k * rows_box * 128,
                                is_v ? &v_map : &k_map, &sh.full[stage], c * 64, h,
                                token & ((1 << p.page_shift) - 1), here[k]);
              }
              ++it;
            }
          }
        }
        ++n;
        rest = 0;
      }
    }
    if (ok) {
      AtSeg s = {};
      s.request = -1;
      place(s);
    }
    if (one) p.meta[cta] = meta;
    if (!ok) {
      // copies in flight land before the shared memory is given back
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 20000000ull) __nanosleep(1000);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------ products
    const uint32_t one = at_elect();
    const uint32_t q_lo = at_desc_k(smem_u32(smem)), ring0 = smem_u32(ring);
    constexpr uint32_t idesc_s = umma_idesc_bf16_f32(AT_ROWS, AT_TOKENS);
    constexpr uint32_t idesc_o = umma_idesc_bf16_f32(AT_ROWS, HD) | 1u << 16;
    bool ok = true;
    int it = 0, gi = 0, segs = 0;  // ring, tiles, segments so far
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      ok = ok && __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, abort_flag, p.status));
      tc_fence_after();
      return ok;
    };
    while (ok) {
      const int si = segs % AT_SEGS;
      if (!wait(&sh.seg_full[si], (segs / AT_SEGS) & 1)) break;
      const int request = sh.seg[si].request, T = sh.seg[si].t1 - sh.seg[si].t0;
      __syncwarp();
      if (one) mbar_arrive(&sh.seg_empty[si]);
      if (request < 0) break;
      if (!wait(&sh.q_full, segs & 1)) break;
      ++segs;
      auto score = [&](int i) {
        // the buffer's last P has been multiplied
        const int g = gi + i;
        if (g >= 2 && !wait(&sh.pv_done[g & 1], ((g >> 1) - 1) & 1)) return;
        const int stage = it % Sh::kStages;
        if (!wait(&sh.full[stage], (it / Sh::kStages) & 1)) return;
        const uint32_t k_lo = at_desc_k(ring0 + stage * Sh::kStage);
        const uint32_t d = tmem + (g & 1) * AT_TOKENS;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          umma_ss(one, d, q_lo + (kk / 4) * (AT_ROWS * 128 >> 4) + (kk % 4) * 2,
                  k_lo + (kk / 4) * (AT_TOKENS * 128 >> 4) + (kk % 4) * 2, kAtDescHi, idesc_s, kk);
        umma_commit_one(one, &sh.empty[stage]);
        umma_commit_one(one, &sh.s_full[g & 1]);
        ++it;
      };
      score(0);
      for (int i = 0; ok && i < T; ++i) {
        if (i + 1 < T) score(i + 1);
        const int g = gi + i;
        if (!ok || !wait(&sh.p_full[g & 1], (g >> 1) & 1)) break;
        const int stage = it % Sh::kStages;
        if (!wait(&sh.full[stage], (it / Sh::kStages) & 1)) break;
        const uint32_t v_lo = at_desc_mn(ring0 + stage * Sh::kStage);
        const uint32_t a = tmem + (g & 1) * AT_TOKENS, d = tmem + 2 * AT_TOKENS;
#pragma unroll
        for (int kk = 0; kk < AT_TOKENS / 16; ++kk)
          umma_ts(one, d, a + kk * 8, v_lo + kk * 128, kAtDescHi, idesc_o, i | kk);
        umma_commit_one(one, &sh.empty[stage]);
        umma_commit_one(one, &sh.pv_done[g & 1]);
        ++it;
      }
      gi += T;
    }
    if (!ok) {
      // products in flight end before their memory is given back
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 20000000ull) __nanosleep(1000);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t o_tmem = tmem + lanes + 2 * AT_TOKENS;
    const int row = warp * 32 + lane;
    const float c = p.scale_log2;
    bool ok = true;
    int it = 0, gi = 0, segs = 0, scans = 0;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      ok = ok && __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, abort_flag, p.status));
      return ok;
    };
    while (ok) {
      const int si = segs % AT_SEGS;
      if (!wait(&sh.seg_full[si], (segs / AT_SEGS) & 1)) break;
      const AtSeg s = sh.seg[si];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.seg_empty[si]);
      if (s.request < 0) break;
      const int T = s.t1 - s.t0;
      const int m = s.block * AT_ROWS + row, j = m / p.group;
      const int head = s.head * p.group + (m - j * p.group);
      const bool mine = j < s.count;
      const bool any = __any_sync(0xFFFFFFFFu, mine);
      const int64_t q_row = s.first + j;
      // ---- Q: each thread its row
      if (mine) {
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q.p) +
                                   q_row * p.q.stride + head * p.q.head_stride;
        const uint32_t dst = smem_u32(smem) + row * 128;
#pragma unroll 4
        for (int c = 0; c < HD / 8; ++c) {
          const uint32_t at = dst + (c / 8) * (AT_ROWS * 128) + (((c & 7) ^ (row & 7)) << 4);
          if (c * 8 < p.d) cp_async_16(at, src + c * 8);
          else st_shared_zero16(at);
        }
        cp_async_wait_all();
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);

      // ---- tokens
      const uint64_t bits =
          s.tree && mine ? tree_bits(p.tree, p.tree_width, s.request, j, s.count) : 0ull;
      const int first_j = s.block * AT_ROWS / p.group;
      // before this token every row attends every token
      const int common = s.ctx + (s.tree ? 0 : first_j + 1);
      uint64_t(&poison)[4][3] = sh.poison[segs & 1];
      if (lane < 3) poison[warp][lane] = 0ull;
      __syncwarp();
      const bool scans_here = s.t1 * AT_TOKENS > common;
      float top = -INFINITY, sum = 0.0f;
      for (int i = 0; i < T; ++i) {
        const int g = gi + i, tile = s.t0 + i, token = tile * AT_TOKENS;
        if (!wait(&sh.info_full[g % AT_INFOS], (g / AT_INFOS) & 1)) break;
        const uint64_t valid = sh.valid[g % AT_INFOS];
        const bool inner = token + AT_TOKENS <= common;
        if (!wait(&sh.s_full[g & 1], (g >> 1) & 1)) break;
        tc_fence_after();
        if (any) {
          uint32_t s0[32], s1[32];
          const uint32_t s_tmem = tmem + lanes + (g & 1) * AT_TOKENS;
          tmem_ld_32x32b_x32(s_tmem, s0);
          tmem_ld_32x32b_x32(s_tmem + 32, s1);
          tmem_ld_wait(s0);
          tmem_ld_wait(s1);
          if (!inner || valid != ~0ull) {
            uint64_t seen;
            if (s.tree) {
              const int shift = s.ctx - token;
              seen = low_bits(shift);
              if (shift >= 0 && shift < 64) seen |= bits << shift;
              else if (shift < 0 && shift > -64) seen |= bits >> -shift;
            } else {
              seen = low_bits(s.ctx + j + 1 - token);
            }
            seen &= valid;
            const uint32_t lo = static_cast<uint32_t>(seen), hi = static_cast<uint32_t>(seen >> 32);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              s0[e] = (lo >> e & 1u) ? s0[e] : 0xFF800000u;
              s1[e] = (hi >> e & 1u) ? s1[e] : 0xFF800000u;
            }
          }
          float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            t0 = fmaxf(t0, __uint_as_float(s0[e]));
            t1 = fmaxf(t1, __uint_as_float(s1[e]));
          }
          const float high = fmaxf(t0, t1);
          const bool grow =
              mine && ((high - top) * c > kRescale || (top == -INFINITY && high > top));
          if (__any_sync(0xFFFFFFFFu, grow)) {
            const float by = grow ? exp2_approx(at_difference(top, high, c)) : 1.0f;
            if (grow) {
              top = high;
              sum *= by;
            }
            __syncwarp();
            if (i > 0) {
              // O holds the tiles before once their product is through
              if (!wait(&sh.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1)) break;
              tc_fence_after();
#pragma unroll
              for (int at = 0; at < HD; at += 32) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(o_tmem + at, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
                tmem_st_32x32b_x32(o_tmem + at, o);
              }
              tmem_st_wait();
            }
          }
          const float m = top == -INFINITY ? 0.0f : top;
          float base = __fmul_rn(m, c);
          const bool large = fabsf(base) > kLarge;
          if (__any_sync(0xFFFFFFFFu, large)) {
            const float off = large ? m : 0.0f;  // a row's bits are its own affair
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              s0[e] = __float_as_uint(__uint_as_float(s0[e]) - off);
              s1[e] = __float_as_uint(__uint_as_float(s1[e]) - off);
            }
            if (large) base = 0.0f;
          }
          uint32_t pk[32];
          float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t(&x)[32] = e < 16 ? s0 : s1;
            const float a = exp2_approx(fmaf(__uint_as_float(x[(2 * e) & 31]), c, -base));
            const float b = exp2_approx(fmaf(__uint_as_float(x[(2 * e + 1) & 31]), c, -base));
            l0 += a;
            l1 += b;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pk[e]) : "f"(b), "f"(a));
          }
          sum += l0 + l1;
          tmem_st_32x32b_x32(s_tmem, pk);
          tmem_st_wait();
          tc_fence_before();
        }
        // ---- values of tokens that are not there are 0, and those that are not
        // finite where not every row attends them: 0 times them would be NaN
        if (valid != ~0ull || !inner) {
          const int x = it + (i < T - 1 ? 2 * i + 2 : 2 * T - 1);
          const int stage = x % Sh::kStages;
          if (!wait(&sh.full[stage], (x / Sh::kStages) & 1)) break;
          const uint32_t v = smem_u32(ring + stage * Sh::kStage);
          uint32_t bad = 0u;
          for (int k = lane; k < 16 * (HD / 8); k += 32) {
            const int r = k / (HD / 8), c = k - r * (HD / 8), tr = warp * 16 + r;
            const uint32_t at = v + (c / 8) * (AT_TOKENS * 128) + tr * 128 + ((c & 7) << 4);
            if ((valid >> tr & 1ull) == 0ull) {
              st_shared_zero16(at);
            } else if (!inner) {
              uint4 w = ld_shared_v4(at);
              uint32_t *e = &w.x;
              bool found = false;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if ((e[q] & 0x7F80u) == 0x7F80u) {
                  e[q] &= 0xFFFF0000u;
                  found = true;
                }
                if ((e[q] & 0x7F800000u) == 0x7F800000u) {
                  e[q] &= 0xFFFFu;
                  found = true;
                }
              }
              if (found) {
                st_shared_v4(at, w);
                bad |= 1u << r;
              }
            }
          }
          bad = __reduce_or_sync(0xFFFFFFFFu, bad);
          if (!inner && lane == 0)
            poison[warp][tile - common / AT_TOKENS] = static_cast<uint64_t>(bad) << (warp * 16);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[g & 1]);
      }
      if (!ok) break;
      gi += T;
      it += 2 * T;
      if (scans_here) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.scanned);
        if (!wait(&sh.scanned, scans & 1)) break;
        ++scans;
      }
      // ---- the item's rows, or what is to be joined
      if (!wait(&sh.pv_done[(gi - 1) & 1], ((gi - 1) >> 1) & 1)) break;
      tc_fence_after();
      uint64_t nonfinite[3] = {0ull, 0ull, 0ull};
      if (scans_here) {
        for (int k = 0; k < 3; ++k) {
          const int token = (common / AT_TOKENS + k) * AT_TOKENS;
          uint64_t x = poison[0][k] | poison[1][k] | poison[2][k] | poison[3][k];
          if (s.tree) {
            const int shift = s.ctx - token;
            uint64_t seen = low_bits(shift);
            if (shift >= 0 && shift < 64) seen |= bits << shift;
            else if (shift < 0 && shift > -64) seen |= bits >> -shift;
            x &= seen;
          } else {
            x &= low_bits(s.ctx + j + 1 - token);
          }
          nonfinite[k] = x;
        }
      }
      if (any) {
        const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(o_tmem + c, o);
          tmem_ld_wait(o);
          if (mine && c < p.d) {
          if ((nonfinite[0] | nonfinite[1] | nonfinite[2]) != 0ull) {
            for (int k = 0; k < 3; ++k) {
              for (uint64_t x = nonfinite[k]; x != 0ull; x &= x - 1ull) {
                const int token = (common / AT_TOKENS + k) * AT_TOKENS + __ffsll(x) - 1;
                const int id = p.block_table[s.request * p.table_stride + (token >> p.page_shift)];
                const __nv_bfloat16 *v =
                    p.v_cache + id * p.page_stride +
                    (token & ((1 << p.page_shift) - 1)) * p.token_stride +
                    s.head * p.head_stride;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  if (c + e < p.d) {
                    const float f = __bfloat162float(v[c + e]);
                    if (!(fabsf(f) < INFINITY))
                      o[e] = __float_as_uint(__uint_as_float(o[e]) + f);
                  }
                }
              }
            }
          }
          if (s.part < 0) {
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out.p) + q_row * p.out.stride +
                                 head * p.out.head_stride + c;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              if (c + e >= p.d) break;
              uint4 w;
              uint32_t *u = &w.x;
#pragma unroll
              for (int q = 0; q < 4; ++q)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                    : "=r"(u[q])
                    : "f"(__uint_as_float(o[e + 2 * q + 1]) * by),
                      "f"(__uint_as_float(o[e + 2 * q]) * by));
              *reinterpret_cast<uint4 *>(dst + e) = w;
            }
          } else {
            float *dst =
                p.part_o + (static_cast<int64_t>(s.part) * p.tile_rows + row) * HD + c;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4 *>(dst + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          }
          __syncwarp();
        }
        if (mine && s.part >= 0)
          p.part_ml[static_cast<int64_t>(s.part) * p.tile_rows + row] = make_float2(top, sum);
        else if (mine && p.lse != nullptr)
          p.lse[q_row * (p.Hk * p.group) + head] =
              sum == 0.0f ? -INFINITY : at_base(top, c) * kLn2 + logf(sum);
      }
      tc_fence_before();
      ++segs;
    }
  }
  if (lane == 0 && *abort_flag) raise_status(p.status, DSPARK_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, Sh::kTmem);
}

// Joins the pieces of the items that were cut: a warp a row.
template <int HD>
__global__ void __launch_bounds__(256) attention_join_kernel(const AtParams p) {
  wait_for_earlier_kernel();
  const int cta = static_cast<int>(blockIdx.x), lane = threadIdx.x & 31;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
  const AtMeta meta = p.meta[cta];
  const int m = meta.block * AT_ROWS + row, j = m / p.group;
  if (meta.last == 0 || row >= AT_ROWS || j >= meta.count) return;
  const int head = meta.head * p.group + (m - j * p.group);
  const int pieces = meta.last - cta + 1;
  // the first piece is in the CTA's second slot, the others in first ones
  auto slot = [&](int k) {
    return (static_cast<int64_t>(k == 0 ? 2 * cta + 1 : 2 * (cta + k))) * p.tile_rows + row;
  };
  float top = -INFINITY;
  for (int k = lane; k < pieces; k += 32) top = fmaxf(top, p.part_ml[slot(k)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const float above = top == -INFINITY ? 0.0f : top;
  constexpr int E = HD / 32;
  float acc[E] = {}, sum = 0.0f;
  for (int k = 0; k < pieces; ++k) {
    const float2 ml = p.part_ml[slot(k)];
    const float w = exp2_approx(at_difference(ml.x, above, p.scale_log2));
    const float *o = p.part_o + slot(k) * HD + lane * E;
    sum = fmaf(w, ml.y, sum);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 v = *reinterpret_cast<const float2 *>(o + e);
      acc[e] = fmaf(w, v.x, acc[e]);
      acc[e + 1] = fmaf(w, v.y, acc[e + 1]);
    }
  }
  const int64_t q_row = meta.first + j;
  const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
  __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out.p) + q_row * p.out.stride +
                       head * p.out.head_stride + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    if (lane * E + e < p.d) {
      uint32_t w;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(acc[e + 1] * by), "f"(acc[e] * by));
      *reinterpret_cast<uint32_t *>(dst + e) = w;
    }
  if (lane == 0 && p.lse != nullptr)
    p.lse[q_row * (p.Hk * p.group) + head] =
        sum == 0.0f ? -INFINITY : at_base(top, p.scale_log2) * kLn2 + logf(sum);
}

// ==========================================================================
// host side
// ==========================================================================
static int padded_head(int32_t d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
static int tile_rows(int32_t max_len, int32_t group) {
  return static_cast<int>(
      std::min<int64_t>(AT_ROWS, (static_cast<int64_t>(max_len) * group + 7) / 8 * 8));
}
constexpr size_t kAtMetaOffset = 256;
constexpr size_t kAtPartOffset = kAtMetaOffset + (AT_MAX_CTAS * sizeof(AtMeta) + 255) / 256 * 256;

size_t attention_workspace_bytes(int32_t max_len, int32_t Hq, int32_t Hk, int32_t d) {
  return kAtPartOffset + static_cast<size_t>(2 * AT_MAX_CTAS) * tile_rows(max_len, Hq / Hk) *
                             (8 + 4 * static_cast<size_t>(padded_head(d)));
}

static std::mutex g_at_mu;
static bool g_at_attr[3][128];

static bool encode_cache(EncodeTiledFn enc, CUtensorMap *map, const void *p,
                         const AttentionArgs &a) {
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.d), static_cast<cuuint64_t>(a.Hk),
                        static_cast<cuuint64_t>(1) << a.page_shift,
                        static_cast<cuuint64_t>(a.num_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.head_stride) * 2,
                           static_cast<cuuint64_t>(a.token_stride) * 2,
                           static_cast<cuuint64_t>(a.page_stride) * 2};
  cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(std::min(1 << a.page_shift, AT_TOKENS)), 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <int HD>
static dspark_status launch(const AttentionArgs &a, int which, int dev, int sms,
                            cudaStream_t stream) {
  using Sh = AtShape<HD>;
  {
    std::lock_guard<std::mutex> lk(g_at_mu);
    if (!g_at_attr[which][dev]) {
      if (cudaFuncSetAttribute(attention_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Sh::kBytes) != cudaSuccess)
        return DSPARK_ERR_CUDA;
      g_at_attr[which][dev] = true;
    }
  }
  EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return DSPARK_ERR_CUDA;
  CUtensorMap k_map, v_map;
  if (!encode_cache(enc, &k_map, a.k_cache, a) || !encode_cache(enc, &v_map, a.v_cache, a))
    return DSPARK_ERR_INVALID_ARG;
  AtParams p = {};
  p.q = a.q;
  p.out = a.out;
  p.block_table = a.block_table;
  p.table_stride = a.table_stride;
  p.ctx_len = a.ctx_len;
  p.cu_rows = a.cu_rows;
  p.tree = a.tree;
  p.v_cache = static_cast<const __nv_bfloat16 *>(a.v_cache);
  p.page_stride = a.page_stride;
  p.token_stride = a.token_stride;
  p.head_stride = a.head_stride;
  p.tree_width = a.tree_width;
  p.N = a.N;
  p.R = a.R;
  p.max_len = a.max_len;
  p.Hk = a.Hk;
  p.group = a.Hq / a.Hk;
  p.d = a.d;
  p.page_shift = a.page_shift;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.least_tiles = 4;
  p.tile_rows = tile_rows(a.max_len, p.group);
  p.scale_log2 = a.scale * kLog2e;
  p.lse = a.lse;
  p.status = reinterpret_cast<uint32_t *>(a.workspace);
  p.meta = reinterpret_cast<AtMeta *>(a.workspace + kAtMetaOffset);
  p.part_o = reinterpret_cast<float *>(a.workspace + kAtPartOffset);
  p.part_ml = reinterpret_cast<float2 *>(
      p.part_o + static_cast<size_t>(2 * AT_MAX_CTAS) * p.tile_rows * HD);
  const int grid = std::min(AT_MAX_CTAS, Sh::kCtas * sms);
  if (launch_overlapped(attention_kernel<HD>, dim3(grid), dim3(AT_THREADS), Sh::kBytes, stream,
                        k_map, v_map, p) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  return launch_overlapped(attention_join_kernel<HD>, dim3(grid, (p.tile_rows + 7) / 8),
                           dim3(256), 0, stream, p) == cudaSuccess
             ? DSPARK_OK
             : DSPARK_ERR_CUDA;
}

dspark_status attention_launch(const AttentionArgs &a, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return DSPARK_ERR_CUDA;
  const int sms = device_sm_count(dev);
  if (sms <= 0) return DSPARK_ERR_CUDA;
  switch (padded_head(a.d)) {
    case 64:
      return launch<64>(a, 0, dev, sms, stream);
    case 128:
      return launch<128>(a, 1, dev, sms, stream);
    default:
      return launch<256>(a, 2, dev, sms, stream);
  }
}

}  // namespace dspark
