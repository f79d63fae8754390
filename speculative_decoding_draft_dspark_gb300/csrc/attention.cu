// Attention of a step's rows over the paged cache, on sm_103a.
//
// For one request, key head and block of packed rows (row m = j * G + g: token j, query
// head g of the group of G that shares the key head) and the request's tokens, a tile
// at a time:
//     S = Q K^T                     tcgen05, fp32 in tensor memory
//     P = exp2((S - m) c)           m: running maximum, c = scale log2 e
//     O = O + P V,  l = l + sum P   tcgen05, P in bf16 from tensor memory
// and out = O / l at the end.  O is scaled only where the maximum grew by more than
// 2^8 (P is then at most 2^8 in bf16, which has fp32's range; l is summed in fp32).
//
// Packing the group's heads into the tile's rows reads each key and value once for
// all of them.  Two kernels:
//
//   narrow: 128 rows, 64 tokens.  With few rows the time is the cache's bytes: K and V
//   tiles come by TMA through the block table into rings, several tiles ahead, the
//   scores of the next tile are computed during the softmax of this one, and two CTAs
//   an SM hide each other's chain of dependent steps.
//
//   wide: 2 x 128 rows, 128 tokens, for requests with more than 128 packed rows.  The
//   time is the tensor cores' and the operands' way into the SM: two blocks of rows
//   share each K and V tile, and one's softmax runs beside the other's products.
//
// Work is split by tiles of tokens, not by rows: all (request, head, block) items
// laid end to end are cut into equal runs, one a CTA, so that one long context
// occupies the whole GPU and short ones leave no tail.  An item counts as some tiles
// more than it has, for its queries' way in and its results' way out (prompts: 826 us
// where it counts none, 490 at four).  A cut item leaves its O, m and l in the
// workspace and a last kernel joins them, in order.
//
// Warps: softmax (a lane a row), then one each for K (which also walks the work and
// tells the others), for V, for the products, and one that looks V over.
//
// Measured on a GB300, 32 query heads, 8 key heads, 128 columns: 64 requests x 8 rows
// over up to 8192 tokens 180-184 us, 5.9-6.0 TB/s, 0.87-0.89 of measured HBM.  One token
// over 8192: 22 us, of which the cache's bytes are 5; starting, planning and joining are
// chains of dependent loads.  16 chunks of 512 rows: 477-500 us, 1.10-1.15 PFLOP/s, 0.57-0.60
// of measured bf16; a tile's 3000 cycles are a block's softmax (1800) and its two products
// (1024), which tensor memory has no room to overlap within the block.  256 trees of 25
// rows, 24 query heads, 4 key heads, 64 columns: 135-138 us, 2.2-2.3 TB/s; tiles of 2500
// cycles where the products need 1024, 22 of the second block's 128 rows in use, and
// some 10000 cycles around an item's eight tiles.
#include <algorithm>
#include <cuda_bf16.h>
#include <mutex>

#include "chain_common.cuh"
#include "launch.cuh"
#include "ptx_pair.cuh"
#include "target_internal.h"

namespace dspark {

constexpr int AT_ROWS = 128;       // rows of a product
constexpr int AT_MAX_NARROW = 320;  // CTAs that leave partial results
constexpr int AT_MAX_WIDE = 160;
constexpr int AT_SEGS = 4;         // segments told ahead
constexpr int AT_POISON = 8;       // segments looked over ahead: more than AT_SEGS + 1
constexpr float kRescale = 8.0f;   // log2 of what the maximum may grow by
// Up to this a maximum is taken off as fma(s, c, -round(m c)): whatever m c was rounded
// to is in lse too, so nothing is lost.  A larger m is taken off first, (s - m) c: at
// 2^24 and more m c would round by whole units.  Where a row passes from one form to
// the other they differ by 2^-17.
constexpr float kLarge = 256.0f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

template <int HD, bool WIDE>
struct AtShape {
  static constexpr int kGroups = WIDE ? 2 : 1;                   // blocks of rows, warpgroups
  static constexpr int kRows = kGroups * AT_ROWS;
  static constexpr int kTokens = WIDE ? 128 : 64;                // of a tile
  static constexpr int kWords = kTokens / 64;                    // of a tile's mask
  static constexpr int kBoxes = HD / 64;                         // 64 columns each
  static constexpr int kBox = kTokens * 128;                     // bytes
  static constexpr int kTile = kBoxes * kBox;                    // of K or V
  static constexpr int kQ = kBoxes * AT_ROWS * 128;
  static constexpr int kK = HD == 64 ? 5 : HD == 128 ? 3 : 2;    // tiles of the rings
  static constexpr int kV = HD == 64 ? 5 : 2;
  static constexpr int kCtas = WIDE || HD == 256 ? 1 : 2;        // an SM
  static constexpr int kTmem = kCtas == 1 ? 512 : 256;           // columns: S, S, O, (O)
  static constexpr int kO = 2 * kTokens;                         // where O begins
  static constexpr int kTiles = kGroups * kQ + (kK + kV) * kTile;
  static constexpr int kThreads = kGroups * 128 + 128;           // softmax; K, V, products
  // tiles that an item costs besides (2, 3, 4, 5: prompts 598, 528, 495, 490 us, trees
  // 147, 140, 139, 139, 64 x 8 rows 190, 185, 184, 184)
  static constexpr int kItem = WIDE ? 4 : 3;
  // registers of the two kinds of warpgroups: together at most the launch's
  static constexpr int kLaunchRegs = kCtas == 1 ? 168 : 128;
  static constexpr int kSoftmaxRegs = WIDE ? 208 : 176;
  static constexpr int kOtherRegs = 80;
  static constexpr bool kSplitRegs = HD != 256;
  static_assert(!kSplitRegs || kGroups * kSoftmaxRegs + kOtherRegs <= (kGroups + 1) * kLaunchRegs,
                "registers of the launch");
};

// What the joining kernel needs about an item that begins in a CTA and is cut.
struct AtMeta {
  int32_t last;    // CTA that holds its end; 0: nothing is cut here
  int32_t request, first, count, head, block;
};

// Partial results: slots 2 c (a run's beginning) and 2 c + 1 (an item's) of CTA c.
struct AtParts {
  AtMeta *meta;
  float2 *ml;  // [slot][rows]: maximum, sum
  float *o;    // [slot][rows / 8][HD / 4][8][4]: eight rows' pieces side by side
  int32_t rows, ctas;  // rows: a multiple of 8
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
  uint32_t group_magic, group_shift;  // for divisions by group
  int32_t page_shift, num_pages, max_pages, least_tiles;
  int32_t both;  // both kernels run: each takes its requests
  float scale_log2;
  float *lse;
  uint32_t *status;
  AtParts parts;
};

// A run of an item's tiles that one CTA computes.
struct AtSeg {
  int32_t request, first, count, ctx, head, block;  // request < 0: the end
  int32_t t0, t1;                                   // of the item's tiles
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

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
// adds to one column of the warp's lanes
__device__ __forceinline__ void tmem_add(uint32_t taddr, float by) {
  float v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(v) : "r"(taddr) : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(v)::"memory");
  v += by;
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "f"(v) : "memory");
  tmem_st_wait();
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
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
// of 64 columns; for V, whose rows run along the product's columns, boxes of 64
// columns.
constexpr uint32_t kAtDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t at_desc_k(uint32_t addr) {
  return ((addr & 0x3FFFFu) >> 4) | 1u << 16;
}
__device__ __forceinline__ uint32_t at_desc_mn(uint32_t addr, int box) {
  return ((addr & 0x3FFFFu) >> 4) | static_cast<uint32_t>(box >> 4) << 16;
}

__device__ __forceinline__ uint64_t pair_f32(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpair_f32(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// m / group for m below 2^29
__device__ __forceinline__ int at_token(const AtParams &p, int m) {
  return p.group == 1 ? m
                      : static_cast<int>(__umulhi(static_cast<uint32_t>(m), p.group_magic) >>
                                         p.group_shift);
}

// ----------------------------------------------------------------- planning
struct AtRequest {
  int first, count, ctx, blocks;
  bool tree;
  uint32_t flags;  // what is wrong with its lengths
};

template <int HD, bool WIDE>
struct AtPlan {
  using Sh = AtShape<HD, WIDE>;
  // a request's rows; no blocks where they are the other kernel's
  static __device__ __forceinline__ AtRequest request(const AtParams &p, int n) {
    AtRequest r;
    const RowSpan rows = row_span(p.cu_rows, n, p.R);
    r.first = rows.first;
    r.count = min(rows.count, p.max_len);
    const int64_t room = static_cast<int64_t>(p.max_pages) << p.page_shift;
    const int ctx = p.ctx_len[n];
    r.ctx = static_cast<int>(min(static_cast<int64_t>(max(ctx, 0)), room));
    r.tree = is_tree(p.tree, p.tree_width, n, rows.count);
    r.flags = rows.count > p.max_len || (ctx < 0 && rows.count > 0) ? DSPARK_DEV_LEN_OOR : 0u;
    if (r.count > 0 && r.ctx + static_cast<int64_t>(r.count) > room)
      r.flags |= DSPARK_DEV_PAGE_OOR;
    const int packed = r.count * p.group;
    r.blocks = p.both && (packed > AT_ROWS) != WIDE ? 0 : (packed + Sh::kRows - 1) / Sh::kRows;
    return r;
  }
  // Tokens that some row of a block attends, as an end: those in the cache and the
  // step's, up to the block's last row where the request is a chain.
  static __device__ __forceinline__ int end(const AtParams &p, const AtRequest &r, int b) {
    const int last = r.tree ? r.count : min(r.count, at_token(p, (b + 1) * Sh::kRows - 1) + 1);
    const int64_t e = static_cast<int64_t>(r.ctx) + last;
    return static_cast<int>(min(e, static_cast<int64_t>(p.max_pages) << p.page_shift));
  }
  static __device__ __forceinline__ int tiles(int end) {
    return (end + Sh::kTokens - 1) / Sh::kTokens;
  }
  // what one head costs, in tiles
  static __device__ __forceinline__ int64_t head_units(const AtParams &p, const AtRequest &r) {
    int64_t sum = 0;
    for (int b = 0; b < r.blocks; ++b) sum += Sh::kItem + tiles(end(p, r, b));
    return sum;
  }
};

// a / b for numbers of units, which hardly ever need 64 bits
__device__ __forceinline__ int64_t at_divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The CTAs' equal shares of all units (each item's kItem, then its tiles): the first
// `more` CTAs have one more.
struct AtShares {
  int64_t each;
  int more, ctas;
  __device__ __forceinline__ void split(int64_t units, int most, int least) {
    ctas = static_cast<int>(
        min(static_cast<int64_t>(most), at_divide(units + least - 1, least)));
    each = ctas > 0 ? at_divide(units, ctas) : 0;
    more = static_cast<int>(units - each * ctas);
  }
  __device__ __forceinline__ int64_t begin(int c) const { return each * c + min(c, more); }
  __device__ __forceinline__ int holder(int64_t unit) const {
    const int64_t first = begin(more);
    return unit < first ? static_cast<int>(at_divide(unit, each + 1))
                        : more + static_cast<int>(at_divide(unit - first, each));
  }
};

// A bounded wait (see common.cuh) in few instructions: what a CTA that gave up has to say
// is said once, at its end.
__device__ __forceinline__ bool at_wait(uint64_t *bar, uint32_t parity,
                                        volatile uint32_t *abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait_sleep(bar, parity, 20000u)) {
    if (*abort_flag != 0u || global_timer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1u;
      return false;
    }
  }
  return true;
}

// Shared state besides the tiles
template <int HD, bool WIDE>
struct AtShared {
  using Sh = AtShape<HD, WIDE>;
  uint64_t k_full[Sh::kK], k_empty[Sh::kK], v_full[Sh::kV], v_ready[Sh::kV],
      v_empty[Sh::kV];
  // by block of rows (wide) or by tile, in turn (narrow)
  uint64_t s_full[2], p_full[2][Sh::kWords], pv_done[2];  // p: 64 tokens at a time
  uint64_t q_full, scanned[AT_POISON];
  uint64_t seg_full[AT_SEGS], seg_empty[AT_SEGS];
  uint32_t poison[AT_POISON][3][Sh::kTokens / 32];  // tokens with values that are not finite
  AtSeg seg[AT_SEGS];
  int64_t scan[Sh::kThreads / 32];
  AtRequest start;
  int64_t start_rest;
  int32_t start_request;
  uint32_t tmem, abort;
};

// A partial O's four columns from `column` on, of one row; the next four are eight further.
template <int HD>
__device__ __forceinline__ float4 *at_part(const AtParts &parts, int slot, int row, int column) {
  return reinterpret_cast<float4 *>(parts.o) +
         (static_cast<int64_t>(slot) * (parts.rows / 8) + row / 8) * (2 * HD) + column / 4 * 8 +
         (row & 7);
}

// The tokens of a tile's word that a row attends: of the cache, and of the step's rows
// (`bits` in a tree, the first `upto` tokens in a chain).
__device__ __forceinline__ uint64_t at_seen(const AtSeg &s, uint64_t bits, int upto, int token) {
  if (!s.tree) return low_bits(upto - token);
  const int shift = s.ctx - token;
  uint64_t seen = low_bits(shift);
  if (shift >= 0 && shift < 64) seen |= bits << shift;
  else if (shift < 0 && shift > -64) seen |= bits >> -shift;
  return seen;
}

// Before this token every row of a segment's block attends every token.
template <class Sh>
__device__ __forceinline__ int at_common(const AtParams &p, const AtSeg &s) {
  return s.ctx + (s.tree ? 0 : at_token(p, s.block * Sh::kRows) + 1);
}

// A segment's pages, 32 at a time: which of them there are.
struct AtPages {
  const int32_t *table;
  int base = -1, page0;
  uint32_t good = 0u;
  __device__ __forceinline__ AtPages(const AtParams &p, const AtSeg &s)
      : table(p.block_table + static_cast<int64_t>(s.request) * p.table_stride),
        shift(p.page_shift) {}
  int shift;
  // by the whole warp, for every tile in turn: those of the tile at this token
  __device__ __forceinline__ void at(const AtParams &p, int token) {
    page0 = token >> shift;
    if (base == (page0 & ~31)) return;
    base = page0 & ~31;
    const int k = base + static_cast<int>(threadIdx.x & 31);
    const int id = k < p.max_pages ? table[k] : -1;
    good = __ballot_sync(0xFFFFFFFFu, id >= 0 && id < p.num_pages);
  }
  // of 32 tokens from the tile's 32 q on, the ones that there are
  __device__ __forceinline__ uint32_t there(const AtSeg &s, int token, int q) const {
    const int from = token + 32 * q;
    const uint32_t lo = good >> (from >> shift & 31) & 1u ? 0xFFFFu : 0u;
    const uint32_t hi = good >> ((from + 16) >> shift & 31) & 1u ? 0xFFFF0000u : 0u;
    return (lo | hi) & static_cast<uint32_t>(low_bits(s.end - from));
  }
  template <int TOK>
  __device__ __forceinline__ bool whole(const AtSeg &s, int token) const {
    const uint32_t all = (1u << (TOK >> shift > 1 ? TOK >> shift : 1)) - 1u;
    return token + TOK <= s.end && (good >> (page0 & 31) & all) == all;
  }
};

template <int HD, bool WIDE>
__global__ void __launch_bounds__(AtShape<HD, WIDE>::kThreads, AtShape<HD, WIDE>::kCtas)
    attention_kernel(const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const AtParams p) {
  using Sh = AtShape<HD, WIDE>;
  using Plan = AtPlan<HD, WIDE>;
  constexpr int TOK = Sh::kTokens, WORDS = Sh::kWords, SOFTMAX = 4 * Sh::kGroups;
  // Nothing else is in shared memory, so that it begins on a multiple of 1024 bytes:
  // with room to align it, two narrow CTAs would not fit an SM.
  extern __shared__ __align__(1024) uint8_t smem[];
  AtShared<HD, WIDE> &sh = *reinterpret_cast<AtShared<HD, WIDE> *>(smem + Sh::kTiles);
  uint8_t *k_ring = smem + Sh::kGroups * Sh::kQ, *v_ring = k_ring + Sh::kK * Sh::kTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile uint32_t *abort_flag = &sh.abort;

  if (tid == 0) {
    for (int i = 0; i < Sh::kK; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < Sh::kV; ++i) {
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_ready[i], 1);
      mbar_init(&sh.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      for (int w = 0; w < WORDS; ++w) mbar_init(&sh.p_full[i][w], 4);
      mbar_init(&sh.pv_done[i], 1);
    }
    mbar_init(&sh.q_full, SOFTMAX);
    for (int i = 0; i < AT_POISON; ++i) mbar_init(&sh.scanned[i], 1);
    for (int i = 0; i < AT_SEGS; ++i) {
      mbar_init(&sh.seg_full[i], 1);
      mbar_init(&sh.seg_empty[i], SOFTMAX + 3);
    }
    sh.abort = 0u;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == SOFTMAX && lane == 0) {
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  // Tensor memory after the wait: what waits for an earlier kernel holds none that a CTA
  // of that kernel may still ask for.
  wait_for_earlier_kernel();
  if (warp == SOFTMAX + 2) {
    tmem_alloc(&sh.tmem, Sh::kTmem);
    tmem_relinquish();
  }
  allow_next_kernel();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int cta = static_cast<int>(blockIdx.x);

  // ---- plan: this CTA's run of tiles, and the request that it begins in
  AtShares shares;
  {
    const int C = (p.N + Sh::kThreads - 1) / Sh::kThreads;
    const int n0 = min(p.N, tid * C), n1 = min(p.N, n0 + C);
    int64_t mine = 0, last = 0;  // units of these requests, and of the last of them
    AtRequest r;
    for (int n = n0; n < n1; ++n) {
      r = Plan::request(p, n);
      last = p.Hk * Plan::head_units(p, r);
      mine += last;
      if (cta == 0 && !WIDE && r.flags != 0u) raise_status(p.status, r.flags);
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
#pragma unroll 1
    for (int w = 0; w < Sh::kThreads / 32; ++w) {
      if (w < warp) before += sh.scan[w];
      total += sh.scan[w];
    }
    shares.split(total, static_cast<int>(gridDim.x), p.least_tiles);
    if (cta < shares.ctas) {
      int64_t rest = shares.begin(cta) - before;
      if (rest >= 0 && rest < mine) {
        int n = n1 - 1;
        if (n > n0) {  // several requests: which
          for (n = n0; n < n1; ++n) {
            r = Plan::request(p, n);
            const int64_t units = p.Hk * Plan::head_units(p, r);
            if (rest < units) break;
            rest -= units;
          }
        }
        sh.start = r;
        sh.start_request = n;
        sh.start_rest = rest;
      }
    }
    __syncthreads();
  }

  if (warp >= SOFTMAX) {
    if constexpr (Sh::kSplitRegs) registers_down<Sh::kOtherRegs>();
    const uint32_t one = at_elect();
    bool ok = true;
    int g = 0, segs = 0;  // tiles and segments so far
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      ok = ok && __all_sync(0xFFFFFFFFu, at_wait(bar, parity, abort_flag));
      return ok;
    };
    if (warp <= SOFTMAX + 1) {
      // ------------------------------- segments and K (one warp), V (the other)
      const bool is_v = warp != SOFTMAX;
      const int stages = is_v ? Sh::kV : Sh::kK;
      uint64_t *full = is_v ? sh.v_full : sh.k_full, *empty = is_v ? sh.v_empty : sh.k_empty;
      const uint32_t ring = smem_u32(is_v ? v_ring : k_ring);
      const CUtensorMap *map = is_v ? &v_map : &k_map;
      const int box_rows = min(1 << p.page_shift, TOK);
      // where this CTA's run has got to: request n (r), head h, block b, `rest` units in
      AtMeta meta = {};
      AtRequest r = sh.start;
      const int64_t end_unit = cta < shares.ctas ? shares.begin(cta + 1) : 0;
      int64_t unit = cta < shares.ctas ? shares.begin(cta) : 0, rest = sh.start_rest;
      int n = sh.start_request, h = 0, b = 0;
      if (!is_v && unit < end_unit) {
        const int64_t a_head = Plan::head_units(p, r);
        h = static_cast<int>(at_divide(rest, a_head));
        rest -= h * a_head;
      }
      uint32_t stage = 0, turn = 0;  // of the ring
      while (ok) {
        const int si = segs % AT_SEGS;
        AtSeg s;
        if (is_v) {
          if (!wait(&sh.seg_full[si], (segs / AT_SEGS) & 1)) break;
          s = sh.seg[si];
          __syncwarp();
          if (one) mbar_arrive(&sh.seg_empty[si]);
        } else {
          s.request = -1;
          int64_t cut = -1;  // the last unit of an item that begins here and is cut
          while (unit < end_unit) {
            if (b >= r.blocks) {
              b = 0;
              if (++h >= p.Hk) {
                h = 0;
                if (++n >= p.N) break;
                r = Plan::request(p, n);
              }
              continue;
            }
            const int end = Plan::end(p, r, b), tiles = Plan::tiles(end);
            if (rest >= Sh::kItem + tiles) {  // before this run
              rest -= Sh::kItem + tiles;
              ++b;
              continue;
            }
            const int64_t stop =
                min(static_cast<int64_t>(Sh::kItem + tiles), rest + (end_unit - unit));
            s.t0 = static_cast<int>(max(rest - Sh::kItem, static_cast<int64_t>(0)));
            s.t1 = static_cast<int>(max(stop - Sh::kItem, static_cast<int64_t>(0)));
            unit += stop - rest;
            rest = 0;
            if (s.t1 > s.t0) {  // else this run ends before its first tile
              s.request = n;
              s.first = r.first;
              s.count = r.count;
              s.ctx = r.ctx;
              s.head = h;
              s.block = b;
              s.tree = r.tree;
              s.end = end;
              s.part = -1;
              if (s.t0 > 0) {
                s.part = 2 * cta;
              } else if (s.t1 < tiles) {
                s.part = 2 * cta + 1;
                meta = {0, n, s.first, s.count, h, b};
                cut = unit + (tiles - s.t1) - 1;
              }
            }
            ++b;
            if (s.request >= 0) break;
          }
          if (!wait(&sh.seg_empty[si], ((segs / AT_SEGS) & 1) ^ 1u)) break;
          if (one) {
            sh.seg[si] = s;
            mbar_arrive(&sh.seg_full[si]);
          }
          __syncwarp();
          if (cut >= 0) meta.last = shares.holder(cut);
        }
        ++segs;
        if (s.request < 0) break;
        // the segment's tiles, through its pages: a lane each, 32 at a time
        const int32_t *table = p.block_table + static_cast<int64_t>(s.request) * p.table_stride;
        int base = -1, ids = -1;
        uint32_t good = 0u;  // of these pages, the ones that there are
#pragma unroll 1
        for (int t = s.t0; t < s.t1; ++t) {
          const int token = t * TOK, page0 = token >> p.page_shift;
          if (base != (page0 & ~31)) {
            base = page0 & ~31;
            const int k = base + lane;
            ids = k < p.max_pages ? table[k] : -1;
            good = __ballot_sync(0xFFFFFFFFu, ids >= 0 && ids < p.num_pages);
          }
          if (!wait(&empty[stage], turn ^ 1u)) break;
          const int boxes = (min(TOK, s.end - token) + box_rows - 1) / box_rows;
          const uint32_t here = (good >> (page0 & 31)) & ((1u << boxes) - 1u);
          if (!is_v && one && here != (1u << boxes) - 1u)
            raise_status(p.status, DSPARK_DEV_PAGE_OOR);
          if (one)
            mbar_arrive_expect_tx(&full[stage], __popc(here) * Sh::kBoxes * box_rows * 128);
          __syncwarp();
          uint32_t dst = ring + stage * Sh::kTile;
          const int offset = token & ((1 << p.page_shift) - 1);
#pragma unroll 1
          for (int k = 0; k < boxes; ++k, dst += box_rows * 128) {
            const int id = __shfl_sync(0xFFFFFFFFu, ids, (page0 + k) & 31);
            const uint32_t go = here >> k & 1u ? one : 0u;
#pragma unroll
            for (int c = 0; c < Sh::kBoxes; ++c)
              tma_load_page(go, dst + c * Sh::kBox, map, &full[stage], c * 64, s.head, offset, id);
          }
          if (++stage == static_cast<uint32_t>(stages)) {
            stage = 0;
            turn ^= 1u;
          }
        }
      }
      if (!is_v && one) p.parts.meta[cta] = meta;
    } else if (warp == SOFTMAX + 2) {
      // ----------------------------------------------------------- products
      const uint32_t q_lo = at_desc_k(smem_u32(smem));
      const uint32_t k0 = smem_u32(k_ring), v0 = smem_u32(v_ring);
      constexpr uint32_t idesc_s = umma_idesc_bf16_f32(AT_ROWS, TOK);
      constexpr uint32_t idesc_o = umma_idesc_bf16_f32(AT_ROWS, HD) | 1u << 16;
      int turns[2] = {0, 0};  // wide: tiles of each block of rows so far
      auto arrived = [&](uint64_t *bar, uint32_t parity) {
        wait(bar, parity);
        tc_fence_after();
        return ok;
      };
      while (ok) {
        const int si = segs % AT_SEGS;
        if (!arrived(&sh.seg_full[si], (segs / AT_SEGS) & 1)) break;
        const int request = sh.seg[si].request, T = sh.seg[si].t1 - sh.seg[si].t0;
        const int rows = sh.seg[si].count * p.group - sh.seg[si].block * Sh::kRows;
        __syncwarp();
        if (one) mbar_arrive(&sh.seg_empty[si]);
        if (request < 0) break;
        if (!arrived(&sh.q_full, segs & 1)) break;
        ++segs;
        const int blocks = WIDE && rows > AT_ROWS ? 2 : 1;
        // S of tile i for block r.  The tensor core takes products in the order in
        // which they are issued, so a wide block's S may follow the product that reads
        // the P in its place.
        auto score = [&](int r, int i) {
          const int gt = g + i, buf = WIDE ? r : gt & 1;
          if (!WIDE && gt >= 2 && !arrived(&sh.pv_done[buf], ((gt >> 1) - 1) & 1)) return;
          const int stage = gt % Sh::kK;
          if (r == 0 && !arrived(&sh.k_full[stage], (gt / Sh::kK) & 1)) return;
          const uint32_t a = q_lo + r * (Sh::kQ >> 4);
          const uint32_t b = at_desc_k(k0 + stage * Sh::kTile);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            umma_ss(one, tmem + buf * TOK, a + (kk / 4) * (AT_ROWS * 128 >> 4) + (kk % 4) * 2,
                    b + (kk / 4) * (Sh::kBox >> 4) + (kk % 4) * 2, kAtDescHi, idesc_s, kk);
          if (r == blocks - 1) umma_commit_one(one, &sh.k_empty[stage]);
          umma_commit_one(one, &sh.s_full[buf]);
        };
        auto value = [&](int r, int i) {
          const int gt = g + i, buf = WIDE ? r : gt & 1;
          const uint32_t turn = WIDE ? turns[r] + i : gt >> 1;
          const int stage = gt % Sh::kV;
          if (r == 0 && !arrived(&sh.v_ready[stage], (gt / Sh::kV) & 1)) return;
          const uint32_t b = at_desc_mn(v0 + stage * Sh::kTile, Sh::kBox);
#pragma unroll
          for (int w = 0; w < WORDS; ++w) {
            if (!arrived(&sh.p_full[buf][w], turn & 1)) return;
#pragma unroll
            for (int kk = 4 * w; kk < 4 * w + 4; ++kk)
              umma_ts(one, tmem + Sh::kO + r * HD, tmem + buf * TOK + kk * 8, b + kk * 128,
                      kAtDescHi, idesc_o, i | kk);
          }
          if (r == blocks - 1) umma_commit_one(one, &sh.v_empty[stage]);
          umma_commit_one(one, &sh.pv_done[buf]);
        };
        // wide: P V and the next S of one block, then of the other; narrow: the next S
        // before P V
#pragma unroll 1
        for (int i = -1; ok && i < T; ++i) {
#pragma unroll 1
          for (int r = 0; ok && r < blocks; ++r) {
            if (WIDE && i >= 0) value(r, i);
            if (ok && i + 1 < T) score(r, i + 1);
            if (!WIDE && ok && i >= 0) value(r, i);
          }
        }
        if (WIDE) {
          turns[0] += T;
          if (blocks == 2) turns[1] += T;
        }
        g += T;
      }
    }
    if (warp == SOFTMAX + 3) {
      // ---------------------------------------------------------- V, looked over
      // Values of tokens that are not there are 0, and those that are not finite where
      // not every row attends them: 0 times them would be NaN.
      uint32_t stage = 0, phase = 0;
      while (ok) {
        const int si = segs % AT_SEGS;
        if (!wait(&sh.seg_full[si], (segs / AT_SEGS) & 1)) break;
        const AtSeg s = sh.seg[si];
        __syncwarp();
        if (one) mbar_arrive(&sh.seg_empty[si]);
        if (s.request < 0) break;
        const int slot = segs++ % AT_POISON;
        const int common = at_common<Sh>(p, s);
        uint32_t(&poison)[3][TOK / 32] = sh.poison[slot];
        if (lane < 3 * (TOK / 32)) poison[lane / (TOK / 32)][lane % (TOK / 32)] = 0u;
        __syncwarp();
        AtPages pages(p, s);
#pragma unroll 1
        for (int t = s.t0; t < s.t1; ++t) {
          const int token = t * TOK;
          pages.at(p, token);
          if (!wait(&sh.v_full[stage], phase)) break;
          const bool inner = token + TOK <= common;
          if (!inner || !pages.whole<TOK>(s, token)) {
            const uint32_t v = smem_u32(v_ring) + stage * Sh::kTile;
            constexpr int CHUNKS = HD / 8;
#pragma unroll 1
            for (int q = 0; q < TOK / 32; ++q) {  // 32 tokens at a time
              const uint32_t there = pages.there(s, token, q), v_q = v + q * 32 * 128;
              // k: a row, then 16 bytes of it
              auto chunk = [&](int k) {
                const int r = k / CHUNKS, e = k % CHUNKS;
                return v_q + (e / 8) * Sh::kBox + r * 128 + ((e & 7) << 4);
              };
              if (there != 0xFFFFFFFFu) {
#pragma unroll 1
                for (int k = lane; k < 32 * CHUNKS; k += 32)
                  if ((there >> (k / CHUNKS) & 1u) == 0u) st_shared_zero16(chunk(k));
                __syncwarp();
              }
              if (inner) continue;
              // 0 times a number is 0, 0 times anything else is NaN
              const __nv_bfloat162 zero = __float2bfloat162_rn(0.0f);
              __nv_bfloat162 none = zero;
#pragma unroll 4
              for (int k = lane; k < 32 * CHUNKS; k += 32) {
                const uint4 w = ld_shared_v4(chunk(k));
                const uint32_t *u = &w.x;
#pragma unroll
                for (int h = 0; h < 4; ++h)
                  none = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(u + h), zero, none);
              }
              if (!__any_sync(0xFFFFFFFFu, __hisnan(none.x) || __hisnan(none.y))) continue;
              uint32_t bad = 0u;
#pragma unroll 1
              for (int k = lane; k < 4 * 32 * CHUNKS; k += 32) {  // two values at a time
                const uint32_t at = chunk(k >> 2) + (k & 3) * 4;
                const uint32_t w = ld_shared_u32(at);
                const uint32_t keep = ((w & 0x7F80u) == 0x7F80u ? 0u : 0xFFFFu) |
                                      ((w & 0x7F800000u) == 0x7F800000u ? 0u : 0xFFFF0000u);
                if (keep != 0xFFFFFFFFu) {
                  st_shared_u32(at, w & keep);
                  bad |= 1u << ((k >> 2) / CHUNKS);
                }
              }
              bad = __reduce_or_sync(0xFFFFFFFFu, bad);
              if (lane == 0) poison[t - common / TOK][q] = bad;
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (one) mbar_arrive(&sh.v_ready[stage]);
          if (++stage == Sh::kV) {
            stage = 0;
            phase ^= 1u;
          }
        }
        __syncwarp();
        if (one) mbar_arrive(&sh.scanned[slot]);
      }
    }
    if (!ok) {
      // copies and products in flight end before their memory is given back
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 20000000ull) __nanosleep(1000);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    if constexpr (Sh::kSplitRegs) registers_up<Sh::kSoftmaxRegs>();
    const int block = WIDE ? warp >> 2 : 0;  // of rows
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_tmem = tmem + lanes + Sh::kO + block * HD;
    const int row = warp * 32 + lane;
    const float c = p.scale_log2;
    const uint64_t c2 = pair_f32(__float_as_uint(c), __float_as_uint(c));
    bool ok = true, have = false;
    int g = 0, turn = 0, segs = 0;  // tiles, this block's, segments
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      ok = ok && __all_sync(0xFFFFFFFFu, at_wait(bar, parity, abort_flag));
      return ok;
    };
    AtSeg s = {};
    while (true) {
      // ---- tokens of segment s
      const int T = s.t1 - s.t0, m = s.block * Sh::kRows + row, j = at_token(p, m);
      const bool mine = have && j < s.count;
      // the second block may have no rows; the products leave it out too
      const bool active =
          have && !(block == 1 && s.count * p.group - s.block * Sh::kRows <= AT_ROWS);
      const bool any = __any_sync(0xFFFFFFFFu, mine);
      const uint64_t bits =
          mine && s.tree ? tree_bits(p.tree, p.tree_width, s.request, j, s.count) : 0ull;
      const int upto = s.ctx + j + 1;
      // before this token every row attends every token
      const int common = at_common<Sh>(p, s);
      const int this_seg = segs - 1;
      float top = -INFINITY, sum = 0.0f;
      if (active) {
        AtPages pages(p, s);
#pragma unroll 1
        for (int i = 0; i < T; ++i) {
          const int gt = g + i, token = (s.t0 + i) * TOK;
          const int buf = WIDE ? block : gt & 1;
          const uint32_t phase = WIDE ? turn & 1 : (gt >> 1) & 1;
          ++turn;
          pages.at(p, token);
          const bool inner = token + TOK <= common && pages.whole<TOK>(s, token);
          if (!wait(&sh.s_full[buf], phase)) break;
          tc_fence_after();
          if (!any) {
            __syncwarp();
            if (lane < WORDS) mbar_arrive(&sh.p_full[buf][lane]);
            continue;
          }
          const uint32_t s_tmem = tmem + lanes + buf * TOK;
          if (!inner) {
            // scores of what a row does not attend: -inf
#pragma unroll 1
            for (int k = 0; k < TOK / 32; ++k) {
              const uint32_t seen =
                  static_cast<uint32_t>(at_seen(s, bits, upto, token + 32 * k)) &
                  pages.there(s, token, k);
              uint32_t x[32];
              tmem_ld_32x32b_x32(s_tmem + 32 * k, x);
              tmem_ld_wait(x);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = (seen >> e & 1u) ? x[e] : 0xFF800000u;
              tmem_st_32x32b_x32(s_tmem + 32 * k, x);
            }
            tmem_st_wait();
          }
          uint32_t x[TOK / 32][32];
#pragma unroll
          for (int k = 0; k < TOK / 32; ++k) tmem_ld_32x32b_x32(s_tmem + 32 * k, x[k]);
#pragma unroll
          for (int k = 0; k < TOK / 32; ++k) tmem_ld_wait(x[k]);
          float highs[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < TOK / 32; ++k)
#pragma unroll
            for (int e = 0; e < 32; e += 8)
#pragma unroll
              for (int q = 0; q < 4; ++q)  // three operands at a time
                highs[q] = fmaxf(fmaxf(highs[q], __uint_as_float(x[k][e + q])),
                                 __uint_as_float(x[k][e + 4 + q]));
          const float high = fmaxf(fmaxf(highs[0], highs[1]), fmaxf(highs[2], highs[3]));
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
              // O holds the tiles before once their product is through; a wide block's
              // S was issued after it
              if (!WIDE && !wait(&sh.pv_done[(gt - 1) & 1], ((gt - 1) >> 1) & 1)) break;
              tc_fence_after();
#pragma unroll 1
              for (int at = 0; at < HD; at += 16) {
                uint32_t o[16];
                tmem_ld_32x32b_x16(o_tmem + at, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
                tmem_st_32x32b_x16(o_tmem + at, o);
              }
              tmem_st_wait();
            }
          }
          const float off = top == -INFINITY ? 0.0f : top;
          float base = __fmul_rn(off, c);
          const bool large = fabsf(base) > kLarge;
          if (__any_sync(0xFFFFFFFFu, large)) {
            const float by = large ? off : 0.0f;  // a row's bits are its own affair
#pragma unroll
            for (int k = 0; k < TOK / 32; ++k)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                x[k][e] = __float_as_uint(__uint_as_float(x[k][e]) - by);
            if (large) base = 0.0f;
          }
          const uint64_t base2 = pair_f32(__float_as_uint(-base), __float_as_uint(-base));
          uint64_t sums[2] = {0ull, 0ull};
#pragma unroll
          for (int k = 0; k < WORDS; ++k) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t(&y)[32] = x[2 * k + e / 16];
              float lo, hi;
              unpair_f32(pair_fma(pair_f32(y[(2 * e) & 31], y[(2 * e + 1) & 31]), c2, base2), lo,
                         hi);
              lo = exp2_approx(lo);
              hi = exp2_approx(hi);
              sums[e & 1] =
                  pair_add(sums[e & 1], pair_f32(__float_as_uint(lo), __float_as_uint(hi)));
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pk[e]) : "f"(hi), "f"(lo));
            }
            tmem_st_32x32b_x32(s_tmem + 32 * k, pk);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[buf][k]);
          }
          float lo, hi;
          unpair_f32(pair_add(sums[0], sums[1]), lo, hi);
          sum += lo + hi;
        }
        if (!ok) break;
      }
      g += T;
      // ---- the next segment, and its Q on the way to shared memory (the last scores of
      // this one are there, so its own has been read): a warp its 32 rows, row after row,
      // so that neighbouring lanes read neighbouring bytes
      AtSeg next;
      {
        const int si = segs % AT_SEGS;
        if (!wait(&sh.seg_full[si], (segs / AT_SEGS) & 1)) break;
        next = sh.seg[si];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[si]);
        ++segs;
        const int nm = next.block * Sh::kRows + row, nj = at_token(p, nm);
        const __nv_bfloat16 *src = nullptr;
        if (next.request >= 0 && nj < next.count)
          src = static_cast<const __nv_bfloat16 *>(p.q.p) + (next.first + nj) * p.q.stride +
                (next.head * p.group + nm - nj * p.group) * p.q.head_stride;
        const uint32_t dst = smem_u32(smem) + block * Sh::kQ + (warp & 3) * 32 * 128;
        constexpr int CHUNKS = HD / 8;  // of 16 bytes, a row
        // of the rows that there are
        const int left = next.request < 0 ? 0 : next.count * p.group - (nm - lane);
        const int chunks = min(max(left, 0), 32) * CHUNKS;
#pragma unroll 2
        for (int k = lane; k - lane < chunks; k += 32) {
          const int r = k / CHUNKS, e = k % CHUNKS;
          const __nv_bfloat16 *from = reinterpret_cast<const __nv_bfloat16 *>(
              __shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(src), r));
          const uint32_t at =
              dst + (e / 8) * (AT_ROWS * 128) + r * 128 + (((e & 7) ^ (r & 7)) << 4);
          if (from != nullptr) {
            if (e * 8 < p.d) cp_async_16(at, from + e * 8);
            else st_shared_zero16(at);
          }
        }
      }
      // ---- this segment's rows, or what is to be joined
      if (active) {
        const int buf = WIDE ? block : (g - 1) & 1;
        if (!wait(&sh.pv_done[buf], WIDE ? (turn - 1) & 1 : ((g - 1) >> 1) & 1)) break;
        tc_fence_after();
      }
      if (active && any) {
        const int head = s.head * p.group + (m - j * p.group);
        const int64_t q_row = s.first + j;
        // the tokens with values that are not finite that this row attends, by 32
        uint32_t hit = 0u;
        const uint32_t(&poison)[3][TOK / 32] = sh.poison[this_seg % AT_POISON];
        auto first_token = [&](int k) { return common / TOK * TOK + 32 * k; };
        auto found = [&](int k) {
          return poison[k / (TOK / 32)][k % (TOK / 32)] &
                 static_cast<uint32_t>(at_seen(s, bits, upto, first_token(k)));
        };
        if (s.t1 * TOK > common) {
          if (!wait(&sh.scanned[this_seg % AT_POISON], (this_seg / AT_POISON) & 1)) break;
#pragma unroll 1
          for (int k = 0; k < 3 * (TOK / 32); ++k)
            if (mine && found(k) != 0u) hit |= 1u << k;
        }
        if (__any_sync(0xFFFFFFFFu, hit != 0u)) {
#pragma unroll 1
          for (int at = 0; at < p.d; ++at) {
            float f = 0.0f;
            for (uint32_t left = hit; left != 0u; left &= left - 1u) {
              const int k = __ffs(left) - 1;
              for (uint32_t tokens = found(k); tokens != 0u; tokens &= tokens - 1u) {
                const int token = first_token(k) + __ffs(tokens) - 1;
                const int id =
                    p.block_table[s.request * p.table_stride + (token >> p.page_shift)];
                const float v = __bfloat162float(
                    p.v_cache[id * p.page_stride +
                              (token & ((1 << p.page_shift) - 1)) * p.token_stride +
                              s.head * p.head_stride + at]);
                if (!(fabsf(v) < INFINITY)) f += v;
              }
            }
            __syncwarp();
            tmem_add(o_tmem + at, f);
          }
        }
        const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
        // where this lane's four rows go: 0 for none
        uint64_t rows_out[4];
        {
          const uint64_t mine_out =
              mine ? reinterpret_cast<uint64_t>(static_cast<__nv_bfloat16 *>(p.out.p) +
                                                q_row * p.out.stride + head * p.out.head_stride)
                   : 0ull;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            rows_out[q] = __shfl_sync(0xFFFFFFFFu, mine_out, (lane & ~3) + q);
        }
#pragma unroll 1
        for (int at = 0; at < HD; at += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(o_tmem + at, o);
          tmem_ld_wait(o);
          if (s.part < 0) {
            // Four lanes exchange their 16-byte pieces, so that each stores one of every
            // row: 64 neighbouring bytes a row and store instead of 16.
            uint32_t w[4][4];
#pragma unroll
            for (int q = 0; q < 16; ++q)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                  : "=r"(w[q >> 2][q & 3])
                  : "f"(__uint_as_float(o[2 * q + 1]) * by), "f"(__uint_as_float(o[2 * q]) * by));
#pragma unroll
            for (int step = 1; step <= 2; step *= 2) {
              const bool upper = (lane & step) != 0;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if ((q & step) != 0) continue;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const uint32_t got =
                      __shfl_xor_sync(0xFFFFFFFFu, upper ? w[q][u] : w[q + step][u], step);
                  if (upper) w[q][u] = got;
                  else w[q + step][u] = got;
                }
              }
            }
            const int column = at + (lane & 3) * 8;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (rows_out[q] != 0 && column < p.d)
                *reinterpret_cast<uint4 *>(rows_out[q] + 2 * column) =
                    make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
          } else if (mine) {
            float4 *dst = at_part<HD>(p.parts, s.part, row, at);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[8 * e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                       __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          }
          __syncwarp();
        }
        if (mine && s.part >= 0)
          p.parts.ml[static_cast<int64_t>(s.part) * p.parts.rows + row] = make_float2(top, sum);
        else if (mine && p.lse != nullptr)
          p.lse[q_row * (p.Hk * p.group) + head] =
              sum == 0.0f ? -INFINITY : at_base(top, c) * kLn2 + logf(sum);
      }
      tc_fence_before();
      if (next.request < 0) break;
      s = next;
      have = true;
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
    }
  }
  if (lane == 0 && *abort_flag) raise_status(p.status, DSPARK_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == SOFTMAX + 2) tmem_dealloc(tmem, Sh::kTmem);
}

// Joins the pieces of the items that were cut: a CTA eight rows, a thread four columns of
// one of them, every blockDim.y-th piece.  The pieces' maxima and sums are read once for
// the CTA, AT_JOIN pieces at a time.
constexpr int AT_JOIN = 64;
template <int HD>
__global__ void __launch_bounds__(HD == 64 ? 512 : 1024)
    attention_join_kernel(const AtParams p, const AtParts narrow, const AtParts wide) {
  __shared__ float2 ml[AT_JOIN][8];      // maximum, sum
  __shared__ float4 others[3][2 * HD];   // of the threads (., y > 0)
  wait_for_earlier_kernel();
  const bool second = static_cast<int>(blockIdx.x) >= narrow.ctas;
  const AtParts &parts = second ? wide : narrow;
  const int cta = static_cast<int>(blockIdx.x) - (second ? narrow.ctas : 0);
  const AtMeta meta = parts.meta[cta];
  const int row0 = blockIdx.y * 8, m0 = meta.block * (second ? 2 * AT_ROWS : AT_ROWS) + row0;
  if (meta.last == 0 || row0 >= parts.rows || m0 >= meta.count * p.group) return;
  const int row = row0 + (threadIdx.x & 7), column = (threadIdx.x >> 3) * 4;
  const int pieces = meta.last - cta + 1;
  // the first piece is in the CTA's second slot, the others in first ones
  auto slot = [&](int k) { return k == 0 ? 2 * cta + 1 : 2 * (cta + k); };
  const int threads = blockDim.x * blockDim.y, thread = threadIdx.y * blockDim.x + threadIdx.x;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float sum = 0.0f, top = -INFINITY;
  auto add = [&](float w, const float4 &v) {
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  };
  for (int k0 = 0; k0 < pieces; k0 += AT_JOIN) {
    const int n = min(AT_JOIN, pieces - k0);
    if (k0 > 0) __syncthreads();
    for (int k = thread; k < 8 * n; k += threads)
      ml[k >> 3][k & 7] =
          parts.ml[static_cast<int64_t>(slot(k0 + (k >> 3))) * parts.rows + row0 + (k & 7)];
    __syncthreads();
    float high = top;
#pragma unroll 8
    for (int k = 0; k < n; ++k) high = fmaxf(high, ml[k][threadIdx.x & 7].x);
    const float above = high == -INFINITY ? 0.0f : high;
    if (k0 > 0) {
      const float by = exp2_approx(at_difference(top, above, p.scale_log2));
      sum *= by;
      acc = make_float4(acc.x * by, acc.y * by, acc.z * by, acc.w * by);
    }
    top = high;
#pragma unroll 4
    for (int k = threadIdx.y; k < n; k += blockDim.y) {
      const float4 v = *at_part<HD>(parts, slot(k0 + k), row, column);
      const float2 x = ml[k][threadIdx.x & 7];
      const float w = exp2_approx(at_difference(x.x, above, p.scale_log2));
      sum = fmaf(w, x.y, sum);
      add(w, v);
    }
  }
  if (blockDim.y > 1) {
    // each in its turn, so that the sums have one order
    __shared__ float sums[3][2 * HD];
    if (threadIdx.y > 0) {
      others[threadIdx.y - 1][threadIdx.x] = acc;
      sums[threadIdx.y - 1][threadIdx.x] = sum;
    }
    __syncthreads();
    if (threadIdx.y > 0) return;
    for (int y = 0; y < static_cast<int>(blockDim.y) - 1; ++y) {
      add(1.0f, others[y][threadIdx.x]);
      sum += sums[y][threadIdx.x];
    }
  }
  const int m = m0 + (threadIdx.x & 7), j = m / p.group;
  if (j >= meta.count) return;
  const int head = meta.head * p.group + (m - j * p.group);
  const int64_t q_row = meta.first + j;
  const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (column < p.d) {
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(acc.y * by), "f"(acc.x * by));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(acc.w * by), "f"(acc.z * by));
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out.p) + q_row * p.out.stride +
                               head * p.out.head_stride + column) = w;
  }
  if (column == 0 && p.lse != nullptr)
    p.lse[q_row * (p.Hk * p.group) + head] =
        sum == 0.0f ? -INFINITY : at_base(top, p.scale_log2) * kLn2 + logf(sum);
}

// ==========================================================================
// host side
// ==========================================================================
static int padded_head(int32_t d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

// Rows of a slot, and the workspace: status, then each kernel's meta, sums and O.
struct AtLayout {
  int narrow_rows, wide_rows;  // wide_rows 0: that kernel does not run
  size_t meta[2], ml[2], o[2], total;
};
static AtLayout at_layout(int32_t max_len, int32_t group, int32_t d) {
  AtLayout l = {};
  const int64_t packed = (static_cast<int64_t>(max_len) * group + 7) / 8 * 8;
  const int hd = padded_head(d);
  l.narrow_rows = static_cast<int>(std::min<int64_t>(AT_ROWS, packed));
  l.wide_rows = static_cast<int64_t>(max_len) * group > AT_ROWS && hd <= 128
                    ? static_cast<int>(std::min<int64_t>(2 * AT_ROWS, packed))
                    : 0;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const int rows[2] = {l.narrow_rows, l.wide_rows}, ctas[2] = {AT_MAX_NARROW, AT_MAX_WIDE};
  for (int k = 0; k < 2; ++k) {
    const size_t slots = static_cast<size_t>(2 * ctas[k]) * rows[k];
    l.meta[k] = take(ctas[k] * sizeof(AtMeta));
    l.ml[k] = take(slots * sizeof(float2));
    l.o[k] = take(slots * hd * sizeof(float));
  }
  l.total = at;
  return l;
}

size_t attention_workspace_bytes(int32_t max_len, int32_t Hq, int32_t Hk, int32_t d) {
  return at_layout(max_len, Hq / Hk, d).total;
}

static bool encode_cache(EncodeTiledFn enc, CUtensorMap *map, const void *p,
                         const AttentionArgs &a, int tokens) {
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.d), static_cast<cuuint64_t>(a.Hk),
                        static_cast<cuuint64_t>(1) << a.page_shift,
                        static_cast<cuuint64_t>(a.num_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.head_stride) * 2,
                           static_cast<cuuint64_t>(a.token_stride) * 2,
                           static_cast<cuuint64_t>(a.page_stride) * 2};
  cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(std::min(1 << a.page_shift, tokens)), 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

static std::mutex g_at_mu;

template <int HD, bool WIDE>
static dspark_status launch_one(const AttentionArgs &a, const AtParams &p, int dev,
                                cudaStream_t stream) {
  using Sh = AtShape<HD, WIDE>;
  constexpr int bytes = Sh::kTiles + static_cast<int>(sizeof(AtShared<HD, WIDE>));
  static_assert(Sh::kCtas * (bytes + 1024) <= 228 * 1024, "shared memory of an SM");
  static bool attr[128];
  {
    std::lock_guard<std::mutex> lk(g_at_mu);
    if (!attr[dev]) {
      if (cudaFuncSetAttribute(attention_kernel<HD, WIDE>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return DSPARK_ERR_CUDA;
      attr[dev] = true;
    }
  }
  EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return DSPARK_ERR_CUDA;
  CUtensorMap k_map, v_map;
  if (!encode_cache(enc, &k_map, a.k_cache, a, Sh::kTokens) ||
      !encode_cache(enc, &v_map, a.v_cache, a, Sh::kTokens))
    return DSPARK_ERR_INVALID_ARG;
  return launch_overlapped(attention_kernel<HD, WIDE>, dim3(p.parts.ctas), dim3(Sh::kThreads),
                           bytes, stream, k_map, v_map, p) == cudaSuccess
             ? DSPARK_OK
             : DSPARK_ERR_CUDA;
}

template <int HD>
static dspark_status launch(const AttentionArgs &a, int dev, int sms, cudaStream_t stream) {
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
  while ((1 << p.group_shift) < p.group) ++p.group_shift;
  if (p.group > 1) {
    --p.group_shift;
    p.group_magic = static_cast<uint32_t>(((1ull << (32 + p.group_shift)) + p.group - 1) / p.group);
  }
  p.page_shift = a.page_shift;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.scale_log2 = a.scale * kLog2e;
  p.lse = a.lse;
  p.status = reinterpret_cast<uint32_t *>(a.workspace);
  const AtLayout l = at_layout(a.max_len, p.group, a.d);
  auto parts = [&](int k, int rows, int ctas) {
    AtParts x;
    x.meta = reinterpret_cast<AtMeta *>(a.workspace + l.meta[k]);
    x.ml = reinterpret_cast<float2 *>(a.workspace + l.ml[k]);
    x.o = reinterpret_cast<float *>(a.workspace + l.o[k]);
    x.rows = rows;
    x.ctas = ctas;
    return x;
  };
  const AtParts narrow = parts(
      0, l.narrow_rows, std::min(AT_MAX_NARROW, AtShape<HD, false>::kCtas * sms));
  const AtParts wide = parts(1, l.wide_rows, l.wide_rows > 0 ? std::min(AT_MAX_WIDE, sms) : 0);
  p.both = l.wide_rows > 0;
  dspark_status s;
  if constexpr (HD <= 128) {
    if (l.wide_rows > 0) {
      p.parts = wide;
      p.least_tiles = 2;
      if ((s = launch_one<HD, true>(a, p, dev, stream)) != DSPARK_OK) return s;
    }
  }
  p.parts = narrow;
  // fewer would be joined more often than they are computed sooner (one token over 8192:
  // 4, 8, 12 tiles 21.9, 21.6, 24.8 us)
  p.least_tiles = 8;
  if ((s = launch_one<HD, false>(a, p, dev, stream)) != DSPARK_OK) return s;
  const int rows = std::max(l.narrow_rows, l.wide_rows);
  // few rows: more threads for an item's pieces
  const int share = rows <= 16 ? (HD == 256 ? 2 : 4) : rows <= 64 && HD <= 128 ? 2 : 1;
  return launch_overlapped(attention_join_kernel<HD>,
                           dim3(narrow.ctas + wide.ctas, rows / 8), dim3(2 * HD, share), 0, stream, p,
                           narrow, wide) == cudaSuccess
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
      return launch<64>(a, dev, sms, stream);
    case 128:
      return launch<128>(a, dev, sms, stream);
    default:
      return launch<256>(a, dev, sms, stream);
  }
}

}  // namespace dspark
