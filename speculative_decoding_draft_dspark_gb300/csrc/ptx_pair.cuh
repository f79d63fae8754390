// Inline-PTX wrappers for kernels whose CTAs work in pairs (clusters of two
// sharing one tcgen05 tile), and for TMA stores from shared memory.  Written
// from the PTX ISA's instruction descriptions; no library code is used.
#pragma once

#include "ptx.cuh"

namespace dspark {

// ---------------------------------------------------------------- cluster
__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// the address, in the cluster's shared window, that `addr` has in CTA `rank`
__device__ __forceinline__ uint32_t mapa_u32(uint32_t addr, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(addr), "r"(rank));
  return d;
}

// Without a release: it orders tensor memory only, by the fence before it, and a
// release at the cluster's scope would wait for the thread's earlier stores (some 1000
// cycles, once for every accumulator).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                   cluster_addr)
               : "memory");
}

// ----------------------------------------------------------- one of a warp
// TMA copies, tcgen05 instructions and commits take their operands from uniform
// registers.  Issued from code that only one lane runs, each operand is moved
// there first, every time (an mma then costs its thread about 120 cycles,
// whatever its shape); so the whole warp runs that code, and the instruction
// itself is predicated on `one`, which is 1 in one lane.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one;
}

// -------------------------------------------------------------- TMA, pair
// tile into this CTA's shared memory; the bytes are counted on a barrier of
// either CTA of the pair (`bar`: its address in the cluster's window)
__device__ __forceinline__ void tma_load_2d_pair(uint32_t one, uint32_t dst, const CUtensorMap *m,
                                                 uint32_t bar, int32_t c0, int32_t c1) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "@p cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(one)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t one, uint32_t dst, const CUtensorMap *m,
                                                 uint32_t bar, int32_t c0, int32_t c1,
                                                 int32_t c2) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "@p cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(one)
      : "memory");
}

// -------------------------------------------------------------- TMA stores
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *m, uint32_t src_smem,
                                             int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(m)),
      "r"(src_smem), "r"(c0), "r"(c1)
      : "memory");
}

// element-wise addition to global memory (the type is the tensor map's)
__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap *m, uint32_t src_smem,
                                                  int32_t c0, int32_t c1) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%2, %3}], "
      "[%1];" ::"l"(reinterpret_cast<uint64_t>(m)),
      "r"(src_smem), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// at most N of this thread's store groups still read shared memory
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// every store group of this thread is complete
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ----------------------------------------------------------- tcgen05, pair
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr),
               "r"(ncols)
               : "memory");
}

// D (+)= A B^T over both CTAs' shared memory and tensor memory; issued by the
// pair's first CTA.  The descriptors come in halves, of which only the lower
// ones (with the addresses) change.
__device__ __forceinline__ void umma_bf16_pair(uint32_t one, uint32_t d_tmem, uint32_t a_lo,
                                               uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}

// arrive once on the barrier at this offset in both CTAs when every tcgen05
// operation issued so far by this thread has completed
__device__ __forceinline__ void umma_commit_pair(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster."
      "b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"(static_cast<uint16_t>(3)), "r"(one)
      : "memory");
}

// ------------------------------------------------------------- registers
// The warps of a warpgroup (four, from a multiple of four) give registers back, or
// wait for as many as they then have; by all threads of all four, which meet at a
// barrier between two such changes.
template <int BARRIER>
__device__ __forceinline__ void warpgroup_sync() {
  asm volatile("bar.sync %0, 128;" ::"n"(BARRIER) : "memory");
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace dspark
