// Inline-PTX wrappers for pairs of CTAs (cta_group::2): the two CTAs of a
// cluster whose ranks differ in the last bit run one MMA on both SMs, issued
// by one thread of the even CTA.  A (M rows) and B (N rows) are split in
// halves over the two CTAs' shared memory, at the same offsets in both; each
// CTA's TMEM holds the accumulator rows of its half of M (M = 256: 128 lanes).
// No multicast TMA loads.
#pragma once

#include "sm100.cuh"

namespace mla {
namespace sm100 {

// One thread of the warp (all lanes call it).  MMAs belong in a region chosen
// by this election: the compiler then knows that one thread runs it and keeps
// descriptors in uniform registers.  Measured with M = 256, N = 256: 128
// cycles per MMA (the pipe's rate) against 186-237 in a region of `lane == 0`,
// where the issue is the bound whatever N.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// One warp of each CTA of the pair calls these.
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void pair_tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// D[tmem of both] (+)= A * B, bf16 operands, fp32 accumulation.
__device__ __forceinline__ void pair_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with A in TMEM: row i of a CTA's half of M in lane i, two
// consecutive elements of K per 32-bit column, from column `a` on.
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// In both CTAs, 128 rows x 32 bytes from shared memory into eight columns of
// TMEM.  MMAs that this thread issues later read the copied values.
__device__ __forceinline__ void pair_cp_128x32b(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.128x256b [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Arrive on the barrier at local offset `bar` in every CTA of `mask` once all
// MMAs and copies this thread issued have completed.
__device__ __forceinline__ void pair_commit(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

// TMA load into this CTA whose bytes are counted on a barrier of either CTA of
// the pair (`bar`: a cluster address from map_to_rank).
__device__ __forceinline__ void pair_tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// The same for a box of a 3-D map [chunk][row][64 columns], one instruction for
// several 64-column chunks.
__device__ __forceinline__ void pair_tma_load_3d(uint32_t dst, const CUtensorMap* map, int row, int chunk, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(chunk), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_chunks(uint32_t dst, const CUtensorMap* map, int row, int chunk, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(chunk), "r"(bar)
      : "memory");
}

// Bounded wait that polls without sleeping, for the threads whose next step
// feeds the tensor pipe (measured in the chunk kernel: 2 % of the call with
// the K producer's sleeps gone, another 1.5 % with the MMA thread's).
__device__ __forceinline__ bool spin_phase(uint32_t bar, uint32_t parity, const WaitCtx& w) {
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    if (mbar_test_wait(bar, parity)) return true;
    if ((i & 31u) == 0) {
      if (*w.abort) return false;
      if (clock64() - t0 > w.limit) {
        atomicOr(w.err, kErrTimeout);
        *w.abort = 1;
        return false;
      }
    }
  }
}

// Arrive on a barrier of any CTA of the cluster (cluster address) without
// releasing earlier writes: a release at cluster scope costs 0.5 us here
// (measured: producers that arrived with one issued a 16 KB load per 0.6 us),
// so hand-offs of TMEM, which tcgen05 fences order, do without.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

}  // namespace sm100
}  // namespace mla
