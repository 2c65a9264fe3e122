// tcgen05 / mbarrier helpers of the tensor-core kernels: TMEM allocation and
// loads, fences, commits issued by one elected lane, bounded waits that give
// up together.
#pragma once

#include "qmoe_internal.cuh"

namespace qmoe {

// A kernel with tensor memory takes more than half of a multiprocessor's shared memory,
// so that no two of them meet there: its allocation, which has no limit, then waits
// for nothing that a kernel launched ahead (and itself waiting for this one) holds.
constexpr int kAloneBytes = 114 * 1024;

__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// The MMA-issuing code runs on a whole converged warp and the tcgen05
// instructions are predicated on one lane chosen by elect.sync: the operands
// are then warp-uniform values.  Issued from a single divergent lane, the same
// loop reached about half the MMA rate (measured: 119 vs 65 cycles per
// 128x128x16 MMA).
__device__ __forceinline__ void tc_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
#define TC_LD32(taddr, v)                                                                               \
  asm volatile(                                                                                         \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"  \
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"                        \
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), \
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),        \
        "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),      \
        "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),      \
        "=r"(v[29]), "=r"(v[30]), "=r"(v[31])                                                           \
      : "r"(taddr)                                                                                      \
      : "memory")

#define TC_ST32(taddr, v)                                                                                \
  asm volatile(                                                                                          \
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15," \
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),              \
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), \
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),    \
      "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),    \
      "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])                 \
      : "memory")

__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups
// 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFF) >> 4);          // start address
  d |= (uint64_t)1 << 16;                           // leading byte offset (unused for SW128 K-major)
  d |= (uint64_t)(1024 >> 4) << 32;                 // stride byte offset
  d |= (uint64_t)1 << 46;                           // descriptor version
  d |= (uint64_t)2 << 61;                           // 128-byte swizzle
  return d;
}

// One poll of a phase whose answer is the same for the whole warp: every lane
// polls, lane 0's answer is broadcast.  (Each lane acting on its own answer
// can split the warp when the phase completes during the poll; the split
// halves would then reach different warp-synchronous instructions.)
__device__ __forceinline__ bool warp_test_wait(uint64_t* bar, uint32_t parity) {
  const int done = mbar_test_wait(bar, parity) ? 1 : 0;
  return __shfl_sync(0xffffffffu, done, 0) != 0;
}

// Bounded wait that also gives up when another role has aborted.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, const WaitCfg& w,
                                              volatile int* abort_flag) {
  for (long long i = 0; i < w.limit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 63 && *abort_flag) return false;
  }
  atomicExch(w.status, DEV_TIMEOUT);
  *abort_flag = 1;
  return false;
}

// Bounded wait with non-blocking polls: for the MMA-issuing thread, whose loop
// paces the whole pipeline (a parked poll costs ~250 cycles even when the
// phase has already completed).
__device__ __forceinline__ bool spin_or_abort(uint64_t* bar, uint32_t parity, const WaitCfg& w,
                                              volatile int* abort_flag) {
  const long long limit = w.limit * 64;
  for (long long i = 0; i < limit; ++i) {
    if (mbar_test_wait(bar, parity)) return true;
    if ((i & 255) == 255 && *abort_flag) return false;
  }
  atomicExch(w.status, DEV_TIMEOUT);
  *abort_flag = 1;
  return false;
}

// Waits for the barriers of the last S of `it` stages, with a limit: for copies in
// flight (after a wait that ran out they must land before the CTA leaves), or for the
// commits that free the stages.  A commit arrives on its own, some time after its MMAs,
// and nothing says that the arrivals of two come in order: none may come to a CTA that
// has left, where it would change another CTA's shared memory, so the producer waits
// for each stage's last.
template <int S>
__device__ __forceinline__ void drain_ring(uint64_t* bars, int it, int* status, long long polls) {
  const WaitCfg drain{status, polls};
  for (int i = it > S ? it - S : 0; i < it; ++i) mbar_wait_bounded(&bars[i % S], (i / S) & 1, drain);
}
// Parked polls (about 4 ms) that a copy in flight, or a commit, is given after a wait
// that ran out.
constexpr long long kDrainPolls = 4096;

__device__ __forceinline__ void mbar_arrive_expect_tx_elect(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)), "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void bulk_g2s_elect(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

}  // namespace qmoe
