// tc.cuh -- tcgen05 (5th-generation tensor core) wrappers shared by the kernels
// that use tensor memory: bounded mbarrier waits, fences, MMAs, tensor-memory
// loads and stores, operand and instruction descriptors.
#pragma once
#include "common.cuh"

namespace qnt {

__device__ __forceinline__ uint64_t gt_now() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Bounded wait (gives up `timeout` ns after the first unsuccessful try, or
// when the abort flag is raised).  max_sleep > 0: between tries the thread
// sleeps, 32 ns at first, doubling up to max_sleep ns, so a waiting warp takes
// few issue slots from the decode warps that share its scheduler and sees the
// phase complete at most ~max_sleep ns late.  max_sleep = 0: it spins, looking
// at the flag and the clock every 64 tries (the MMA issuers, whose waits are on
// the critical path).  (A suspend-time hint on try_wait instead was measured to
// wake the thread up to microseconds after the phase completed.)
__device__ __forceinline__ bool gt_wait(uint64_t* bar, uint32_t parity, volatile int* abort_s, uint64_t timeout,
                                        uint32_t max_sleep, bool cluster_scope = false) {
  const uint32_t a = smem_addr(bar);
  uint64_t deadline = 0;
  for (uint32_t n = 0, ns = 0;; ++n) {
    uint32_t done;
    if (cluster_scope)   // the phase was completed by arrivals (with release) from other CTAs of the cluster
      asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                   "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(done) : "r"(a), "r"(parity) : "memory");
    else
      asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                   : "=r"(done) : "r"(a), "r"(parity) : "memory");
    if (done) return true;
    if (max_sleep == 0 && (n & 63u) != 63u) continue;
    if (abort_s && *abort_s) return false;
    const uint64_t now = gt_now();
    if (deadline == 0) deadline = now + timeout;
    else if (now > deadline) return false;
    if (max_sleep) {
      if (ns) __nanosleep(ns);
      ns = ns ? (ns < max_sleep ? 2 * ns : max_sleep) : 32;
    }
  }
}
// Position in a ring of n slots: slot index and the parity of its current use.
struct GtRing {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1u;
    }
  }
  __device__ __forceinline__ void adv(int k, int n) {   // k <= n
    slot += k;
    if (slot >= n) {
      slot -= n;
      phase ^= 1u;
    }
  }
};
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               :: "r"(smem_addr(bar)) : "memory");
}
// D[128 x N] (+)= A[128 x 16] (tensor memory) * B[16 x N] (shared memory, descriptor)
__device__ __forceinline__ void tc_mma_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %5, %5, %5}, p;\n\t}"
      :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(0u) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&d)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]), "=r"(d[7]),
        "=r"(d[8]), "=r"(d[9]), "=r"(d[10]), "=r"(d[11]), "=r"(d[12]), "=r"(d[13]), "=r"(d[14]), "=r"(d[15])
      : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory descriptor of a K-major operand with 128-byte swizzle: rows of
// 128 bytes, 8-row groups 1024 bytes apart (LBO unused: 1), sm_100 version 1.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// Instruction descriptor of kind::f16: fp32 accumulator, A and B fp16 (or
// both bf16), K-major, M = 128, N = n.
__device__ __forceinline__ uint32_t f16_idesc(int n, int bf16) {
  return (1u << 4) | (bf16 ? ((1u << 7) | (1u << 10)) : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

}  // namespace qnt
