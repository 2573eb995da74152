// hyb_tcgen05.cuh -- helpers of the kernels that run on the 5th-generation
// tensor cores: operand descriptors, commits, fences, tensor-memory reads and
// the bounded wait of their rings.
#pragma once

#include "hyb_internal.cuh"

namespace hyb {

// Tensor memory of kernels that are programmatic dependents and allocate it before
// griddepcontrol.wait.  A CTA that holds some while it waits must not keep it from a
// CTA of the kernel it waits for: those that can share an SM never need more than its
// 512 columns together.  Shared memory sees to that, asserted beside each kernel: a
// CTA takes more than a third of an SM's for up to 256 columns, so that two fit an SM,
// and more than two thirds for 512, so that no other fits beside it.
constexpr int kSmemPerSm = 228 << 10;
constexpr bool tmem_fits(int columns, int smem) {
  return smem > (columns <= 256 ? kSmemPerSm / 3 : kSmemPerSm / 3 * 2);
}

// Shared-memory matrix descriptor of a K-major operand in the 128-byte
// swizzle layout: rows 128 bytes apart, 8-row groups 1024 bytes apart
// (stride byte offset), descriptor version 1, layout type 2 (128B swizzle).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1 << 16;             // leading byte offset (unused by swizzled K-major)
  d |= (uint64_t)(1024 >> 4) << 32;   // stride byte offset
  d |= (uint64_t)1 << 46;             // version
  d |= (uint64_t)2 << 61;             // 128-byte swizzle
  return d;
}

// arrives on the mbarrier once every tcgen05.mma this thread issued before
// has completed
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::
                   "r"(smem_u32(bar))
               : "memory");
}
// the same from a warp that runs as a whole, by its leader
__device__ __forceinline__ void umma_commit_if(uint32_t leader, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
// 16 consecutive fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int q = 0; q < 16; ++q) v[q] = __uint_as_float(r[q]);
}

// Waits for the mbarrier phase of the given parity.  The thread sleeps in
// mbarrier.try_wait with an explicit suspend-time hint: in this pipeline a
// blocked try_wait without one woke up late enough to cost most of a
// microsecond per ring slot.  Gives up (returns false) after about 2^31 SM
// clocks, so a phase that never completes ends the CTA's pipeline.
__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity) {
  long long t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(200000u)  // hint: 200 us
        : "memory");
    if (ok) return true;
    const long long now = clock64();
    if (t0 == 0) t0 = now;  // (the clock is read only where the first try did not do)
    if (now - t0 >= (1ll << 31)) return false;
  }
}

}  // namespace hyb
