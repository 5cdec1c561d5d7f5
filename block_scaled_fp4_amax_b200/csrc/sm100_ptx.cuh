// sm100_ptx.cuh — PTX wrappers of the tensor-core pipelines (block-scaled GEMM, attention over the 4-bit
// cache): mbarriers with bounded waits, tcgen05 fences, commits, MMAs, tensor-memory loads and
// stores, shared-memory descriptors.
#pragma once

#include <cstdint>

namespace fp4k {

constexpr unsigned long long kTimeoutNs = 2000000000ull;  // 2 s: default pipeline wait limit, and every drain wait
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Bounded wait: true when the phase completed; false when this or another role gave up.  A wait
// longer than `limit` ns records its site in the status word and tells the other roles to stop.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          uint32_t* status, uint32_t site, unsigned long long limit) {
  if (mbar_try(bar, parity)) return true;
  const unsigned long long t0 = now_ns();
  while (true) {
    if (mbar_try(bar, parity)) return true;
    if (*abort_flag) return false;
    if (now_ns() - t0 > limit) {
      atomicOr(status, 1u << site);
      *abort_flag = 1;
      return false;
    }
  }
}

// mbar_wait for code that every lane of a warp runs up to a warp-collective instruction (the
// epilogue's tcgen05.ld.sync.aligned): the lanes vote, so all of them see the same outcome (one lane
// giving up while another passes would leave the warp diverged at that instruction).  The MMA and
// scale-copy warps run their loops on every lane, lane 0 alone issuing, with no warp-collective
// instruction inside the loop: a lane that gives up simply leaves the loop early, and the lanes
// meet again at the __syncwarp after it.  (Running the loop on lane 0 alone, inside a divergent
// branch, measured 3-4% slower.)
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* status,
                                          uint32_t site, unsigned long long limit) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, status, site, limit));
}

// The same for a wait so short that a try (which may suspend the thread for longer than it takes) hardly
// ever fails: a limit of 0 looks once, without waiting, so that giving up can be brought about.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* status,
                                                uint32_t site, unsigned long long limit) {
  if (limit != 0) return mbar_wait(bar, parity, abort_flag, status, site, limit);
  if (mbar_test(bar, parity)) return true;
  atomicOr(status, 1u << site);
  *abort_flag = 1;
  return false;
}
// Drain wait (exit paths): until the phase completes or kTimeoutNs passes, whatever the flags say.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = now_ns();
  while (!mbar_try(bar, parity) && now_ns() - t0 < kTimeoutNs) {
  }
}

// After `issued` fills of a ring of `stages` full barriers (fill g on stage g % stages, phase
// parity (g / stages) & 1), wait (bounded) until the last fill of every stage has landed.
__device__ __forceinline__ void drain_fills(uint32_t full0, uint32_t issued, uint32_t stages) {
  for (uint32_t s = 0; s < stages && s < issued; ++s) {
    const uint32_t last = s + stages * ((issued - 1 - s) / stages);
    mbar_drain(full0 + 8 * s, (last / stages) & 1);
  }
}

// ---------------------------------------------------------------------------------------------
// tcgen05
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// fp16 operands without block scales (the IF4 GEMM's expanded operands): kind::f16, K = 16 per
// instruction, FP32 accumulation.
__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

#define TC_LD32(taddr, r)                                                                                   \
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15," \
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"                       \
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), \
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),        \
                 "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),      \
                 "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),      \
                 "=r"(r[29]), "=r"(r[30]), "=r"(r[31])                                                           \
               : "r"(taddr))

// Shared-memory matrix descriptor (sm_100 format, version 1) of a K-major operand tile with 128-byte
// swizzle: 8-row groups 1024 bytes apart (SBO), no LBO.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// The same for an operand whose non-contracted extent is contiguous (MN-major), 128-byte swizzle: rows of
// 64 fp16 values (128 bytes), one per k; 8-row groups 1024 bytes apart (SBO), the next 64 values of
// every row `lbo` bytes further on.
__device__ __forceinline__ uint64_t desc_sw128_mn(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}

// True in one lane of a converged warp.  Under this predicate an MMA takes 11 cycles to issue; under
// `lane == 0` it took 51 (128 x 16 x 16 MMAs back to back), too slow to queue work behind a 64-cycle one.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// kind::f16 with the A operand in tensor memory (two fp16 values of a row per 32-bit column).
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               ::"r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

#define TC_ST32(taddr, r)                                                                                          \
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"  \
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),                 \
               "r"((r)[0]), "r"((r)[1]), "r"((r)[2]), "r"((r)[3]), "r"((r)[4]), "r"((r)[5]), "r"((r)[6]), "r"((r)[7]), \
               "r"((r)[8]), "r"((r)[9]), "r"((r)[10]), "r"((r)[11]), "r"((r)[12]), "r"((r)[13]), "r"((r)[14]),         \
               "r"((r)[15]), "r"((r)[16]), "r"((r)[17]), "r"((r)[18]), "r"((r)[19]), "r"((r)[20]), "r"((r)[21]),       \
               "r"((r)[22]), "r"((r)[23]), "r"((r)[24]), "r"((r)[25]), "r"((r)[26]), "r"((r)[27]), "r"((r)[28]),       \
               "r"((r)[29]), "r"((r)[30]), "r"((r)[31]) : "memory")

}  // namespace fp4k
