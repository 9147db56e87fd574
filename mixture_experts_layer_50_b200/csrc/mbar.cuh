// mbarriers with bounded waits, shared by the kernels that are fed by asynchronous copies.
#pragma once

#include "common.cuh"

namespace moe {
namespace tc {

constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// ---- mbarrier ------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Polls after which a wait gives up even if the global timer did not advance (a backstop:
// each poll takes well over 20 ns, so this is more than a second).
constexpr uint64_t kWaitMaxPolls = 50000000ull;

// Wait for the phase of `parity` to complete.  Gives up (false) when another role of the
// CTA has given up, or after limit_ns, recording a timeout.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity,
                                          volatile int* abort_flag, int* status,
                                          uint64_t limit_ns = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint64_t polls = 0;; ++polls) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > limit_ns || polls > kWaitMaxPolls) {
      *abort_flag = 1;
      report_status(status, kStatusTimeout);
      return false;
    }
  }
}

// Wait, after an abort, for copies or MMAs this thread already issued (their barrier phase
// completes when they land); bounded by the same time limit and poll backstop as mbar_wait,
// and records nothing: the abort is reported already.
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  for (uint64_t polls = 0; polls <= kWaitMaxPolls; ++polls)
    if (mbar_try_wait(bar, parity) || global_timer_ns() - t0 >= kWaitLimitNs) return;
}

}  // namespace tc
}  // namespace moe
