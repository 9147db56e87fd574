// mbarriers with bounded waits, for kernels whose warps hand shared memory to one another.
#pragma once

#include "common.cuh"

namespace moe {
namespace mbar {

__device__ __forceinline__ uint32_t address(const uint64_t* bar) {
  return (uint32_t)__cvta_generic_to_shared(bar);
}
__device__ __forceinline__ void init(uint64_t* bar, uint32_t arrivals) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(address(bar)), "r"(arrivals));
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(address(bar)) : "memory");
}
__device__ __forceinline__ bool done(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(address(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Waits for the phase of `parity` to complete.  Gives up (false) when another warp of the block
// has, or after two seconds (or, should the timer stand still, 50 million polls of over 20 ns),
// and records a timeout.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* given_up,
                                     int* status) {
  if (done(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t polls = 0;; ++polls) {
    if (done(bar, parity)) return true;
    if (*given_up) return false;
    if (global_timer_ns() - t0 > 2000000000ull || polls > 50000000u) {
      *given_up = 1;
      __threadfence_block();  // before whatever the caller does without having waited
      report_status(status, kStatusTimeout);
      return false;
    }
  }
}

}  // namespace mbar
}  // namespace moe
