// Bounded waits on mbarriers for kernels whose warps have roles.
#pragma once

#include "common.cuh"

namespace kvq {

// Waits for a phase of an mbarrier.  When a wait runs out, the error is set and
// every later wait of the CTA returns at once: the roles run to their ends (all
// barriers between threads are met, all accesses stay in bounds), and the
// results are void.
// try_wait gets a time for which the hardware may suspend the warp: without it
// the waiting warps' polling takes a large part of the issue slots.
__device__ __forceinline__ bool mbar_suspend_wait(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void mbar_long_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort, unsigned int *err) {
  const long long t0 = clock64();
  while (!mbar_suspend_wait(bar, parity)) {
    if (*abort) return;
    if (clock64() - t0 > kWaitTicks) {
      *abort = 1;
      set_error(err, KVQ_DEVERR_TIMEOUT);
      return;
    }
  }
}

inline __device__ __noinline__ void mbar_slow_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort,
                                                   unsigned int *err) {
  mbar_long_wait(bar, parity, abort, err);
}

struct Waiter {
  uint64_t *bars;
  volatile uint32_t *abort;
  unsigned int *err;
  __device__ __forceinline__ void operator()(int bar, uint32_t parity) const {
    if (!mbar_suspend_wait(&bars[bar], parity)) mbar_slow_wait(&bars[bar], parity, abort, err);
  }
};

// The same without a call: a kernel that moves registers between its warpgroups
// cannot have any.
struct InlineWaiter {
  uint64_t *bars;
  volatile uint32_t *abort;
  unsigned int *err;
  __device__ __forceinline__ void operator()(int bar, uint32_t parity) const {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(smem_u32(&bars[bar])), "r"(parity) : "memory");
    if (ok) return;
    if (!mbar_suspend_wait(&bars[bar], parity)) mbar_long_wait(&bars[bar], parity, abort, err);
  }
};

}  // namespace kvq
