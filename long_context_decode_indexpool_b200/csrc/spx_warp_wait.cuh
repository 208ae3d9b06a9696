// The bounded mbarrier wait of whole warps.
#pragma once

#include "spx_device.cuh"

namespace spx {

constexpr uint32_t kSuspendNs = 1000000;

// One attempt, suspended until the phase completes or `ns` have passed.
__device__ __forceinline__ bool mbar_try_wait_for(uint32_t addr, uint32_t parity, uint32_t ns) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(addr), "r"(parity), "r"(ns)
      : "memory");
  return done != 0;
}

// What follows an attempt of a whole millisecond: never in a run that works.  Out
// of line, so that the loops around the 4-bit attention's twelve waits hold none of
// it (whole cache 4 x 1M 665 us with it inlined, 649 so; a chunk of 1,024
// selections 483 and 479).
static __device__ __noinline__ bool warp_wait_on(uint32_t addr, uint32_t parity,
                                                 volatile int* abort, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_for(addr, parity, kSuspendNs)) {
    if (*abort || globaltimer_ns() - t0 > limit_ns) {
      if (!*abort) atomicExch(&g_device_error, kErrWaitTimeout);
      *abort = 1;
      return false;
    }
  }
  return true;
}

// mbar_wait made by every lane of a warp, suspended for up to a millisecond at a
// time (the waiting warps of a CTA then leave the issue slots to the working ones).
// `ok` is the lane's last answer: a lane whose wait gave up looks at later barriers
// once, without suspending, so what is left of its warp's work waits for nothing
// more.  The lanes' answers may differ only after a timeout.
__device__ __forceinline__ bool warp_wait(bool ok, uint64_t* bar, uint32_t parity,
                                          volatile int* abort, uint64_t limit_ns = kWaitLimitNs) {
  const uint32_t addr = smem_u32(bar);
  if (!mbar_try_wait_for(addr, parity, ok ? kSuspendNs : 0) && ok)
    ok = warp_wait_on(addr, parity, abort, limit_ns);
  __syncwarp();
  return ok;
}

}  // namespace spx
