// wait.cuh -- waiting on barriers and issuing tensor-core work by a warp.
#pragma once

#include "common.cuh"

namespace pkv {

// The bounded barrier wait of common.cuh in few instructions, for kernels whose roles run
// side by side on an SM: unrolled polls of thirty wait sites (9 KB of code each) push the
// roles' loops out of the instruction cache.
//
// As mbar_wait: false (after setting PKV_DEV_TIMEOUT) when the time limit passes, or
// when *abort is set.
__device__ __forceinline__ bool short_wait(uint32_t bar, uint32_t parity, int32_t* status,
                                           volatile int32_t* abort = nullptr) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
#pragma unroll 1
  for (int i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) != 0) continue;
    if (abort && *abort) return false;
    const uint64_t now = globaltimer();
    if (t0 == 0) t0 = now;
    if (now - t0 > PKV_WAIT_TIMEOUT_NS) {
      set_status(status, PKV_DEV_TIMEOUT);
      if (abort) *abort = 1;
      return false;
    }
  }
}

// True for one lane of the (converged) warp, in a form that tells the compiler
// so: the tcgen05 instructions then take their operands from uniform
// registers without a loop over lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

}  // namespace pkv
