// Device functions that the kernels beside the KDA layers share.
#pragma once

#include "kda_common.cuh"
#include "kda_hybrid.h"
#include "kda_sm100.cuh"

namespace kda {

// log(1 + e^x), without overflow for large x
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

namespace sm100 {

// Waits for the phase; after about two seconds records the timeout in the status word and the CTA's abort flag, and later
// waits return at once.  (The clock is read only after many tries.  All lanes of a warp wait: measured, a warp is back 70
// cycles after the arrival so, 290 where one lane polls and the others wait for it.)
__device__ __forceinline__ void wait_or_abort(uint64_t *bar, uint32_t parity, volatile uint32_t *abort_flag,
                                              uint32_t *status) {
  if (mbar_try_wait(bar, parity)) return;
  if (*abort_flag) return;
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if ((i & 255u) == 0) {
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > 2000000000ull) break;
    }
  }
  *abort_flag = 1;
  atomicOr(status, KDA_DEVICE_TIMEOUT);
}

}  // namespace sm100
}  // namespace kda
