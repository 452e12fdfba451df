// Bounded mbarrier waits of the sequence-block kernels.  The clock is read only
// after many failed tries, so that a short wait does not pay for it.
#pragma once

#include "tc_common.cuh"

namespace lr {

constexpr long long kWaitNs = 2000000000LL;

// Waits for the phase of `parity` to end (CLUSTER: and acquires what other blocks
// of the cluster stored before).  false once the limit has passed or
// another wait has recorded a failure; the first to give up records it.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, int* status) {
  unsigned long long t0 = 0;
  for (unsigned it = 1;; ++it) {
    if (CLUSTER ? tc::mbar_try_wait_cluster(bar, parity) : tc::mbar_try_wait(bar, parity)) return true;
    if ((it & 1023u) != 0) continue;
    if (ld_volatile_int(status) != kDevOk) return false;
    const unsigned long long t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    if ((long long)(t - t0) > kWaitNs) {
      atomicCAS(status, kDevOk, kDevTimeout);
      return false;
    }
  }
}

}  // namespace lr
