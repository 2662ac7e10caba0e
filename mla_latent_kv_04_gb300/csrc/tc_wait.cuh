// Bounded mbarrier waits shared by the tensor-core kernels of the prefix and key-weight calls.
#pragma once
#include "common.cuh"
#include "sm100_ptx.cuh"

namespace mla {

constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Polls until the barrier's phase `parity` has completed; false if another wait of this CTA has
// given up, or if this one does (after two seconds: the abort flag is set, MLA_ERR_TIMEOUT is
// recorded).
// kCluster: acquire what another CTA of the cluster wrote before it arrived.
template <bool kCluster = false>
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                             int32_t* status) {
  auto probe = [&]() {
    return kCluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity);
  };
  if (probe()) return true;
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
    if (probe()) return true;
    if (*abort) return false;
    if (ptx::globaltimer() - t0 > kWaitLimitNs) {
      *abort = 1;
      flag_status(status, MLA_ERR_TIMEOUT);
      return false;
    }
  }
}

// After an abort: wait (at most a second) for copies or MMAs still in flight on this barrier.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity) && ptx::globaltimer() - t0 < kWaitLimitNs / 2) {
  }
}

}  // namespace mla
