// Bounded mbarrier waits shared by the tensor-core kernels of the prefix, key-weight, page and 4-bit calls.
#pragma once
#include "common.cuh"
#include "sm100_ptx.cuh"

namespace mla {

constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Polls until the barrier's phase `parity` has completed; false if another wait of this CTA has
// given up, or if this one does (after `limit_ns`: the abort flag is set, MLA_ERR_TIMEOUT is
// recorded).
// kCluster: acquire what another CTA of the cluster wrote before it arrived.
template <bool kCluster = false>
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                             int32_t* status, uint64_t limit_ns = kWaitLimitNs) {
  auto probe = [&]() {
    return kCluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity);
  };
  if (probe()) return true;
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)               // (the clock is slow to read)
      if (probe()) return true;
    if (*abort) return false;
    if (ptx::globaltimer() - t0 > limit_ns) {
      *abort = 1;
      flag_status(status, MLA_ERR_TIMEOUT);
      return false;
    }
  }
}

// After an abort: wait (at most half the limit) for copies or MMAs still in flight on this barrier.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity) && ptx::globaltimer() - t0 < limit_ns / 2) {
  }
}

}  // namespace mla
