// Bounded waits on shared-memory barriers for the pipelined kernels.  A wait that lasts
// longer than the limit raises KD_DEV_TIMEOUT and sets the CTA's abort flag, which ends
// every other wait of the CTA: all roles fall through to the common teardown.
#pragma once

#include "kd_common.cuh"
#include "kd_ptx.cuh"

namespace kd {

constexpr uint64_t PIPE_LIMIT_NS = 2000000000ull;      // 2 s per wait

// The rest of a wait that did not succeed at once.  Everything by value: a wait's state
// stays in registers.  drain: keeps waiting through an abort (used to let copies land before
// the CTA leaves).  remote: arrivals come from other CTAs of the cluster.
static __device__ __noinline__ bool pipe_wait_slow(uint32_t bar, uint32_t par, volatile uint32_t* abort_flag,
                                                   int32_t* err, bool drain, bool remote) {
  uint64_t t0 = 0;
  for (uint32_t spin = 1;; ++spin) {
    if (remote ? ptx::mbar_try_wait_cluster(bar, par) : ptx::mbar_try_wait(bar, par)) return true;
    if ((spin & 31u) == 0u) {
      if (!drain && *abort_flag) return false;
      const uint64_t t = ptx::globaltimer();
      if (t0 == 0) t0 = t;
      else if (t - t0 > PIPE_LIMIT_NS) {
        *abort_flag = 1u;
        raise_dev_error(err, KD_DEV_TIMEOUT);
        return false;
      }
    }
  }
}

struct Pipe {
  uint32_t base;                     // shared address of the barriers
  volatile uint32_t* abort_flag;
  int32_t* err;
  __device__ __forceinline__ uint32_t bar(int i) const { return base + 8u * (uint32_t)i; }

  // Phase with parity `par` of barrier i complete?  False only when the wait was given up.
  __device__ __forceinline__ bool wait(int i, uint32_t par) const {
    return ptx::mbar_try_wait(bar(i), par) || pipe_wait_slow(bar(i), par, abort_flag, err, false, false);
  }
  __device__ __forceinline__ bool wait_remote(int i, uint32_t par) const {
    return ptx::mbar_try_wait_cluster(bar(i), par) || pipe_wait_slow(bar(i), par, abort_flag, err, false, true);
  }
  __device__ __forceinline__ void drain(int i, uint32_t par) const {
    if (!ptx::mbar_try_wait(bar(i), par)) pipe_wait_slow(bar(i), par, abort_flag, err, true, false);
  }
  // The same for a whole warp, with one outcome.
  __device__ __forceinline__ bool wait_warp(int i, uint32_t par) const {
    return __all_sync(0xffffffffu, wait(i, par));
  }
};

}  // namespace kd
