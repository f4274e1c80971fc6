// Bounded mbarrier waits and the device status word, shared by the kernels.
// P: a kernel's parameters, of which `status` and `timeout_ns` are read.
#pragma once
#include <cstdint>

#include "dg_params.h"
#include "ptx.cuh"

namespace dgk {

template <class P>
__device__ __forceinline__ void raise_status(const P& p, unsigned int code) {
  atomicCAS(p.status, 0u, code);
}

// Checked build: record a failed check and abort the CTA (every later wait
// returns at once and no further TMA or MMA is issued).
template <class P>
__device__ __forceinline__ void dbg_fail(const P& p, unsigned int code,
                                         volatile uint32_t* abort_flag) {
  raise_status(p, code);
  *abort_flag = 1;
}

// Checked build: whether [at, at + n) lies in a tensor of `extent` elements (else
// the access is to be skipped, and is reported).  Nothing in the regular build.
template <class P>
__device__ __forceinline__ bool in_bounds(const P& p, size_t at, size_t n, size_t extent) {
  if constexpr (kDebug) {
    if (at > extent || n > extent - at) {
      raise_status(p, ST_DEBUG_BOUNDS);
      return false;
    }
  }
  return true;
}

// Bounded mbarrier wait.  Returns false (without waiting) once the CTA has
// aborted, or after `timeout_ns`, in which case it records the timeout and
// aborts the CTA.
template <bool ACQ_CLUSTER = false, class P>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                         const P& p) {
  auto try_once = [&]() {
    return ACQ_CLUSTER ? mbar_try_wait_acq_cluster(bar, parity) : mbar_try_wait(bar, parity);
  };
  if (try_once()) return true;
  if (*abort_flag) return false;
  const uint64_t t0 = globaltimer_ns();
  uint32_t it = 0;
  while (!try_once()) {
    if ((++it & 15u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > p.timeout_ns) {
        raise_status(p, ST_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
  return true;
}

// Wait used while draining at the end: ignores the abort flag, gives up only
// on the time limit.
template <class P>
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, const P& p) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > p.timeout_ns) {
      raise_status(p, ST_TIMEOUT);
      return;
    }
  }
}

}  // namespace dgk
