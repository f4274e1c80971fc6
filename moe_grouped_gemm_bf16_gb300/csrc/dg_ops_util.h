// Checks that the host files of the operators around the GEMMs share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "dg_host.h"

namespace dgk {

inline dg_status cuda_fail(cudaError_t e, const char* what) {
  return host_fail(DG_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }

// Opts an operator's kernels into their shared memory, once per device.
template <cudaError_t (*SET_UP)()>
dg_status set_up_once(int device) {
  static std::atomic<bool> done[kHostMaxDevices];
  if (done[device].load(std::memory_order_acquire)) return DG_OK;
  const cudaError_t e = SET_UP();
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(max dynamic shared memory)");
  done[device].store(true, std::memory_order_release);
  return DG_OK;
}

}  // namespace dgk
