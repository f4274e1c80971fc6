// State and error reporting that the host files of the C ABI share (defined in
// dg_host.cu).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "dg.h"

namespace dgk {

constexpr int kHostMaxDevices = 64;

struct HostState {
  int device;                     // index, below kHostMaxDevices
  int sms;                        // SMs the kernels may use
  int device_sms;                 // SMs of the device (above sms under a limit)
  unsigned int* status;           // device status word
  unsigned long long timeout_ns;  // limit of every wait inside a kernel
  unsigned int debug_flags;
  PFN_cuTensorMapEncodeTiled_v12000 encode;
};

// Records the detail dg_last_error_string() returns, and returns `s`.
dg_status host_fail(dg_status s, const char* fmt, ...);
dg_status host_ok();
// The current device's state, set up on first use.
dg_status host_state(HostState* out);

}  // namespace dgk
