// Launchers of the root-mean-square norm (dg_norm.cu).
#pragma once
#include <cuda_runtime.h>

namespace dgk {

constexpr int kNormMaxK = 16384;      // longest row the norm kernels hold in registers
constexpr int kNormBwdBlocks = 608;   // most rows of partial weight gradients

// Device pointers of one call; the optional ones may be null.
struct NormFwd {
  const void* X;     // bf16 [M][K]
  const void* R;     // bf16 [M][K] or null: the residual
  const void* W;     // bf16 [K]
  void* H;           // bf16 [M][K] or null: X + R
  void* Y;           // bf16 [M][K] or null
  void* Q;           // e4m3 [M][K] or null
  void* sa;          // scales of Q (fp32, or packed UE8M0 words)
  float* rstd;       // fp32 [M] or null
  int M, K, ld_sa;
  float eps;
  unsigned int* status;           // device status word and the waits' limit
  unsigned long long timeout_ns;
  unsigned int debug_flags;
};

struct NormBwd {
  const void* dY;    // bf16 [M][K]
  const void* H;     // bf16 [M][K]
  const float* rstd; // fp32 [M]
  const void* W;     // bf16 [K]
  const void* dR;    // bf16 [M][K] or null: gradient arriving at H from elsewhere
  void* dX;          // bf16 [M][K] (may be dR)
  float* dW;         // fp32 [K]
  float* part;       // fp32 [blocks][K], blocks <= min(M, kNormBwdBlocks)
  int M, K;
  unsigned int* status;
  unsigned long long timeout_ns;
  unsigned int debug_flags;
};

// The caller has validated the arguments (K % 128 == 0, K <= kNormMaxK,
// 16-byte aligned tensors).
cudaError_t norm_set_up();  // opts the kernels into their shared memory (once per device)
// limited: fewer SMs than the device has, so no grid of more blocks.
cudaError_t launch_rms_norm(const NormFwd& a, bool ue8m0, int num_sms, bool limited,
                            cudaStream_t stream);
cudaError_t launch_rms_norm_backward(const NormBwd& a, int num_sms, bool limited,
                                     cudaStream_t stream);

}  // namespace dgk
