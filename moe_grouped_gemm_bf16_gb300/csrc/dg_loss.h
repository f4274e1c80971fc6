// Launcher of the softmax cross entropy of a product over a vocabulary (dg_loss.cu).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dg_bf16.h"

namespace dgk {

struct LossCall {
  const void* X;            // bf16 [T][K]
  const void* W;            // bf16 [V][K]
  const int32_t* targets;   // [T]
  float* loss;              // [T] or null
  float* lse;               // [T] or null (backward: read)
  const float* d_loss;      // [T] (backward)
  void* dX;                 // bf16 [T][K] or null
  void* dW;                 // bf16 [V][K] or null
  void* workspace;
  int T, V, K;
  unsigned int* status;
  unsigned long long timeout_ns;
  unsigned int debug_flags;
  bool limited;             // fewer SMs than the device has: no grid of more CTAs
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  BfPlan forced;            // lanes > 0: this plan (tests; the logits' product without a split,
                            // the gradients' in whole 64-wide boxes)
};

// Whether T tokens have the words on the accumulator's lanes, in tiles of multiples of 32
// (else of 64).
bool loss_words_on_lanes(long long T);

// Workspace of a call, in bytes.
long long loss_workspace(long long T, long long V);
long long loss_backward_workspace(long long T, long long V, long long K);

cudaError_t loss_set_up();   // opts the kernels into their shared memory (once per device)
// The caller has validated the arguments (T > 0).  cudaErrorInvalidValue if a tensor
// map could not be encoded.
cudaError_t launch_loss(const LossCall& a, int num_sms, cudaStream_t stream);
cudaError_t launch_loss_backward(const LossCall& a, int num_sms, cudaStream_t stream);

}  // namespace dgk
