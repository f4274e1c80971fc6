// Launchers of the gated activation with 8-bit checkpoints (dg_swiglu.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace dgk {

// Device pointers of one call; the optional ones may be null.  Batches z of
// M rows; with masked_m only rows m < masked_m[z] are read and written.
struct SwigluFwd {
  const void* GU;           // bf16 [G][M][2 I]: gate columns, then up columns
  void* Y;                  // bf16 [G][M][I] or null
  void* Q;                  // e4m3 [G][M][I] or null
  void* sa;                 // scales of Q (fp32 [G][I/128][ld], or packed UE8M0)
  void* CQ;                 // e4m3 [G][M][2 I] or null: the checkpoint of GU
  float* csa;               // fp32 [G][2 I / 128][ld]
  const int32_t* masked_m;  // int32 [G] or null
  int G, M, I, ld;
  unsigned int* status;           // device status word and the waits' limit
  unsigned long long timeout_ns;
  unsigned int debug_flags;
};

struct SwigluBwd {
  const void* CQ;
  const float* csa;
  const void* dY;           // bf16 [G][M][I]
  void* dGU;                // bf16 [G][M][2 I]
  void* Y;                  // bf16 [G][M][I] or null: the activation again
  const int32_t* masked_m;
  int G, M, I, ld;
  unsigned int* status;
};

// The caller has validated the arguments (I % 128 == 0, I / 128 <= 32767, G <=
// 65535, 16-byte aligned tensors, ld >= M).  limited: fewer SMs than the device
// has, so no grid of more blocks.
cudaError_t swiglu_set_up();  // opts the kernels into their shared memory (once per device)
cudaError_t launch_swiglu(const SwigluFwd& a, bool ue8m0, int num_sms, bool limited,
                          cudaStream_t stream);
cudaError_t launch_swiglu_backward(const SwigluBwd& a, int num_sms, bool limited,
                                   cudaStream_t stream);

}  // namespace dgk
