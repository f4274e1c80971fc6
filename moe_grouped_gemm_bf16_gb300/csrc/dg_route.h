// Launchers of the routing of tokens to experts (dg_route.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace dgk {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;      // a lane of a warp per choice
constexpr int kRouteMaxGroups = 32;    // a lane (or more) per group

struct RouteFwd {
  const void* logits;    // bf16 or fp32 [T][G]
  const float* bias;     // fp32 [G] or null
  int32_t* experts;      // [T][k]
  float* weights;        // [T][k]
  int T, G, k;
  bool sigmoid;
  int groups, top_groups, best;
  bool renormalize;
  float scale;
  unsigned int* status;
};

struct RouteBwd {
  const void* logits;
  const int32_t* experts;
  const float* d_weights;   // [T][k]
  void* d_logits;           // as the logits
  int T, G, k;
  bool sigmoid, renormalize;
  float scale;
  unsigned int* status;
};

// The caller has validated the arguments.  limited: fewer SMs than the device has,
// so no grid of more blocks.
cudaError_t launch_route(const RouteFwd& a, bool bf16, int num_sms, bool limited, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteBwd& a, bool bf16, int num_sms, bool limited,
                                  cudaStream_t stream);

}  // namespace dgk
