// Launcher of the bf16 products grouped by expert with ragged sizes
// (dg_bf16.cu).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dgk {

// nt: D[t] = A[t] B[e]^T, B [G][N][K];  nn: D[t] = A[t] B[e], B [G][K][N];
// tn: D[e] = A_e^T B_e over the group's rows of A [K][M] and B [K][N].
enum BfForm : int { kBfNT = 0, kBfNN = 1, kBfTN = 2 };

constexpr int kBfMaxGroups = 1024;

// How a call is tiled: CTA pairs or single CTAs, columns and rows of D per tile,
// CTAs (pairs) that share a tile's reduction.
struct BfPlan {
  bool pair;
  int lanes, bc, split;
};

struct BfCall {
  BfForm form;
  const void* A;
  const void* B;
  const void* C;         // tn: addend shaped like D, or null
  void* D;
  const int32_t* sizes;  // [G] rows of each group
  int G;
  int rows;              // rows of A (all groups)
  int M;                 // tn: rows of each D[e]
  int N, K;              // K unused by tn (its reduction runs over the rows)
  unsigned int* status;
  unsigned long long timeout_ns;
  unsigned int debug_flags;
  bool limited;          // fewer SMs than the device has: no grid of more CTAs
  BfPlan forced;         // lanes > 0: this plan (tests)
};

// Opts the kernels into their shared memory (once per device).
cudaError_t bf16_set_up();
// The caller has validated the arguments.  Returns cudaErrorInvalidValue if a
// tensor map could not be encoded.
cudaError_t launch_bf16_grouped(const BfCall& c, PFN_cuTensorMapEncodeTiled_v12000 encode,
                                int num_sms, cudaStream_t stream);

// CTAs of the plan's grid.
long long bf16_grid(const BfCall& c, const BfPlan& plan, int num_sms);

// The form for a few rows in all (dg_bf16_few.cu): whether it takes the call, and
// its launch.
bool bf16_few_rows(const BfCall& c);
cudaError_t launch_bf16_few(const BfCall& c, int num_sms, cudaStream_t stream);

}  // namespace dgk
