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

// What becomes of a tile's sums: D itself, or, of the loss over a vocabulary, the
// logits' largest values and sums (nt), the gradient of the logits (nt), or a
// multiple of them, added up over pieces of the vocabulary (nn, tn).
enum BfEpilogue : int { kBfPlain = 0, kBfStats = 1, kBfGrad = 2, kBfSum = 3 };

struct BfLoss {
  // nt: the rows of A are the words word0 .. of `words` and the rows of B tokens, or
  // (words_on_lanes) the other way round
  bool words_on_lanes;
  const int32_t* targets;   // [tokens]: a word, or outside [0, words)
  int words, word0, tokens;
  // stats: per share of a tile's words and token the largest logit times log2(e) and
  // the sum of 2^(z log2(e) - it); the target's logit where there is a target
  float2* pair;             // [pairs][tokens]
  float* hit;               // [tokens]
  int pairs;
  // gradient: D [tokens][pitch] = (softmax - 1 at the target) * d_loss
  const float* lse;         // [tokens]
  const float* d_loss;      // [tokens], taken relative to *unit
  int pitch;
  // sum: fp32, shaped like D; first: nothing before, last: D = *unit times it is written
  // (first of a gradient: *unit is found and written).  With parts > 1 (nn): parts of the
  // reduction, `depth` deep, a sum for each
  float* sum;
  float* unit;
  int parts, depth;
  bool first, last;
};

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
  const int32_t* sizes;  // [G] rows of each group (null: G = 1, all rows)
  int G;
  int rows;              // rows of A (all groups)
  int M;                 // tn: rows of each D[e]
  int N, K;              // K unused by tn (its reduction runs over the rows)
  int pitch;             // elements from row to row of A (0: K, tn: M), a multiple of 8
  BfEpilogue epilogue;
  BfLoss loss;
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

// The plan that dg_debug_force_ragged_plan asks for (lanes = 0: none).
BfPlan bf16_forced_plan();

// CTAs of the plan's grid.
long long bf16_grid(const BfCall& c, const BfPlan& plan, int num_sms);

// The form for a few rows in all (dg_bf16_few.cu): whether it takes the call, and
// its launch.
bool bf16_few_rows(const BfCall& c);
cudaError_t launch_bf16_few(const BfCall& c, int num_sms, cudaStream_t stream);

}  // namespace dgk
