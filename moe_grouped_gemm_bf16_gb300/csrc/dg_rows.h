// Launchers of what moves rows between tokens and experts (dg_rows.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace dgk {

constexpr int kRowsMaxExperts = 1024;
constexpr int kRowsMaxTopK = 32;   // a lane of a warp per choice

enum RowsLayout : int { kRowsRagged = 0, kRowsContiguous = 1, kRowsMasked = 2 };

// Rows of the experts from the tokens' choices.
struct RowsCall {
  const int32_t* experts;   // [pairs]: -1, or an expert
  int32_t* sizes;           // [G]
  int32_t* rows;            // [pairs]
  int32_t* m_indices;       // contiguous: [room]
  int pairs;                // tokens x choices
  int G;
  int room;                 // contiguous: rows in all; masked: rows of each expert
  unsigned int* status;
};

// Rows of 16-byte vectors from the tokens' matrix into the experts'.
struct DispatchCall {
  const void* X;            // [T][vecs]
  const int32_t* rows;      // [T][k]
  void* D;                  // [num_rows][vecs]
  int T, k, vecs;
  int num_rows;
  // scales of four bytes each (null: none): [kb][ld] -> [num_rows / per][kb][ld_out]
  const uint32_t* sa;
  uint32_t* sa_out;
  int kb, ld, ld_out, per;  // per: rows of D that share a matrix of scales
  unsigned int* status;
};

struct CombineCall {
  const void* Y;            // bf16 [num_rows][K]
  const int32_t* rows;      // [T][k]
  const float* weights;     // [T][k] or null
  const void* R;            // bf16 [T][K] or null
  void* out;                // bf16 [T][K]
  int T, K, k, num_rows;
  unsigned int* status;
};

struct CombineBwd {
  const void* dO;           // bf16 [T][K]
  const void* Y;            // bf16 [num_rows][K] (with dw)
  const int32_t* rows;
  const float* weights;     // [T][k] or null
  void* dY;                 // bf16 [num_rows][K]
  float* dw;                // [T][k] or null
  int T, K, k, num_rows;
  unsigned int* status;
};

// The caller has validated the arguments.  limited: fewer SMs than the device has,
// so no grid of more blocks.
cudaError_t rows_set_up();   // opts the kernels into their shared memory (once per device)
cudaError_t launch_rows(const RowsCall& a, RowsLayout layout, int num_sms, cudaStream_t stream);
cudaError_t launch_dispatch(const DispatchCall& a, int num_sms, bool limited, cudaStream_t stream);
cudaError_t launch_combine(const CombineCall& a, int num_sms, bool limited, cudaStream_t stream);
cudaError_t launch_combine_backward(const CombineBwd& a, int num_sms, int device_sms,
                                    cudaStream_t stream);

// Threads of a block, blocks per SM and 16-byte vectors that a thread has in flight in combine
// and its gradient (dg_rows.cu says why).
constexpr int kSumThreads = 256, kSumPerSm = 3, kSumLoads = 8;

// Threads to a token in the gradient of combine, `rows` of its k rows of `vecs` vectors at a
// time: those with the least rounds of tokens times what one takes (a round of loads for each of its
// iterations, and one more for the sums): 9451 tokens of one row of 360 take 9.3, 14, 24 and 39 us
// with 32, 64, 128 and 256, 480 of 8 rows of 7688 82, 48, 34 and 35, 4096 of 8 rows of 7168 216,
// 185, 170 and 174.  (By the whole device's SMs, whatever the limit: the sums' order is the
// team's.)
inline int combine_team(int T, int vecs, int k, int rows, int device_sms) {
  const long long threads = 1ll * device_sms * kSumPerSm * kSumThreads;
  int best = kSumThreads;
  long long least = -1;
  for (int team = kSumThreads; team >= 32; team /= 2) {
    const long long each = team * (kSumLoads / rows);
    const long long turns = (vecs + each - 1) / each * ((k + rows - 1) / rows);
    const long long cost = ((T + threads / team - 1) / (threads / team)) * (1 + turns);
    if (least < 0 || cost < least) {
      least = cost;
      best = team;
    }
  }
  return best;
}

}  // namespace dgk
