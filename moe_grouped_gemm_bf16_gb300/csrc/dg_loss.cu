// Softmax cross entropy of the product z = X W^T over a vocabulary of V words, in
// pieces that stay on the chip, and its gradient.  Per token t, with y its target:
//
//   lse = log sum_v exp(z_v);   loss = lse - z_y        (0 without a target)
//   p_v = (exp(z_v - lse) - [v = y]) d_loss             (0 without a target)
//   dX = p W,   dW = p^T X
//
// Forward: the bf16 product's kernel (dg_bf16_kernel.cuh, form nt) with W's rows on
// the accumulator's columns and tokens on its lanes.  A lane then has 256 logits of
// one token, and leaves the largest of them and the sum of the exponentials relative to
// it; a second kernel joins the tiles' pairs.  The logits never leave tensor memory.
//
// Backward: per piece of the vocabulary the logits again, whose epilogue writes p in
// bf16 (as every operand of these products; one rounding, by 2^-9 of itself at most),
// then the piece's rows of dW (form tn) and its share of dX (form nn), which is added
// up in fp32 over the pieces and rounded once with the last.  p is written relative
// to the largest |d_loss|, the unit, and the products' sums are multiplied by it: with
// the same d_loss for all tokens, as in a mean, its rounding then is none of p's, and
// the -1 at the targets, the largest entries of all, stay near -1 (with d_loss in p,
// 1 / T rounded to bf16 in every token's largest entry: dX and dW off by up to 0.0037
// of themselves, so 0.0017, which is their own rounding).  A piece is as wide as makes
// p about 96 MB, which L2 holds until both products have read it.
//
// Bounded by the tensor cores; with few tokens by reading W (and writing dW).
#include <algorithm>

#include "dg_bf16_kernel.cuh"
#include "dg_launch.h"
#include "dg_loss.h"

namespace dgk {
namespace {

constexpr long long kPieceBytes = 96ll << 20;   // of p
constexpr int kPieceLeast = 4096;               // words: whole waves of tiles

long long round_up(long long x, long long to) { return (x + to - 1) / to * to; }

// Words of a piece, a multiple of 8 (of 256 where there are more pieces).
long long piece_words(long long T, long long V) {
  const long long most = std::max<long long>(kPieceLeast, kPieceBytes / (2 * std::max(1ll, T)));
  if (V <= most) return round_up(V, 8);
  const long long pieces = (V + most - 1) / most;
  return round_up((V + pieces - 1) / pieces, 256);
}

// Pairs of a token that the forward kernel may leave: two per tile of at least 64
// words (16 in a vocabulary of up to 128).
long long most_parts(long long V) { return 2 * ((V + 63) / 64 + 8); }

constexpr long long kHead = 256;   // bytes of the backward workspace before p: the unit

template <bool PAIR, int BC>
cudaError_t opt_in() {
  const void* kernels[] = {reinterpret_cast<const void*>(bf16_grouped_kernel<PAIR, BC, kBfNT, kBfStats>),
                           reinterpret_cast<const void*>(bf16_grouped_kernel<PAIR, BC, kBfNT, kBfGrad>),
                           reinterpret_cast<const void*>(bf16_grouped_kernel<PAIR, BC, kBfNN, kBfSum>),
                           reinterpret_cast<const void*>(bf16_grouped_kernel<PAIR, BC, kBfTN, kBfSum>)};
  for (const void* k : kernels) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kBfMaxSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int FORM, int EPI>
cudaError_t launch_product(BfCall& c, const LossCall& a, int num_sms, cudaStream_t stream) {
  c.epilogue = static_cast<BfEpilogue>(EPI);
  BfPlan f = a.forced.lanes > 0 ? a.forced : bf_plan(c, num_sms);
  if (FORM == kBfNT) f.split = 1;
  c.loss.parts = 2 * ((c.rows + f.bc - 1) / f.bc);
  return f.pair       ? launch_tiles<true, 256, FORM, EPI>(c, a.encode, f, num_sms, stream)
         : f.bc <= 64 ? launch_tiles<false, 64, FORM, EPI>(c, a.encode, f, num_sms, stream)
                      : launch_tiles<false, 128, FORM, EPI>(c, a.encode, f, num_sms, stream);
}

BfCall product(const LossCall& a, BfForm form, const void* A, const void* B, void* D, int rows, int M,
               int N, int K) {
  BfCall c{};
  c.form = form;
  c.A = A;
  c.B = B;
  c.D = D;
  c.G = 1;
  c.rows = rows;
  c.M = M;
  c.N = N;
  c.K = K;
  c.status = a.status;
  c.timeout_ns = a.timeout_ns;
  c.debug_flags = a.debug_flags;
  c.limited = a.limited;
  return c;
}

// The pairs (largest, sum) of a token's parts into one: a block takes 32 tokens, a
// warp every eighth part.
constexpr int FIN_WARPS = 8;

struct LossEnd {
  const float2* part;   // [parts][T]
  const float* hit;     // [T]
  const int32_t* targets;
  float* loss;
  float* lse;
  int T, V, parts;
};

__device__ __forceinline__ void join(float& top, float& sum, float m, float s) {
  const float t = fmaxf(top, m);
  if (t == -INFINITY) return;
  sum = sum * exp2f(top - t) + s * exp2f(m - t);
  top = t;
}

__global__ void __launch_bounds__(32 * FIN_WARPS)
loss_end_kernel(const LossEnd a) {
  __shared__ float2 share[FIN_WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch_dependents();
  for (int t0 = blockIdx.x * 32; t0 < a.T; t0 += gridDim.x * 32) {
    const int t = t0 + lane;
    float top = -INFINITY, sum = 0.f;
    if (t < a.T) {
#pragma unroll 4
      for (int i = warp; i < a.parts; i += FIN_WARPS) {
        const float2 x = __ldg(a.part + static_cast<size_t>(i) * a.T + t);
        join(top, sum, x.x, x.y);
      }
    }
    share[warp][lane] = make_float2(top, sum);
    __syncthreads();
    if (warp == 0 && t < a.T) {
#pragma unroll
      for (int w = 1; w < FIN_WARPS; ++w) join(top, sum, share[w][lane].x, share[w][lane].y);
      constexpr float kLn2 = 0.6931471805599453f;
      const float lse = (top + log2f(sum)) * kLn2;
      const int y = __ldg(a.targets + t);
      if (a.lse) a.lse[t] = lse;
      if (a.loss) a.loss[t] = y >= 0 && y < a.V ? lse - __ldg(a.hit + t) : 0.f;
    }
    __syncthreads();
  }
}

// The unit: the largest |d_loss| of the tokens with a target (one block).
constexpr int UNIT_THREADS = 1024;

__global__ void __launch_bounds__(UNIT_THREADS)
loss_unit_kernel(const float* d_loss, const int32_t* targets, float* unit, int T, int V) {
  __shared__ float share[UNIT_THREADS / 32];
  grid_dep_wait();
  grid_dep_launch_dependents();
  float m = 0.f;
#pragma unroll 4
  for (int t = threadIdx.x; t < T; t += UNIT_THREADS) {
    const int y = __ldg(targets + t);
    if (y >= 0 && y < V) m = fmaxf(m, fabsf(__ldg(d_loss + t)));
  }
  // (not negative: in the order of their bits)
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  if ((threadIdx.x & 31) == 0) share[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x < 32) {
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(share[threadIdx.x])));
    if (threadIdx.x == 0) *unit = m;
  }
}

}  // namespace

long long loss_workspace(long long T, long long V) { return T * (8 * most_parts(V) + 4); }

long long loss_backward_workspace(long long T, long long V, long long K) {
  if (T == 0) return 0;
  const long long words = piece_words(T, V);
  return kHead + round_up(2 * T * words, 256) + (words < V ? 4 * T * K : 0);
}

cudaError_t loss_set_up() {
  cudaError_t e = opt_in<true, 256>();
  if (e == cudaSuccess) e = opt_in<false, 128>();
  if (e == cudaSuccess) e = opt_in<false, 64>();
  return e;
}

cudaError_t launch_loss(const LossCall& a, int num_sms, cudaStream_t stream) {
  BfCall c = product(a, kBfNT, a.W, a.X, nullptr, a.V, 0, a.T, a.K);
  c.loss.targets = a.targets;
  c.loss.words = a.V;
  c.loss.part = static_cast<float2*>(a.workspace);
  c.loss.hit = reinterpret_cast<float*>(c.loss.part + most_parts(a.V) * a.T);
  cudaError_t e = launch_product<kBfNT, kBfStats>(c, a, num_sms, stream);
  if (e != cudaSuccess) return e;
  const int blocks = (a.T + 31) / 32;
  return launch_dependent(loss_end_kernel, dim3(std::min(blocks, a.limited ? num_sms : 8 * num_sms)),
                          32 * FIN_WARPS, stream, 0,
                          LossEnd{c.loss.part, c.loss.hit, a.targets, a.loss, a.lse, a.T, a.V, c.loss.parts});
}

cudaError_t launch_loss_backward(const LossCall& a, int num_sms, cudaStream_t stream) {
  const int words = static_cast<int>(piece_words(a.T, a.V));
  float* unit = static_cast<float*>(a.workspace);
  uint8_t* p = static_cast<uint8_t*>(a.workspace) + kHead;
  float* sum = reinterpret_cast<float*>(p + round_up(2ll * a.T * words, 256));
  cudaError_t e = launch_dependent(loss_unit_kernel, dim3(1), UNIT_THREADS, stream, 0, a.d_loss, a.targets,
                                   unit, a.T, a.V);
  if (e != cudaSuccess) return e;
  for (long long w0 = 0; w0 < a.V; w0 += words) {
    const int n = static_cast<int>(std::min<long long>(words, a.V - w0));
    const uint8_t* W = static_cast<const uint8_t*>(a.W) + 2 * w0 * a.K;
    BfCall c = product(a, kBfNT, W, a.X, p, n, 0, a.T, a.K);
    c.loss.targets = a.targets;
    c.loss.words = a.V;
    c.loss.word0 = static_cast<int>(w0);
    c.loss.lse = a.lse;
    c.loss.d_loss = a.d_loss;
    c.loss.unit = unit;
    c.loss.pitch = words;
    e = launch_product<kBfNT, kBfGrad>(c, a, num_sms, stream);
    if (e == cudaSuccess && a.dW) {
      c = product(a, kBfTN, p, a.X, static_cast<uint8_t*>(a.dW) + 2 * w0 * a.K, a.T, n, a.K, 0);
      c.pitch = words;
      c.loss.unit = unit;
      c.loss.first = c.loss.last = true;
      e = launch_product<kBfTN, kBfSum>(c, a, num_sms, stream);
    }
    if (e == cudaSuccess && a.dX) {
      c = product(a, kBfNN, p, W, a.dX, a.T, 0, a.K, n);
      c.pitch = words;
      c.loss.sum = sum;
      c.loss.unit = unit;
      c.loss.first = w0 == 0;
      c.loss.last = a.V - w0 <= words;
      e = launch_product<kBfNN, kBfSum>(c, a, num_sms, stream);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dgk
