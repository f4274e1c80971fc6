// Softmax cross entropy of the product z = X W^T over a vocabulary of V words, in
// pieces that stay on the chip, and its gradient.  Per token t, with y its target:
//
//   lse = log sum_v exp(z_v);   loss = lse - z_y        (0 without a target)
//   p_v = (exp(z_v - lse) - [v = y]) d_loss             (0 without a target)
//   dX = p W,   dW = p^T X
//
// Forward: the bf16 product's kernel (dg_bf16_kernel.cuh, form nt) with W's rows on
// the accumulator's columns and tokens on its lanes (of few tokens the other way
// round).  A lane then has 256 logits of one token, and leaves the largest of them and
// the sum of the exponentials relative to it; a second kernel joins the tiles' pairs.
// The logits never leave the SM.
//
// Backward: per piece of the vocabulary the logits again, whose epilogue writes p in
// bf16 (as every operand of these products; one rounding, by 2^-8 of itself at most; a
// component that W's rows share is multiplied by what a token's roundings come to, as p itself
// sums to 0),
// then the piece's rows of dW (form tn) and its share of dX (form nn), which is added
// up in fp32 over the pieces and rounded once with the last.  p is written relative
// to the largest |d_loss|, the unit, and the products' sums are multiplied by it: with
// the same d_loss for all tokens, as in a mean, its rounding then is none of p's, and
// the -1 at the targets, the largest entries of all, stay near -1 (with d_loss in p,
// 1 / T rounded to bf16 in every token's largest entry: dX and dW off by up to 0.0037
// of themselves, so 0.0017, which is their own rounding).  A piece is as wide as makes
// p 384 MB at most: fewer sums of dX in fp32 and fewer last waves of tiles than with
// pieces that stay in L2 (4095 tokens of 50003 x 4096, pieces of 24 / 96 / 384 MB: 3370 /
// 3070 / 2950 us; 4096 of 131072 x 2048: 4640 / 4065 / 3850; 8192 of 32000 x 2048: 2140 /
// 2110 / 1950; 2048 of 50003 x 7168: 2860 / 2578 / 2602).
//
// Bounded by the tensor cores; with few tokens by reading W (and writing dW).
#include <algorithm>

#include "dg_bf16_kernel.cuh"
#include "dg_launch.h"
#include "dg_loss.h"

namespace dgk {
namespace {

constexpr long long kPieceBytes = 384ll << 20;  // of p
constexpr int kPieceLeast = 4096;               // words: whole waves of tiles
// and at most: dX's sum over a piece drops up to half of 2^-23 of itself at each 16 words (of
// 4e8 words in two pieces it was off by 0.06 of itself)
constexpr int kPieceMost = 1 << 20;

long long round_up(long long x, long long to) { return (x + to - 1) / to * to; }

// Words of a piece, a multiple of 8 (of 256 where there are more pieces).
long long piece_words(long long T, long long V) {
  const long long most = std::clamp<long long>(kPieceBytes / (2 * std::max(1ll, T)), kPieceLeast, kPieceMost);
  if (V <= most) return round_up(V, 8);
  const long long pieces = (V + most - 1) / most;
  return round_up((V + pieces - 1) / pieces, 256);
}

// Up to how many tokens the words are on the accumulator's lanes.  A tile then is up to
// 256 words by as many tokens as there are, and the time that of reading W once (forward, 7
// tokens of 50003 x 4096: 70 us so, 97 with tokens on the lanes, 1 of 8000 x 1000: 11 and 16, 61 of
// 32000 x 2048: 29.4 and 31.9); with more tokens the exchange between the lanes costs more
// (65 of 32000 x 2048: 33.6 and 31.9, 128: 34.6 and 32.1, 300 of 20000 x 1024: 27.7 and 23.9,
// 4096 of 131072 x 2048, a dozen calls by themselves, before the power cap lowers the clock:
// 1409 and 1100).
constexpr int kWordsOnLanes = 64;

// Pairs of a token that the forward kernel may leave: with words on the lanes four per
// 64 of them or more, else two per tile of at least 64 words (16 in a vocabulary of up
// to 128).
long long most_pairs(long long T, long long V) {
  return (T <= kWordsOnLanes ? 4 : 2) * ((V + 63) / 64 + 8);
}

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

// Parts of dX's reduction over the vocabulary, where the tiles of a few tokens leave
// SMs without work (61 tokens of 32000 x 2048: 8 tiles, 38 us as clusters of 8 CTAs that
// share a reduction, 29 so); a part at least 1024 words.
constexpr int kPartDepth = 1024, kPartMost = 64;

long long most_reduction_parts(long long T, long long V, long long K) {
  // (for any number of SMs up to 256, and tiles of at most 256 x 256)
  const long long tiles = ((T + 255) / 256) * ((K + 255) / 256);
  return std::max<long long>(1, std::min<long long>({256 / std::max(1ll, tiles), V / kPartDepth, kPartMost}));
}

// Sets c.loss.parts and depth for dX of one piece.
void reduction_parts(BfCall& c, const LossCall& a, int num_sms) {
  if (a.forced.lanes > 0 && a.forced.split > 1) return;
  const long long tiles = static_cast<long long>((a.T + 127) / 128) * ((a.K + 255) / 256);
  const long long parts = std::min(most_reduction_parts(a.T, a.V, a.K), num_sms / std::max(1ll, tiles));
  if (parts < 2) return;
  c.loss.depth = static_cast<int>(round_up((c.K + parts - 1) / parts, 128));
  c.loss.parts = (c.K + c.loss.depth - 1) / c.loss.depth;
  c.loss.last = c.loss.parts < 2;
}

template <int FORM, int EPI>
cudaError_t launch_product(BfCall& c, const LossCall& a, int num_sms, cudaStream_t stream) {
  c.epilogue = static_cast<BfEpilogue>(EPI);
  BfPlan f = a.forced.lanes > 0 ? a.forced : bf_plan(c, num_sms);
  if (FORM == kBfNT) f.split = 1;
  else f.lanes = static_cast<int>(round_up(f.lanes, 64));   // (W's and X's boxes; of a forced plan)
  if (FORM == kBfTN && f.pair) f.bc = 256;   // (whole 128-wide halves)
  if (EPI == kBfSum) c.loss.parts = std::max(1, c.loss.parts);
  if (EPI == kBfStats)   // (of the words, for the joining kernel)
    c.loss.pairs = c.loss.words_on_lanes ? 4 * (f.pair ? 2 : 1) * ((c.N + f.lanes - 1) / f.lanes)
                                         : 2 * ((c.rows + f.bc - 1) / f.bc);
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

// The product whose sums are the logits of n words from w0 on.
BfCall logits(const LossCall& a, int w0, int n) {
  const void* W = static_cast<const uint8_t*>(a.W) + 2ll * w0 * a.K;
  const bool lanes = a.T <= kWordsOnLanes;
  BfCall c = lanes ? product(a, kBfNT, a.X, W, nullptr, a.T, 0, n, a.K)
                   : product(a, kBfNT, W, a.X, nullptr, n, 0, a.T, a.K);
  c.loss.words_on_lanes = lanes;
  c.loss.targets = a.targets;
  c.loss.words = a.V;
  c.loss.word0 = w0;
  c.loss.tokens = a.T;
  return c;
}

// The pairs (largest, sum) of a token's parts into one: a block takes four tokens (a
// sector of each part), its threads the parts, eight asked for at a time.  (A lane per
// token, a warp every 32nd part, joined one by one: 9 us for 61 tokens of 250 parts.)
constexpr int END_THREADS = 512, END_TOKENS = 4, END_SLICES = END_THREADS / END_TOKENS;

struct LossEnd {
  const float2* pair;   // [pairs][T]
  const float* hit;     // [T]
  const int32_t* targets;
  float* loss;
  float* lse;
  int T, V, pairs;
  unsigned int* status;
};

__device__ __forceinline__ void join(float& top, float& sum, float m, float s) {
  const float t = fmaxf(top, m);
  if (t == -INFINITY) return;
  sum = sum * exp2f(top - t) + s * exp2f(m - t);
  top = t;
}

__global__ void __launch_bounds__(END_THREADS)
loss_end_kernel(const LossEnd a) {
  constexpr int N = 8;
  __shared__ float2 share[END_THREADS / 32][END_TOKENS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = threadIdx.x % END_TOKENS, slice = threadIdx.x / END_TOKENS;
  grid_dep_wait();
  grid_dep_launch_dependents();
  for (long long t0 = static_cast<long long>(blockIdx.x) * END_TOKENS; t0 < a.T;
       t0 += static_cast<long long>(gridDim.x) * END_TOKENS) {
    const long long t = t0 + j;
    float top = -INFINITY, sum = 0.f;
    if (t < a.T) {
      for (int i = slice; i < a.pairs; i += N * END_SLICES) {
        float2 x[N];
#pragma unroll
        for (int n = 0; n < N; ++n)
          x[n] = i + n * END_SLICES < a.pairs
                     ? __ldg(a.pair + static_cast<size_t>(i + n * END_SLICES) * a.T + t)
                     : make_float2(-INFINITY, 0.f);
        float m = x[0].x, s = 0.f;
#pragma unroll
        for (int n = 1; n < N; ++n) m = fmaxf(m, x[n].x);
        if (m == -INFINITY) continue;
#pragma unroll
        for (int n = 0; n < N; ++n) s += x[n].y * exp2f(x[n].x - m);
        join(top, sum, m, s);
      }
    }
#pragma unroll
    for (int o = 16; o >= END_TOKENS; o >>= 1)
      join(top, sum, __shfl_xor_sync(0xffffffffu, top, o), __shfl_xor_sync(0xffffffffu, sum, o));
    if (lane < END_TOKENS) share[warp][lane] = make_float2(top, sum);
    __syncthreads();
    if (threadIdx.x < END_TOKENS && t < a.T && in_bounds(a, t, 1, a.T)) {
#pragma unroll
      for (int w = 1; w < END_THREADS / 32; ++w) join(top, sum, share[w][lane].x, share[w][lane].y);
      constexpr float kLn2 = 0.6931471805599453f;
      const float rest = log2f(sum);
      const int y = __ldg(a.targets + t);
      if (a.lse) a.lse[t] = (top + rest) * kLn2;
      if (a.loss) {
        // Not as lse less the target's logit, which may be hundreds and their difference 1e-3 or,
        // rounded, negative: `top` is a logit times log2(e), rounded, and `rest` counts for what
        // that is off by.
        float loss = 0.f;
        if (y >= 0 && y < a.V) {
          loss = (fmaf(-__ldg(a.hit + t), kLog2e, top) + rest) * kLn2;
          loss = loss < 0.f ? 0.f : loss;
        }
        a.loss[t] = loss;
      }
    }
    __syncthreads();
  }
}

// dX from the sums of the parts of its reduction, in their order.
struct LossJoin {
  const float* sum;   // [parts][elements]
  const float* unit;
  void* dX;           // bf16 [elements]
  long long elements; // a multiple of 8
  int parts;
  unsigned int* status;
};

constexpr int JOIN_THREADS = 256;

__global__ void __launch_bounds__(JOIN_THREADS)
loss_join_kernel(const LossJoin a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const float u = *a.unit;
  const long long step = static_cast<long long>(gridDim.x) * JOIN_THREADS * 4;
  for (long long i = (static_cast<long long>(blockIdx.x) * JOIN_THREADS + threadIdx.x) * 4; i < a.elements; i += step) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int j = 0; j < a.parts; ++j) {
      const float4 x = *reinterpret_cast<const float4*>(a.sum + j * a.elements + i);
      s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    if (!in_bounds(a, i, 4, a.elements)) continue;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dX) + i) =
        make_uint2(pack_bf16x2(u * s.x, u * s.y), pack_bf16x2(u * s.z, u * s.w));
  }
}

}  // namespace

bool loss_words_on_lanes(long long T) { return T <= kWordsOnLanes; }

long long loss_workspace(long long T, long long V) { return T * (8 * most_pairs(T, V) + 4); }

long long loss_backward_workspace(long long T, long long V, long long K) {
  if (T == 0) return 0;
  const long long words = piece_words(T, V);
  const long long parts = most_reduction_parts(T, V, K);
  return kHead + round_up(2 * T * words, 256) + 4 * T * K * (words < V ? 1 : parts > 1 ? parts : 0);
}

cudaError_t loss_set_up() {
  cudaError_t e = opt_in<true, 256>();
  if (e == cudaSuccess) e = opt_in<false, 128>();
  if (e == cudaSuccess) e = opt_in<false, 64>();
  return e;
}

cudaError_t launch_loss(const LossCall& a, int num_sms, cudaStream_t stream) {
  BfCall c = logits(a, 0, a.V);
  c.loss.pair = static_cast<float2*>(a.workspace);
  c.loss.hit = reinterpret_cast<float*>(c.loss.pair + most_pairs(a.T, a.V) * a.T);
  cudaError_t e = launch_product<kBfNT, kBfStats>(c, a, num_sms, stream);
  if (e != cudaSuccess) return e;
  const int blocks = (a.T + END_TOKENS - 1) / END_TOKENS;
  return launch_dependent(loss_end_kernel, dim3(std::min(blocks, a.limited ? num_sms : 4 * num_sms)),
                          END_THREADS, stream, 0,
                          LossEnd{c.loss.pair, c.loss.hit, a.targets, a.loss, a.lse, a.T, a.V, c.loss.pairs,
                                  a.status});
}

cudaError_t launch_loss_backward(const LossCall& a, int num_sms, cudaStream_t stream) {
  const int words = static_cast<int>(piece_words(a.T, a.V));
  float* unit = static_cast<float*>(a.workspace);
  uint8_t* p = static_cast<uint8_t*>(a.workspace) + kHead;
  float* sum = reinterpret_cast<float*>(p + round_up(2ll * a.T * words, 256));
  for (long long w0 = 0; w0 < a.V; w0 += words) {
    const int n = static_cast<int>(std::min<long long>(words, a.V - w0));
    const uint8_t* W = static_cast<const uint8_t*>(a.W) + 2 * w0 * a.K;
    BfCall c = logits(a, static_cast<int>(w0), n);
    c.D = p;
    c.loss.lse = a.lse;
    c.loss.d_loss = a.d_loss;
    c.loss.unit = unit;
    c.loss.first = w0 == 0;
    c.loss.pitch = words;
    cudaError_t e = launch_product<kBfNT, kBfGrad>(c, a, num_sms, stream);
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
      const bool whole = c.loss.first && c.loss.last;
      if (whole) reduction_parts(c, a, num_sms);
      e = launch_product<kBfNN, kBfSum>(c, a, num_sms, stream);
      if (e == cudaSuccess && c.loss.parts > 1) {
        const long long n = static_cast<long long>(a.T) * a.K;
        const long long blocks = (n / 4 + JOIN_THREADS - 1) / JOIN_THREADS;
        e = launch_dependent(
            loss_join_kernel,
            dim3(static_cast<unsigned>(std::min<long long>(blocks, a.limited ? num_sms : 8 * num_sms))),
            JOIN_THREADS, stream, 0, LossJoin{sum, unit, a.dX, n, c.loss.parts, a.status});
      }
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dgk
