// Root-mean-square norm of x + residual with its output quantised 1x128 to
// e4m3 (the left operand of the FP8 GEMMs and its scales, as the quantiser
// writes them), and its gradient.  Per row m of K columns, in fp32:
//
//   h    = X[m] + R[m]                       (H = bf16(h): the residual stream)
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y    = h * rstd * W                      (Y = bf16(y))
//   Q, sa = 1x128 quantisation of y (not of Y: one rounding, to 8 bits)
//
// and with dY the gradient of y, xh = H * rstd, g = dY * W:
//
//   dX = rstd * (g - xh * mean(g * xh)) + dR,    dW[k] = sum_m dY[m,k] * xh[m,k]
//
// Both are memory-bound: a row is read once and stays on the chip between the
// statistics and the output.  A thread takes VPT vectors of 8 columns.  Two
// forms of each:
//  * one block per row, loads straight to registers (the gradient of few rows:
//    further blocks of the same launch sum the weight's gradient by columns);
//  * persistent blocks fed by bulk copies, several rows ahead, into a ring in
//    shared memory (the gradient: each keeps its share of the weight's in
//    registers, and a second kernel adds the shares).
// Under a limit on the SMs a grid has one block per SM, whose threads are teams that
// stand in for such blocks (132 of the 152 SMs: 4096 x 2048 forward 17.8 us, with all
// 13.4; backward 27.6 and 24.8).
// Measured: 4096 x 7168 forward 45 us (5.9 TB/s; one block per row 47 us), 3333 x
// 6656 without a residual 27 us; 8192 x 7168 backward 77 us (6.1 TB/s; the
// one-launch form 171 us), without dR 61 us (5.8 TB/s), 8192 x 4224 40 us.

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dg_fp8.cuh"
#include "dg_launch.h"
#include "dg_norm.h"
#include "dg_ring.cuh"

namespace dgk {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The threads that take a row together, whole warps: a block or, with FOLD, one of
// several teams of a block (under a limit on the SMs, where a grid has one block
// per SM).  tid: thread of the team, rank: the team among all in the grid.
constexpr int kMaxTeams = 15;   // of a block: a named barrier each, 1 .. 15
constexpr int kTeamsBytes = 6144;   // what their sums and barriers take from the rings at most

template <bool FOLD>
struct Team {
  int tid, size, id, rank;
  __device__ __forceinline__ explicit Team(int threads) {
    if constexpr (FOLD) {
      id = threadIdx.x / threads;
      tid = threadIdx.x - id * threads;
      size = threads;
      rank = id * gridDim.x + blockIdx.x;
    } else {
      id = 0;
      tid = threadIdx.x;
      size = blockDim.x;
      rank = blockIdx.x;
    }
  }
  __device__ __forceinline__ void sync() const {
    if constexpr (FOLD) named_bar_sync(1 + id, size);
    else __syncthreads();
  }
};

// Sum over the team of up to 32 warps; `red` is 32 floats that the previous
// call did not use (one barrier per call).
template <bool FOLD>
__device__ __forceinline__ float team_sum(const Team<FOLD>& t, float v, float* red) {
  v = warp_sum(v);
  if ((t.tid & 31) == 0) red[t.tid >> 5] = v;
  t.sync();
  const int warps = (t.size + 31) >> 5;
  v = (t.tid & 31) < warps ? red[t.tid & 31] : 0.f;
  return warp_sum(v);
}

// Checked build: vector `at` of a tensor [M][K].
template <class P>
__device__ __forceinline__ bool in_tensor(const P& a, size_t at) {
  return in_bounds(a, at, 1, static_cast<size_t>(a.M) * (a.K >> 3));
}

// Output of a normalised row: the thread's VPT vectors h (w: the weight's,
// packed), those below nv stored.
template <int VPT, bool UE8M0>
__device__ __forceinline__ void norm_output(const NormFwd& a, int m, int nv, int tid, int T,
                                            Pairs (&h)[VPT], float rs, const uint4 (&w)[VPT]) {
  const int kb = a.K >> 7;
  const size_t base = static_cast<size_t>(m) * (a.K >> 3);
  const float2 rs2 = make_float2(rs, rs);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * T + tid;
    const Pairs wp = bf16x8_to_pairs(w[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[i].v[j] = mul2(mul2(h[i].v[j], rs2), wp.v[j]);
    if (a.Y && v < nv && in_tensor(a, base + v))
      static_cast<uint4*>(a.Y)[base + v] = pairs_to_bf16x8(h[i]);
    if (!a.Q) continue;
    // a 128-column group is 16 consecutive lanes (T is a multiple of 32); its
    // even lanes compute 448 / a, which all take, its odd ones the scale a / 448
    float amax = pairs_amax(h[i]);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    amax = fminf(fmaxf(amax, kScaleFloor), kScaleTop);
    if constexpr (UE8M0) {
      float f;
      uint32_t e8;
      group_factor<true>(amax, f, e8);
      if (v < nv && in_tensor(a, base + v)) {
        static_cast<uint2*>(a.Q)[base + v] = pairs_to_e4m3x8(h[i], f);
        if ((v & 15) == 1 &&
            in_bounds(a, static_cast<size_t>(v >> 6) * a.ld_sa + m, 1, static_cast<size_t>((kb + 3) >> 2) * a.ld_sa))
          store_scale<true>(static_cast<float*>(a.sa), 0, kb, a.ld_sa, v >> 4, m, amax, e8);
      }
    } else {
      const bool odd = v & 1;
      const float quot = __fdiv_rn(odd ? amax : 448.0f, odd ? 448.0f : amax);
      const float f = __shfl_sync(0xffffffffu, quot, threadIdx.x & 30);
      if (v < nv && in_tensor(a, base + v)) {
        static_cast<uint2*>(a.Q)[base + v] = pairs_to_e4m3x8(h[i], f);
        const size_t at = static_cast<size_t>(v >> 4) * a.ld_sa + m;
        if ((v & 15) == 1 && in_bounds(a, at, 1, static_cast<size_t>(kb) * a.ld_sa))
          static_cast<float*>(a.sa)[at] = quot;
      }
    }
  }
}

template <int VPT>
__device__ __forceinline__ void load_weight(const void* W, int nv, int tid, int T, uint4 (&w)[VPT]) {
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * T + tid;
    w[i] = v < nv ? __ldg(static_cast<const uint4*>(W) + v) : make_uint4(0, 0, 0, 0);
  }
}

// h = x (+ r), its sum of squares, and the residual stream's output.
__device__ __forceinline__ float add_residual(const NormFwd& a, size_t at, const uint4& x,
                                              const uint4& r, Pairs& h) {
  h = bf16x8_to_pairs(x);
  if (a.R) {
    const Pairs rp = bf16x8_to_pairs(r);
#pragma unroll
    for (int j = 0; j < 4; ++j) h.v[j] = add2(h.v[j], rp.v[j]);
    if (a.H && in_tensor(a, at)) static_cast<uint4*>(a.H)[at] = pairs_to_bf16x8(h);
  }
  float2 ss = mul2(h.v[0], h.v[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) ss = fma2(h.v[j], h.v[j], ss);
  return ss.x + ss.y;
}

// One row by a team, loads straight to registers.
template <int VPT, bool UE8M0, bool FOLD>
__device__ __forceinline__ void norm_row(const NormFwd& a, const Team<FOLD>& t, int m, float* red) {
  const int T = t.size, nv = a.K >> 3;
  const uint4* X = static_cast<const uint4*>(a.X);
  const uint4* R = static_cast<const uint4*>(a.R);
  const size_t base = static_cast<size_t>(m) * nv;
  uint4 x[VPT], r[VPT], w[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * T + t.tid;
    x[i] = r[i] = make_uint4(0, 0, 0, 0);
    if (v < nv) {
      x[i] = ld_stream_v4(X + base + v);
      if (R) r[i] = ld_stream_v4(R + base + v);
    }
  }
  load_weight<VPT>(a.W, nv, t.tid, T, w);
  Pairs h[VPT] = {};
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * T + t.tid;
    if (v < nv) ss += add_residual(a, base + v, x[i], r[i], h[i]);
  }
  ss = team_sum(t, ss, red);
  const float rs = __frsqrt_rn(ss / static_cast<float>(a.K) + a.eps);
  if (t.tid == 0 && a.rstd && in_bounds(a, m, 1, a.M)) a.rstd[m] = rs;
  norm_output<VPT, UE8M0>(a, m, nv, t.tid, T, h, rs, w);
}

template <int VPT, bool UE8M0>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormFwd a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float red[32];
  const Team<false> t(0);
  norm_row<VPT, UE8M0>(a, t, t.rank, red);
}

// The same by teams of `threads` threads, which take row after row.
template <int VPT, bool UE8M0>
__global__ void __launch_bounds__(1024) rms_norm_teams_kernel(const NormFwd a, int threads) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float red[kMaxTeams][2][32];
  const Team<true> t(threads);
  const int step = gridDim.x * (blockDim.x / threads);
  int par = 0;
  for (long long m = t.rank; m < a.M; m += step, par ^= 1)
    norm_row<VPT, UE8M0>(a, t, static_cast<int>(m), red[t.id][par]);
}

template <int VPT, bool UE8M0>
__global__ void __launch_bounds__(1024) rms_norm_ring_kernel(const NormFwd a, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][32];
  __shared__ __align__(8) uint64_t full[kMaxRing];
  __shared__ uint32_t aborted, fills[kDebugRing];
  volatile uint32_t* abort_flag = &aborted;
  const int T = blockDim.x, nv = a.K >> 3, step = gridDim.x;
  ChunkRing ring{{a.X, a.R, nullptr}, smem, full, stages, a.R ? 2 : 1, a.K * 2,
                 {static_cast<size_t>(a.M) * a.K * 2, a.status, abort_flag, fills}, a.debug_flags, 0, 0};
  if (threadIdx.x == 0) ring.init(abort_flag);
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && blockIdx.x + static_cast<long long>(s) * step < a.M; ++s)
      ring.fill(blockIdx.x + s * step, s);
  const Team<false> t(0);
  uint4 w[VPT];
  load_weight<VPT>(a.W, nv, t.tid, T, w);
  __syncthreads();
  int s = 0, par = 0;
  uint32_t ph = 0;
  bool go = true;
  for (long long m = blockIdx.x; m < a.M; m += step, par ^= 1) {
    // (once a wait has failed a later turn of the ring may look complete)
    const bool ok = wait_bar(smem_u32(full + s), ph, abort_flag, a) && go &&
                    ring.holds(s, (m - blockIdx.x) / step / stages + 1);
    const size_t base = static_cast<size_t>(m) * nv;
    const uint4* x = reinterpret_cast<const uint4*>(ring.slot(s));
    Pairs h[VPT] = {};
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + threadIdx.x;
      if (v < nv && ok) ss += add_residual(a, base + v, x[v], a.R ? x[nv + v] : x[v], h[i]);
    }
    ss = team_sum(t, ss, red[par]);
    // every thread has read the slot: the row `stages` turns ahead may follow
    // (after a failed wait nothing more is loaded or stored)
    go = *abort_flag == 0;
    if (threadIdx.x == 0 && go && m + static_cast<long long>(stages) * step < a.M)
      ring.fill(static_cast<int>(m) + stages * step, s);
    const float rs = __frsqrt_rn(ss / static_cast<float>(a.K) + a.eps);
    if (threadIdx.x == 0 && a.rstd && go && in_bounds(a, m, 1, a.M)) a.rstd[m] = rs;
    norm_output<VPT, UE8M0>(a, static_cast<int>(m), go ? nv : 0, t.tid, T, h, rs, w);
    if (++s == stages) { s = 0; ph ^= 1; }
  }
  if (threadIdx.x == 0 && *abort_flag) ring.drain(a);
}

// Gradient, a vector of a row: its share of sum(g xh), the block's of dW.
__device__ __forceinline__ float grad_sums(const uint4& dy, const uint4& hv, const uint4& wv, float rs,
                                           Pairs& g, Pairs& xh, Pairs& dw) {
  const Pairs w = bf16x8_to_pairs(wv);
  const float2 rs2 = make_float2(rs, rs);
  g = bf16x8_to_pairs(dy);
  xh = bf16x8_to_pairs(hv);
  float2 dot = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    xh.v[j] = mul2(xh.v[j], rs2);
    dw.v[j] = fma2(g.v[j], xh.v[j], dw.v[j]);
    g.v[j] = mul2(g.v[j], w.v[j]);
    dot = fma2(g.v[j], xh.v[j], dot);
  }
  return dot.x + dot.y;
}

__device__ __forceinline__ uint4 grad_row(const Pairs& g, const Pairs& xh, float rs, float mean,
                                          const uint4& dr) {
  const float2 rs2 = make_float2(rs, rs), minus = make_float2(-mean, -mean);
  Pairs r = bf16x8_to_pairs(dr);
#pragma unroll
  for (int j = 0; j < 4; ++j) r.v[j] = fma2(rs2, fma2(xh.v[j], minus, g.v[j]), r.v[j]);
  return pairs_to_bf16x8(r);
}

// Few rows: blocks [0, M) take a row each, the blocks behind them 64 columns of
// dW each over all rows (which they read again, out of L2).
template <int VPT>
__global__ void __launch_bounds__(1024) rms_norm_backward_kernel(const NormBwd a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int T = blockDim.x, nv = a.K >> 3;
  const uint4* dY = static_cast<const uint4*>(a.dY);
  const uint4* H = static_cast<const uint4*>(a.H);
  const uint4* dR = static_cast<const uint4*>(a.dR);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (blockIdx.x < a.M) {
    __shared__ float red[32];
    const int m = blockIdx.x;
    const size_t base = static_cast<size_t>(m) * nv;
    const float rs = __ldg(a.rstd + m);
    uint4 w[VPT], dy[VPT], hv[VPT], r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + threadIdx.x;
      dy[i] = hv[i] = r[i] = zero;
      if (v < nv) {
        dy[i] = ld_stream_v4(dY + base + v);
        hv[i] = ld_stream_v4(H + base + v);
        if (dR) r[i] = ld_stream_v4(dR + base + v);
      }
    }
    const Team<false> t(0);
    load_weight<VPT>(a.W, nv, t.tid, T, w);
    Pairs g[VPT], xh[VPT], dw = {};
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) dot += grad_sums(dy[i], hv[i], w[i], rs, g[i], xh[i], dw);
    const float mean = team_sum(t, dot, red) * (1.0f / static_cast<float>(a.K));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + threadIdx.x;
      if (v < nv && in_tensor(a, base + v))
        static_cast<uint4*>(a.dX)[base + v] = grad_row(g[i], xh[i], rs, mean, r[i]);
    }
    return;
  }
  // 8 vectors of columns x T / 8 chains of rows
  extern __shared__ float part[];   // [T / 8][64]
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3, chains = T >> 3;
  const int v = (blockIdx.x - a.M) * 8 + c;
  float dw[8] = {};
#pragma unroll 4
  for (int m = r; m < a.M; m += chains) {
    const size_t at = static_cast<size_t>(m) * nv + v;
    const float rs = __ldg(a.rstd + m);
    float g[8], h[8];
    bf16x8_to_float(__ldg(dY + at), g);
    bf16x8_to_float(__ldg(H + at), h);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = fmaf(g[j], h[j] * rs, dw[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[r * 64 + c * 8 + j] = dw[j];
  __syncthreads();
  for (int k = threadIdx.x; k < 64; k += T) {
    float sum = 0.f;
    for (int i = 0; i < chains; ++i) sum += part[i * 64 + k];
    const int at = (blockIdx.x - a.M) * 64 + k;
    if (in_bounds(a, at, 1, a.K)) a.dW[at] = sum;
  }
}

// Rows by `teams` teams (FOLD; else a block each), with a ring each.
template <int VPT, bool FOLD>
__global__ void __launch_bounds__(1024)
rms_norm_backward_ring_kernel(const NormBwd a, int threads, int teams, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int TEAMS = FOLD ? kMaxTeams : 1;
  __shared__ float reds[TEAMS][2][32];
  __shared__ __align__(8) uint64_t fulls[TEAMS][kMaxRing];
  __shared__ uint32_t aborts[TEAMS], fills[TEAMS][kDebugRing];
  const Team<FOLD> t(threads);
  float(*red)[32] = reds[t.id];
  uint64_t* full = fulls[t.id];
  volatile uint32_t* abort_flag = &aborts[t.id];
  const int T = t.size, nv = a.K >> 3, step = FOLD ? teams : static_cast<int>(gridDim.x);
  const int ops = a.dR ? 3 : 2, bytes = a.K * 2;
  ChunkRing ring{{a.dY, a.H, a.dR}, smem + t.id * stages * ops * bytes, full, stages, ops, bytes,
                 {static_cast<size_t>(a.M) * bytes, a.status, abort_flag, fills[t.id]}, a.debug_flags, 0,
                 0};
  if (t.tid == 0) ring.init(abort_flag);
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (FOLD && t.rank >= teams) return;   // (the last block's; from here on a team is by itself)
  if (t.tid == 0)
    for (int s = 0; s < stages && t.rank + static_cast<long long>(s) * step < a.M; ++s)
      ring.fill(t.rank + s * step, s);
  uint4 w[VPT];
  load_weight<VPT>(a.W, nv, t.tid, T, w);
  t.sync();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // With one vector a thread keeps what it has read of a row for the output; with
  // two (which 64 registers do not hold) it reads the slot again, which then is
  // free a row later.
  constexpr bool KEEP = VPT == 1;
  const int ahead = (KEEP ? stages : stages - 1) * step;
  Pairs dw[VPT] = {};
  int s = 0, par = 0;
  uint32_t ph = 0;
  for (long long m = t.rank; m < a.M; m += step, par ^= 1) {
    const float rs = __ldg(a.rstd + m);
    const bool ok = wait_bar(smem_u32(full + s), ph, abort_flag, a) &&
                    ring.holds(s, (m - t.rank) / step / stages + 1);
    const size_t base = static_cast<size_t>(m) * nv;
    const uint4* x = reinterpret_cast<const uint4*>(ring.slot(s));
    Pairs g[VPT], xh[VPT];
    float dot = 0.f;
    uint4 r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + t.tid;
      const bool on = v < nv && ok;
      if (KEEP) r[i] = on && a.dR ? x[2 * nv + v] : zero;
      dot += grad_sums(on ? x[v] : zero, on ? x[nv + v] : zero, w[i], rs, g[i], xh[i], dw[i]);
    }
    const float mean = team_sum(t, dot, red[par]) * (1.0f / static_cast<float>(a.K));
    // every thread has read the slot (two vectors: the one before) for the last
    // time; after a failed wait nothing more is loaded or stored
    const bool go = *abort_flag == 0;
    if (t.tid == 0 && go && (KEEP || m != t.rank) && m + ahead < a.M)
      ring.fill(static_cast<int>(m) + ahead, KEEP ? s : (s == 0 ? stages : s) - 1);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + t.tid;
      if (v >= nv || !go || !in_tensor(a, base + v)) continue;
      if (!KEEP) {
        Pairs unused = {};
        grad_sums(x[v], x[nv + v], w[i], rs, g[i], xh[i], unused);
        r[i] = a.dR ? x[2 * nv + v] : zero;
      }
      static_cast<uint4*>(a.dX)[base + v] = grad_row(g[i], xh[i], rs, mean, r[i]);
    }
    if (++s == stages) { s = 0; ph ^= 1; }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * T + t.tid;
    const size_t at = static_cast<size_t>(t.rank) * a.K + 8 * v;
    if (v >= nv || !in_bounds(a, at, 8, static_cast<size_t>(min(a.M, kNormBwdBlocks)) * a.K)) continue;
    float4* out = reinterpret_cast<float4*>(a.part + at);
    out[0] = make_float4(dw[i].v[0].x, dw[i].v[0].y, dw[i].v[1].x, dw[i].v[1].y);
    out[1] = make_float4(dw[i].v[2].x, dw[i].v[2].y, dw[i].v[3].x, dw[i].v[3].y);
  }
  if (t.tid == 0 && *abort_flag) ring.drain(a);
}

struct StatusWord {
  unsigned int* status;
};

// dW[k] = sum of the blocks' (teams') partial sums, in a fixed order: 32 columns
// per block (WALK: at a time), 32 chains over the partials.
template <bool WALK>
__global__ void __launch_bounds__(1024)
rms_norm_weight_grad_kernel(const float* __restrict__ part, float* __restrict__ dW, int blocks,
                            int K, const StatusWord word) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  auto sum_up = [&](int k0) {
    const int k = k0 + c;
    float acc = 0.f;
    for (int b = r; b < blocks; b += 32) acc += part[static_cast<size_t>(b) * K + k];
    s[r][c] = acc;
    __syncthreads();
    // (transposed: warp r now sums the chains of column r)
    const float sum = warp_sum(s[c][r]);
    if (c == 0 && in_bounds(word, k0 + r, 1, K)) dW[k0 + r] = sum;
  };
  if constexpr (WALK) {
    for (int k0 = blockIdx.x * 32; k0 < K; k0 += gridDim.x * 32) {
      sum_up(k0);
      __syncthreads();   // the chains have been read
    }
  } else {
    sum_up(blockIdx.x * 32);
  }
}

// Threads of a block whose rows of K columns take `vpt` vectors per thread.
int row_threads(int K, int vpt) { return ((K / 8 + vpt - 1) / vpt + 31) / 32 * 32; }

// threads: of a team (a block, or with `teams` > 0 one of that many over the blocks)
struct RingShape {
  int blocks, threads, stages, smem, teams, per_block;
};

// A ring per block, as many blocks per SM as a thousand threads make (their
// rings share the SM's memory), at least three slots each.
RingShape ring_shape(int M, int K, int ops, int vpt, int num_sms, int max_blocks) {
  RingShape r;
  r.threads = row_threads(K, vpt);
  const int slot = 2 * K * ops;
  const int per_sm = std::max(1, std::min(1024 / r.threads, ring_bytes(1) / (3 * slot)));
  // (two slots of the longest rows fit; the gradient's two-vector form needs them)
  r.stages = std::max(2, std::min(kMaxRing, ring_bytes(per_sm) / slot));
  r.blocks = std::min(std::min(M, per_sm * num_sms), max_blocks);
  r.smem = r.stages * slot;
  r.teams = 0;
  r.per_block = 1;
  return r;
}

// The same folded into one block per SM: teams in place of the blocks that share
// an SM.
RingShape ring_fold(int M, int K, int ops, int vpt, int num_sms, int max_teams) {
  RingShape r;
  r.threads = row_threads(K, vpt);
  const int slot = 2 * K * ops, room = ring_bytes(1) - kTeamsBytes;
  const int most = std::max(1, std::min(std::min(kMaxTeams, 1024 / r.threads), room / (3 * slot)));
  r.teams = std::min(std::min(M, most * num_sms), max_teams);
  r.blocks = std::min(r.teams, num_sms);
  r.per_block = (r.teams + r.blocks - 1) / r.blocks;
  r.stages = std::max(2, std::min(kMaxRing, room / r.per_block / slot));
  r.smem = r.per_block * r.stages * slot;
  return r;
}

template <class... P, class... A>
cudaError_t launch_ring(void (*kernel)(P...), const RingShape& r, cudaStream_t stream, A... args) {
  return launch_dependent(kernel, dim3(r.blocks), r.threads, stream, r.smem, args..., r.stages);
}

template <bool UE8M0>
cudaError_t launch_fwd(const NormFwd& a, int num_sms, bool limited, cudaStream_t stream) {
  const int vpt = a.K <= 8192 ? 1 : 2;
  // Long rows leave room for one or two blocks per SM, which wait for their
  // loads in turn: the ring is ahead from some 12 rows per SM (2432 x 7168: 27.7
  // against 29.7 us).  Shorter rows, with more blocks per SM, need none (4864 x
  // 4096: 32.2 with it, 29.6 without; 2432 x 1024: 4.8, 3.9).
  if (a.K > 6144 && a.M >= 12 * num_sms) {
    const RingShape r = ring_shape(a.M, a.K, a.R ? 2 : 1, vpt, num_sms, a.M);
    return vpt == 1 ? launch_ring(rms_norm_ring_kernel<1, UE8M0>, r, stream, a)
                    : launch_ring(rms_norm_ring_kernel<2, UE8M0>, r, stream, a);
  }
  const int threads = row_threads(a.K, vpt);
  if (limited && a.M > num_sms) {
    const int teams = std::min(kMaxTeams, 1024 / threads);
    const dim3 grid(std::min(num_sms, a.M));
    return vpt == 1 ? launch_dependent(rms_norm_teams_kernel<1, UE8M0>, grid, teams * threads, stream, 0, a,
                                       threads)
                    : launch_dependent(rms_norm_teams_kernel<2, UE8M0>, grid, teams * threads, stream, 0, a,
                                       threads);
  }
  return vpt == 1 ? launch_dependent(rms_norm_kernel<1, UE8M0>, dim3(a.M), threads, stream, 0, a)
                  : launch_dependent(rms_norm_kernel<2, UE8M0>, dim3(a.M), threads, stream, 0, a);
}

}  // namespace

cudaError_t norm_set_up() {
  const void* kernels[] = {reinterpret_cast<const void*>(rms_norm_ring_kernel<1, false>),
                           reinterpret_cast<const void*>(rms_norm_ring_kernel<2, false>),
                           reinterpret_cast<const void*>(rms_norm_ring_kernel<1, true>),
                           reinterpret_cast<const void*>(rms_norm_ring_kernel<2, true>),
                           reinterpret_cast<const void*>(rms_norm_backward_ring_kernel<1, false>),
                           reinterpret_cast<const void*>(rms_norm_backward_ring_kernel<2, false>)};
  const void* teams[] = {reinterpret_cast<const void*>(rms_norm_backward_ring_kernel<1, true>),
                         reinterpret_cast<const void*>(rms_norm_backward_ring_kernel<2, true>)};
  auto opt_in = [](const void* k, int bytes) {
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  cudaError_t e = cudaSuccess;
  for (const void* k : kernels)
    if (e == cudaSuccess) e = opt_in(k, ring_bytes(1));
  for (const void* k : teams)
    if (e == cudaSuccess) e = opt_in(k, ring_bytes(1) - kTeamsBytes);
  return e;
}

cudaError_t launch_rms_norm(const NormFwd& a, bool ue8m0, int num_sms, bool limited,
                            cudaStream_t stream) {
  return ue8m0 ? launch_fwd<true>(a, num_sms, limited, stream)
               : launch_fwd<false>(a, num_sms, limited, stream);
}

cudaError_t launch_rms_norm_backward(const NormBwd& a, int num_sms, bool limited,
                                     cudaStream_t stream) {
  const int vpt = a.K <= 8192 ? 1 : 2;
  // The one-launch form reads its rows a second time, in chains that grow with
  // M; the ring pays a second kernel (about 1.5 us).  Measured with both, 456
  // rows of 512, 2048, 7168 columns: 5.0, 5.5, 9.3 us in one launch, 5.0, 6.7,
  // 8.8 us with the ring; 608 rows: 6.0, 7.2, 11.9 and 5.4, 7.1, 10.1 us.
  if (limited ? a.M + a.K / 64 <= num_sms : a.M <= 3 * num_sms) {
    // (at least 32 chains of rows in a block of dW's columns)
    const int threads = std::max(256, row_threads(a.K, vpt));
    const dim3 grid(a.M + a.K / 64);
    const int smem = threads / 8 * 64 * 4;
    return vpt == 1 ? launch_dependent(rms_norm_backward_kernel<1>, grid, threads, stream, smem, a)
                    : launch_dependent(rms_norm_backward_kernel<2>, grid, threads, stream, smem, a);
  }
  // Two vectors a thread also where that makes two blocks per SM, each with three
  // slots, of rows that otherwise take one alone, whose barriers then leave the SM
  // idle (8192 rows: K = 4224 57 to 40 us, 7168 without dR 71 to 61; with dR, two
  // slots each, 77 to 78); not worth a longer start for a few rows (614 rows, K =
  // 5120: 8.7 to 10.7, 1254 rows 16.4 to 15.5).
  const int ops = a.dR ? 3 : 2;
  const bool split = a.K > 4096 && a.K <= 8192 && a.M > 6 * num_sms &&
                     ring_bytes(2) >= 3 * 2 * a.K * ops;
  const int per_thread = split ? 2 : vpt;
  auto launch = [&](auto kernel, const RingShape& r) {
    return launch_dependent(kernel, dim3(r.blocks), r.per_block * r.threads, stream, r.smem, a, r.threads,
                            r.teams, r.stages);
  };
  auto add_up = [&](auto kernel, int parts, int blocks) {
    return launch_dependent(kernel, dim3(blocks), 1024, stream, 0, static_cast<const float*>(a.part), a.dW,
                            parts, a.K, StatusWord{a.status});
  };
  if (limited) {
    const int sums = std::min(num_sms, a.K / 32);
    if (a.M == 0) return add_up(rms_norm_weight_grad_kernel<true>, 0, sums);
    const RingShape r = ring_fold(a.M, a.K, ops, per_thread, num_sms, kNormBwdBlocks);
    const cudaError_t e = per_thread == 1 ? launch(rms_norm_backward_ring_kernel<1, true>, r)
                                          : launch(rms_norm_backward_ring_kernel<2, true>, r);
    return e != cudaSuccess ? e : add_up(rms_norm_weight_grad_kernel<true>, r.teams, sums);
  }
  const RingShape r = ring_shape(a.M, a.K, ops, per_thread, num_sms, kNormBwdBlocks);
  const cudaError_t e = per_thread == 1 ? launch(rms_norm_backward_ring_kernel<1, false>, r)
                                        : launch(rms_norm_backward_ring_kernel<2, false>, r);
  return e != cudaSuccess ? e : add_up(rms_norm_weight_grad_kernel<false>, r.blocks, a.K / 32);
}

}  // namespace dgk
