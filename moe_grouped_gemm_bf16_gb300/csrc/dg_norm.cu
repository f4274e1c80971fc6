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
//  * one block per row, loads straight to registers: the shortest latency, for
//    few rows;
//  * persistent blocks fed by bulk copies, several rows ahead, into a ring in
//    shared memory: a block that waits for its row's loads, reduces, and only
//    then stores keeps too few bytes in flight (4096 x 7168: 56 us at two
//    blocks per SM).
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

// Sum over the block of up to 32 warps; `red` is 32 floats that the previous
// call did not use (one barrier per call).
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = (blockDim.x + 31) >> 5;
  v = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
  return warp_sum(v);
}

// Output of a normalised row: the thread's VPT vectors h (w: the weight's,
// packed), those below nv stored.
template <int VPT, bool UE8M0>
__device__ __forceinline__ void norm_output(const NormFwd& a, int m, int nv, float (&h)[VPT][8],
                                            float rs, const uint4 (&w)[VPT]) {
  const int T = blockDim.x, kb = a.K >> 7;
  const size_t base = static_cast<size_t>(m) * (a.K >> 3);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * T + threadIdx.x;
    float wf[8];
    bf16x8_to_float(w[i], wf);
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[i][j] = h[i][j] * rs * wf[j];
      amax = fmaxf(amax, fabsf(h[i][j]));
    }
    if (a.Y && v < nv) static_cast<uint4*>(a.Y)[base + v] = float_to_bf16x8(h[i]);
    if (!a.Q) continue;
    // a 128-column group is 16 consecutive lanes (T is a multiple of 32)
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    amax = fmaxf(amax, kScaleFloor);
    float f;
    uint32_t e8;
    group_factor<UE8M0>(amax, f, e8);
    if (v < nv) {
      uint2 q;
      q.x = cvt_e4m3x4(h[i][0] * f, h[i][1] * f, h[i][2] * f, h[i][3] * f);
      q.y = cvt_e4m3x4(h[i][4] * f, h[i][5] * f, h[i][6] * f, h[i][7] * f);
      static_cast<uint2*>(a.Q)[base + v] = q;
      if ((v & 15) == 0)
        store_scale<UE8M0>(static_cast<float*>(a.sa), 0, kb, a.ld_sa, v >> 4, m, amax, e8);
    }
  }
}

template <int VPT>
__device__ __forceinline__ void load_weight(const void* W, int nv, uint4 (&w)[VPT]) {
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * blockDim.x + threadIdx.x;
    w[i] = v < nv ? __ldg(static_cast<const uint4*>(W) + v) : make_uint4(0, 0, 0, 0);
  }
}

// h = x (+ r), its sum of squares, and the residual stream's output.
__device__ __forceinline__ float add_residual(const NormFwd& a, size_t at, const uint4& x,
                                              const uint4& r, float (&h)[8]) {
  bf16x8_to_float(x, h);
  if (a.R) {
    float rf[8];
    bf16x8_to_float(r, rf);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] += rf[j];
    if (a.H) static_cast<uint4*>(a.H)[at] = float_to_bf16x8(h);
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) ss = fmaf(h[j], h[j], ss);
  return ss;
}

template <int VPT, bool UE8M0>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormFwd a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float red[32];
  const int T = blockDim.x, nv = a.K >> 3, m = blockIdx.x;
  const uint4* X = static_cast<const uint4*>(a.X);
  const uint4* R = static_cast<const uint4*>(a.R);
  const size_t base = static_cast<size_t>(m) * nv;
  uint4 x[VPT], r[VPT], w[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * T + threadIdx.x;
    x[i] = r[i] = make_uint4(0, 0, 0, 0);
    if (v < nv) {
      x[i] = ld_stream_v4(X + base + v);
      if (R) r[i] = ld_stream_v4(R + base + v);
    }
  }
  load_weight<VPT>(a.W, nv, w);
  float h[VPT][8], ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * T + threadIdx.x;
    if (v < nv) {
      ss += add_residual(a, base + v, x[i], r[i], h[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
    }
  }
  ss = block_sum(ss, red);
  const float rs = __frsqrt_rn(ss / static_cast<float>(a.K) + a.eps);
  if (threadIdx.x == 0 && a.rstd) a.rstd[m] = rs;
  norm_output<VPT, UE8M0>(a, m, nv, h, rs, w);
}

template <int VPT, bool UE8M0>
__global__ void __launch_bounds__(1024) rms_norm_ring_kernel(const NormFwd a, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][32];
  __shared__ __align__(8) uint64_t full[kMaxRing];
  __shared__ uint32_t aborted;
  volatile uint32_t* abort_flag = &aborted;
  const int T = blockDim.x, nv = a.K >> 3, step = gridDim.x;
  ChunkRing ring{{a.X, a.R, nullptr}, smem, full, stages, a.R ? 2 : 1, a.K * 2, 0, 0};
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(full + s), 1);
    aborted = 0;
    fence_mbarrier_init();
  }
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && blockIdx.x + static_cast<long long>(s) * step < a.M; ++s)
      ring.fill(blockIdx.x + s * step, s);
  uint4 w[VPT];
  load_weight<VPT>(a.W, nv, w);
  __syncthreads();
  int s = 0, par = 0;
  uint32_t ph = 0;
  for (long long m = blockIdx.x; m < a.M; m += step, par ^= 1) {
    const bool ok = wait_bar(smem_u32(full + s), ph, abort_flag, a);
    const size_t base = static_cast<size_t>(m) * nv;
    const uint4* x = reinterpret_cast<const uint4*>(ring.slot(s));
    float h[VPT][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + threadIdx.x;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
      if (v < nv && ok) ss += add_residual(a, base + v, x[v], a.R ? x[nv + v] : x[v], h[i]);
    }
    ss = block_sum(ss, red[par]);
    // every thread has read the slot: the row `stages` turns ahead may follow
    // (after a failed wait nothing more is loaded or stored)
    const bool go = *abort_flag == 0;
    if (threadIdx.x == 0 && go && m + static_cast<long long>(stages) * step < a.M)
      ring.fill(static_cast<int>(m) + stages * step, s);
    const float rs = __frsqrt_rn(ss / static_cast<float>(a.K) + a.eps);
    if (threadIdx.x == 0 && a.rstd && go) a.rstd[m] = rs;
    norm_output<VPT, UE8M0>(a, static_cast<int>(m), go ? nv : 0, h, rs, w);
    if (++s == stages) { s = 0; ph ^= 1; }
  }
  if (threadIdx.x == 0 && *abort_flag) ring.drain(a);
}

// Gradient, a row: the products' sum for dX, and the block's share of dW.
__device__ __forceinline__ float grad_sums(const uint4& dy, const uint4& hv, const uint4& wv, float rs,
                                           float (&g)[8], float (&xh)[8], float (&dw)[8]) {
  float w[8], dot = 0.f;
  bf16x8_to_float(dy, g);
  bf16x8_to_float(hv, xh);
  bf16x8_to_float(wv, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    xh[j] *= rs;
    dw[j] = fmaf(g[j], xh[j], dw[j]);
    g[j] *= w[j];
    dot = fmaf(g[j], xh[j], dot);
  }
  return dot;
}

__device__ __forceinline__ uint4 grad_row(const float (&g)[8], const float (&xh)[8], float rs,
                                          float mean, const uint4& dr) {
  float r[8];
  bf16x8_to_float(dr, r);
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = fmaf(rs, g[j] - xh[j] * mean, r[j]);
  return float_to_bf16x8(r);
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
    load_weight<VPT>(a.W, nv, w);
    float g[VPT][8], xh[VPT][8], dw[8] = {}, dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) dot += grad_sums(dy[i], hv[i], w[i], rs, g[i], xh[i], dw);
    const float mean = block_sum(dot, red) / static_cast<float>(a.K);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + threadIdx.x;
      if (v < nv) static_cast<uint4*>(a.dX)[base + v] = grad_row(g[i], xh[i], rs, mean, r[i]);
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
    a.dW[(blockIdx.x - a.M) * 64 + k] = sum;
  }
}

template <int VPT>
__global__ void __launch_bounds__(1024) rms_norm_backward_ring_kernel(const NormBwd a, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][32];
  __shared__ __align__(8) uint64_t full[kMaxRing];
  __shared__ uint32_t aborted;
  volatile uint32_t* abort_flag = &aborted;
  const int T = blockDim.x, nv = a.K >> 3, step = gridDim.x;
  ChunkRing ring{{a.dY, a.H, a.dR}, smem, full, stages, a.dR ? 3 : 2, a.K * 2, 0, 0};
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(full + s), 1);
    aborted = 0;
    fence_mbarrier_init();
  }
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && blockIdx.x + static_cast<long long>(s) * step < a.M; ++s)
      ring.fill(blockIdx.x + s * step, s);
  uint4 w[VPT];
  load_weight<VPT>(a.W, nv, w);
  __syncthreads();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  float dw[VPT][8] = {};
  int s = 0, par = 0;
  uint32_t ph = 0;
  for (long long m = blockIdx.x; m < a.M; m += step, par ^= 1) {
    const float rs = __ldg(a.rstd + m);
    const bool ok = wait_bar(smem_u32(full + s), ph, abort_flag, a);
    const size_t base = static_cast<size_t>(m) * nv;
    const uint4* x = reinterpret_cast<const uint4*>(ring.slot(s));
    float g[VPT][8], xh[VPT][8], dot = 0.f;
    uint4 r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + threadIdx.x;
      const bool on = v < nv && ok;
      r[i] = on && a.dR ? x[2 * nv + v] : zero;
      dot += grad_sums(on ? x[v] : zero, on ? x[nv + v] : zero, w[i], rs, g[i], xh[i], dw[i]);
    }
    const float mean = block_sum(dot, red[par]) / static_cast<float>(a.K);
    // (as in the forward kernel)
    const bool go = *abort_flag == 0;
    if (threadIdx.x == 0 && go && m + static_cast<long long>(stages) * step < a.M)
      ring.fill(static_cast<int>(m) + stages * step, s);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + threadIdx.x;
      if (v < nv && go) static_cast<uint4*>(a.dX)[base + v] = grad_row(g[i], xh[i], rs, mean, r[i]);
    }
    if (++s == stages) { s = 0; ph ^= 1; }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * T + threadIdx.x;
    if (v >= nv) continue;
    float4* out = reinterpret_cast<float4*>(a.part + static_cast<size_t>(blockIdx.x) * a.K) + 2 * v;
    out[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
    out[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
  }
  if (threadIdx.x == 0 && *abort_flag) ring.drain(a);
}

// dW[k] = sum of the blocks' partial sums, in a fixed order (32 columns per
// block, 32 chains over the partials).
__global__ void __launch_bounds__(1024)
rms_norm_weight_grad_kernel(const float* __restrict__ part, float* __restrict__ dW, int blocks,
                            int K) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5, k = blockIdx.x * 32 + c;
  float acc = 0.f;
  for (int b = r; b < blocks; b += 32) acc += part[static_cast<size_t>(b) * K + k];
  s[r][c] = acc;
  __syncthreads();
  // (transposed: warp r now sums the chains of column r)
  const float sum = warp_sum(s[c][r]);
  if (c == 0) dW[blockIdx.x * 32 + r] = sum;
}

// Threads of a block whose rows of K columns take `vpt` vectors per thread.
int row_threads(int K, int vpt) { return ((K / 8 + vpt - 1) / vpt + 31) / 32 * 32; }

struct RingShape {
  int blocks, threads, stages, smem;
};

// A ring per block, as many blocks per SM as a thousand threads make (their
// rings share the SM's memory), at least three slots each.
RingShape ring_shape(int M, int K, int ops, int vpt, int num_sms, int max_blocks) {
  RingShape r;
  r.threads = row_threads(K, vpt);
  const int slot = 2 * K * ops;
  const int per_sm = std::max(1, std::min(1024 / r.threads, ring_bytes(1) / (3 * slot)));
  r.stages = std::max(1, std::min(kMaxRing, ring_bytes(per_sm) / slot));
  r.blocks = std::min(std::min(M, per_sm * num_sms), max_blocks);
  r.smem = r.stages * slot;
  return r;
}

template <class... P, class... A>
cudaError_t launch_ring(void (*kernel)(P...), const RingShape& r, cudaStream_t stream, A... args) {
  return launch_dependent(kernel, dim3(r.blocks), r.threads, stream, r.smem, args..., r.stages);
}

template <bool UE8M0>
cudaError_t launch_fwd(const NormFwd& a, int num_sms, cudaStream_t stream) {
  const int vpt = a.K <= 8192 ? 1 : 2;
  if (a.M > 2 * num_sms) {
    const RingShape r = ring_shape(a.M, a.K, a.R ? 2 : 1, vpt, num_sms, a.M);
    return vpt == 1 ? launch_ring(rms_norm_ring_kernel<1, UE8M0>, r, stream, a)
                    : launch_ring(rms_norm_ring_kernel<2, UE8M0>, r, stream, a);
  }
  const int threads = row_threads(a.K, vpt);
  return vpt == 1 ? launch_dependent(rms_norm_kernel<1, UE8M0>, dim3(a.M), threads, stream, 0, a)
                  : launch_dependent(rms_norm_kernel<2, UE8M0>, dim3(a.M), threads, stream, 0, a);
}

}  // namespace

cudaError_t norm_set_up() {
  const void* kernels[] = {reinterpret_cast<const void*>(rms_norm_ring_kernel<1, false>),
                           reinterpret_cast<const void*>(rms_norm_ring_kernel<2, false>),
                           reinterpret_cast<const void*>(rms_norm_ring_kernel<1, true>),
                           reinterpret_cast<const void*>(rms_norm_ring_kernel<2, true>),
                           reinterpret_cast<const void*>(rms_norm_backward_ring_kernel<1>),
                           reinterpret_cast<const void*>(rms_norm_backward_ring_kernel<2>)};
  for (const void* k : kernels) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ring_bytes(1));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_rms_norm(const NormFwd& a, bool ue8m0, int num_sms, cudaStream_t stream) {
  return ue8m0 ? launch_fwd<true>(a, num_sms, stream) : launch_fwd<false>(a, num_sms, stream);
}

cudaError_t launch_rms_norm_backward(const NormBwd& a, int num_sms, cudaStream_t stream) {
  const int vpt = a.K <= 8192 ? 1 : 2;
  if (a.M <= 4 * num_sms) {
    const int threads = row_threads(a.K, vpt);
    const dim3 grid(a.M + a.K / 64);
    const int smem = threads / 8 * 64 * 4;
    return vpt == 1 ? launch_dependent(rms_norm_backward_kernel<1>, grid, threads, stream, smem, a)
                    : launch_dependent(rms_norm_backward_kernel<2>, grid, threads, stream, smem, a);
  }
  const RingShape r = ring_shape(a.M, a.K, a.dR ? 3 : 2, vpt, num_sms, kNormBwdBlocks);
  const cudaError_t e = vpt == 1 ? launch_ring(rms_norm_backward_ring_kernel<1>, r, stream, a)
                                 : launch_ring(rms_norm_backward_ring_kernel<2>, r, stream, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(rms_norm_weight_grad_kernel, dim3(a.K / 32), 1024, stream, 0,
                          static_cast<const float*>(a.part), a.dW, r.blocks, a.K);
}

}  // namespace dgk
