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
// Both are memory-bound: a row is read once and stays in registers between
// the statistics and the output (8 columns per 16-byte vector, VPT vectors per
// thread).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dg_fp8.cuh"
#include "dg_launch.h"
#include "dg_norm.h"

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

template <int VPT, bool UE8M0>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormFwd a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ float red[2][32];
  const int T = blockDim.x, nv = a.K >> 3, kb = a.K >> 7;
  const uint4* X = static_cast<const uint4*>(a.X);
  const uint4* R = static_cast<const uint4*>(a.R);
  const uint4* W = static_cast<const uint4*>(a.W);
  int par = 0;
  for (int m = blockIdx.x; m < a.M; m += gridDim.x, par ^= 1) {
    const size_t base = static_cast<size_t>(m) * nv;
    float h[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + threadIdx.x;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
      if (v < nv) {
        bf16x8_to_float(ld_stream_v4(X + base + v), h[i]);
        if (R) {
          float r[8];
          bf16x8_to_float(ld_stream_v4(R + base + v), r);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += r[j];
          if (a.H) static_cast<uint4*>(a.H)[base + v] = float_to_bf16x8(h[i]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    }
    ss = block_sum(ss, red[par]);
    const float rs = __frsqrt_rn(ss / static_cast<float>(a.K) + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[m] = rs;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + threadIdx.x;
      float w[8] = {};
      if (v < nv) bf16x8_to_float(__ldg(W + v), w);
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] = h[i][j] * rs * w[j];
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
}

template <int VPT>
__global__ void __launch_bounds__(1024) rms_norm_backward_kernel(const NormBwd a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ float red[2][32];
  const int T = blockDim.x, nv = a.K >> 3;
  const uint4* dY = static_cast<const uint4*>(a.dY);
  const uint4* H = static_cast<const uint4*>(a.H);
  const uint4* dR = static_cast<const uint4*>(a.dR);
  const uint4* W = static_cast<const uint4*>(a.W);
  float dw[VPT][8] = {};
  int par = 0;
  for (int m = blockIdx.x; m < a.M; m += gridDim.x, par ^= 1) {
    const size_t base = static_cast<size_t>(m) * nv;
    const float rs = __ldg(a.rstd + m);
    float g[VPT][8], xh[VPT][8];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + threadIdx.x;
      float w[8] = {};
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = xh[i][j] = 0.f;
      if (v < nv) {
        bf16x8_to_float(ld_stream_v4(dY + base + v), g[i]);
        bf16x8_to_float(ld_stream_v4(H + base + v), xh[i]);
        bf16x8_to_float(__ldg(W + v), w);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] *= rs;
        dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
        g[i][j] *= w[j];
        dot = fmaf(g[i][j], xh[i][j], dot);
      }
    }
    dot = block_sum(dot, red[par]) / static_cast<float>(a.K);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * T + threadIdx.x;
      if (v >= nv) continue;
      float r[8] = {};
      if (dR) bf16x8_to_float(ld_stream_v4(dR + base + v), r);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = fmaf(rs, g[i][j] - xh[i][j] * dot, r[j]);
      static_cast<uint4*>(a.dX)[base + v] = float_to_bf16x8(r);
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * T + threadIdx.x;
    if (v >= nv) continue;
    float4* out = reinterpret_cast<float4*>(a.part + static_cast<size_t>(blockIdx.x) * a.K) + 2 * v;
    out[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
    out[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
  }
}

// dW[k] = sum of the blocks' partial sums, in a fixed order (32 columns per
// block, 8 rows of threads over the partials).
__global__ void __launch_bounds__(256)
rms_norm_weight_grad_kernel(const float* __restrict__ part, float* __restrict__ dW, int blocks,
                            int K) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ float s[8][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5, k = blockIdx.x * 32 + c;
  float acc = 0.f;
  for (int b = r; b < blocks; b += 8) acc += part[static_cast<size_t>(b) * K + k];
  s[r][c] = acc;
  __syncthreads();
  if (r == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += s[i][c];
    dW[k] = acc;
  }
}

// Threads per row and vectors per thread for rows of K columns.
void row_shape(int K, int vpt, int* threads) {
  const int nv = K / 8;
  *threads = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
}

template <bool UE8M0>
cudaError_t launch_fwd(const NormFwd& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const int vpt = a.K <= 8192 ? 1 : 2;
  int threads = 0;
  row_shape(a.K, vpt, &threads);
  return vpt == 1 ? launch_dependent(rms_norm_kernel<1, UE8M0>, dim3(a.M), threads, stream, a)
                  : launch_dependent(rms_norm_kernel<2, UE8M0>, dim3(a.M), threads, stream, a);
}

}  // namespace

cudaError_t launch_rms_norm(const NormFwd& a, bool ue8m0, int num_sms, cudaStream_t stream) {
  return ue8m0 ? launch_fwd<true>(a, num_sms, stream) : launch_fwd<false>(a, num_sms, stream);
}

cudaError_t launch_rms_norm_backward(const NormBwd& a, int num_sms, cudaStream_t stream) {
  const int blocks = std::min(std::min(a.M, 2 * num_sms), kNormBwdBlocks);
  cudaError_t e = cudaSuccess;
  if (blocks > 0) {
    const int vpt = a.K <= 8192 ? 1 : 2;
    int threads = 0;
    row_shape(a.K, vpt, &threads);
    e = vpt == 1 ? launch_dependent(rms_norm_backward_kernel<1>, dim3(blocks), threads, stream, a)
                 : launch_dependent(rms_norm_backward_kernel<2>, dim3(blocks), threads, stream, a);
  }
  if (e != cudaSuccess) return e;
  return launch_dependent(rms_norm_weight_grad_kernel, dim3(a.K / 32), 256, stream,
                    static_cast<const float*>(a.part), a.dW, blocks, a.K);
}

}  // namespace dgk
