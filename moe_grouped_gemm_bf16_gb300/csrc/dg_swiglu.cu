// Gated activation between an expert's two products, with its output
// quantised 1x128 to e4m3 (the left operand of the second product), an 8-bit
// checkpoint of its input for the backward pass, and the gradient computed
// from that checkpoint.  Per element, in fp32:
//
//   s = 1 / (1 + exp(-g)),   y = g s u
//   dg = dy u s (1 + g (1 - s)),   du = dy g s
//
// g and u are the two halves of a row of GU; the checkpoint (CQ, csa) is GU's
// 1x128 quantisation, with which the backward pass reads g = code * scale.
//
// Memory-bound: 4 bytes read and 1 to 5 written per element forward, 4 read
// and 4 to 6 written backward.  Eight lanes take one row's 128-column group, 16
// columns each (the quantiser's split), so a group's maximum is a 3-step
// shuffle; a block takes ROWS rows of 32 of one group in each pass.
#include <cuda_runtime.h>
#include <stdint.h>

#include "dg_fp8.cuh"
#include "dg_launch.h"
#include "dg_params.h"
#include "dg_swiglu.h"

namespace dgk {
namespace {

constexpr int SG_THREADS = 256;   // 32 rows of one 128-column group
constexpr int SG_ROWS = 1;        // rows per thread

__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// Rows of batch z that hold a token, the count clamped to [0, M] (reported).
__device__ __forceinline__ int valid_rows(const int32_t* masked_m, int z, int M,
                                          unsigned int* status) {
  if (!masked_m) return M;
  const int v = __ldg(masked_m + z);
  const int c = min(max(v, 0), M);
  if (c != v && threadIdx.x == 0) atomicCAS(status, 0u, ST_MASK_RANGE);
  return c;
}

// Maximum over the 8 lanes of a group.
__device__ __forceinline__ float group_max(const float* x) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return fmaxf(a, kScaleFloor);
}

__device__ __forceinline__ uint4 quantise16(const float* x, float f) {
  uint4 w;
  w.x = cvt_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
  w.y = cvt_e4m3x4(x[4] * f, x[5] * f, x[6] * f, x[7] * f);
  w.z = cvt_e4m3x4(x[8] * f, x[9] * f, x[10] * f, x[11] * f);
  w.w = cvt_e4m3x4(x[12] * f, x[13] * f, x[14] * f, x[15] * f);
  return w;
}

__device__ __forceinline__ void dequantise16(const uint4& w, float s, float* x) {
  const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = e4m3x2_to_float2(c[i] & 0xFFFFu), hi = e4m3x2_to_float2(c[i] >> 16);
    x[4 * i] = lo.x * s;
    x[4 * i + 1] = lo.y * s;
    x[4 * i + 2] = hi.x * s;
    x[4 * i + 3] = hi.y * s;
  }
}

template <bool UE8M0>
__global__ void __launch_bounds__(SG_THREADS) swiglu_kernel(const SwigluFwd a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int sub = threadIdx.x & 7;
  const int row0 = blockIdx.x * (32 * SG_ROWS) + (threadIdx.x >> 3);
  const int grp = blockIdx.y, z = blockIdx.z, kb = a.I >> 7;
  const int rows = valid_rows(a.masked_m, z, a.M, a.status);
  if (blockIdx.x * (32 * SG_ROWS) >= rows) return;
#pragma unroll
  for (int j = 0; j < SG_ROWS; ++j) {
    const int m = row0 + 32 * j;
    const bool on = m < rows;
    const size_t row = static_cast<size_t>(z) * a.M + m;
    // in 16-column units: this thread's columns of a row of I columns
    const size_t at = row * (a.I >> 4) + grp * 8 + sub;
    const size_t gate = row * (a.I >> 3) + grp * 8 + sub, up = gate + (a.I >> 4);
    float g[16] = {}, u[16] = {}, y[16];
    if (on) {
      const uint4* GU = static_cast<const uint4*>(a.GU);
      const uint4 v0 = ld_stream_v4(GU + 2 * gate), v1 = ld_stream_v4(GU + 2 * gate + 1);
      const uint4 v2 = ld_stream_v4(GU + 2 * up), v3 = ld_stream_v4(GU + 2 * up + 1);
      bf16x8_to_float(v0, g);
      bf16x8_to_float(v1, g + 8);
      bf16x8_to_float(v2, u);
      bf16x8_to_float(v3, u + 8);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = g[i] * sigmoid(g[i]) * u[i];
    if (a.Y && on) {
      uint4* Y = static_cast<uint4*>(a.Y) + 2 * at;
      Y[0] = float_to_bf16x8(y);
      Y[1] = float_to_bf16x8(y + 8);
    }
    float f;
    uint32_t e8;
    if (a.Q) {
      const float amax = group_max(y);
      group_factor<UE8M0>(amax, f, e8);
      const uint4 q = quantise16(y, f);
      if (on) {
        static_cast<uint4*>(a.Q)[at] = q;
        if (sub == 0) store_scale<UE8M0>(static_cast<float*>(a.sa), z, kb, a.ld, grp, m, amax, e8);
      }
    }
    if (a.CQ) {
      const float ag = group_max(g), au = group_max(u);
      uint4* CQ = static_cast<uint4*>(a.CQ);
      group_factor<false>(ag, f, e8);
      const uint4 qg = quantise16(g, f);
      group_factor<false>(au, f, e8);
      const uint4 qu = quantise16(u, f);
      if (on) {
        CQ[gate] = qg;
        CQ[up] = qu;
        if (sub == 0) {
          store_scale<false>(a.csa, z, 2 * kb, a.ld, grp, m, ag, 0);
          store_scale<false>(a.csa, z, 2 * kb, a.ld, kb + grp, m, au, 0);
        }
      }
    }
  }
}

__global__ void __launch_bounds__(SG_THREADS) swiglu_backward_kernel(const SwigluBwd a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int sub = threadIdx.x & 7;
  const int row0 = blockIdx.x * (32 * SG_ROWS) + (threadIdx.x >> 3);
  const int grp = blockIdx.y, z = blockIdx.z, kb = a.I >> 7;
  const int rows = valid_rows(a.masked_m, z, a.M, a.status);
#pragma unroll
  for (int j = 0; j < SG_ROWS; ++j) {
    const int m = row0 + 32 * j;
    if (m >= rows) continue;
    const size_t row = static_cast<size_t>(z) * a.M + m;
    const size_t at = row * (a.I >> 4) + grp * 8 + sub;
    const size_t gate = row * (a.I >> 3) + grp * 8 + sub, up = gate + (a.I >> 4);
    const uint4* CQ = static_cast<const uint4*>(a.CQ);
    const uint4* dY = static_cast<const uint4*>(a.dY);
    const uint4 cg = ld_stream_v4(CQ + gate), cu = ld_stream_v4(CQ + up);
    const uint4 d0 = ld_stream_v4(dY + 2 * at), d1 = ld_stream_v4(dY + 2 * at + 1);
    const float* cs = a.csa + static_cast<size_t>(z) * (2 * kb) * a.ld + m;
    const float sg = __ldg(cs + static_cast<size_t>(grp) * a.ld);
    const float su = __ldg(cs + static_cast<size_t>(kb + grp) * a.ld);
    float g[16], u[16], d[16], y[16];
    dequantise16(cg, sg, g);
    dequantise16(cu, su, u);
    bf16x8_to_float(d0, d);
    bf16x8_to_float(d1, d + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float s = sigmoid(g[i]), gs = g[i] * s;
      y[i] = gs * u[i];
      // s (1 + g (1 - s)) = s + g s (1 - s)
      g[i] = d[i] * u[i] * fmaf(gs, 1.0f - s, s);
      u[i] = d[i] * gs;
    }
    uint4* dGU = static_cast<uint4*>(a.dGU);
    dGU[2 * gate] = float_to_bf16x8(g);
    dGU[2 * gate + 1] = float_to_bf16x8(g + 8);
    dGU[2 * up] = float_to_bf16x8(u);
    dGU[2 * up + 1] = float_to_bf16x8(u + 8);
    if (a.Y) {
      uint4* Y = static_cast<uint4*>(a.Y) + 2 * at;
      Y[0] = float_to_bf16x8(y);
      Y[1] = float_to_bf16x8(y + 8);
    }
  }
}

dim3 grid_of(int G, int M, int I) {
  return dim3((M + 32 * SG_ROWS - 1) / (32 * SG_ROWS), I / 128, G);
}

}  // namespace

cudaError_t launch_swiglu(const SwigluFwd& a, bool ue8m0, cudaStream_t stream) {
  return launch_dependent(ue8m0 ? swiglu_kernel<true> : swiglu_kernel<false>,
                          grid_of(a.G, a.M, a.I), SG_THREADS, stream, 0, a);
}

cudaError_t launch_swiglu_backward(const SwigluBwd& a, cudaStream_t stream) {
  return launch_dependent(swiglu_backward_kernel, grid_of(a.G, a.M, a.I), SG_THREADS, stream, 0, a);
}

}  // namespace dgk
