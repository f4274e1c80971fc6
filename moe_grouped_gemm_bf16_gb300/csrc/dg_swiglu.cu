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
// and 4 to 6 written backward.  Eight lanes take one row's 128-column group,
// columns 8 j .. 8 j + 7 and 64 + 8 j .. each (lane j), so a group's maximum is
// a 3-step shuffle and the lanes' 16-byte accesses are consecutive.  Two forms:
//  * one block per 32 rows of a group, loads straight to registers: few rows,
//    and the masked layout;
//  * persistent blocks fed by bulk copies of whole rows into a ring in shared
//    memory, for many rows (registers alone do not keep enough loads in
//    flight).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dg_fp8.cuh"
#include "dg_launch.h"
#include "dg_params.h"
#include "dg_ring.cuh"
#include "dg_swiglu.h"

namespace dgk {
namespace {

constexpr int SG_THREADS = 256;   // direct form: 32 rows of one 128-column group

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

// Maximum over the 8 lanes of a group, floored.
__device__ __forceinline__ float lanes_max(float a) {
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return fmaxf(a, kScaleFloor);
}

__device__ __forceinline__ float group_max(const float* x) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]));
  return lanes_max(a);
}

__device__ __forceinline__ uint2 quantise8(const float* x, float f) {
  return make_uint2(cvt_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f),
                    cvt_e4m3x4(x[4] * f, x[5] * f, x[6] * f, x[7] * f));
}

__device__ __forceinline__ void dequantise8(const uint2& w, float s, float* x) {
  const uint32_t c[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 lo = e4m3x2_to_float2(c[i] & 0xFFFFu), hi = e4m3x2_to_float2(c[i] >> 16);
    x[4 * i] = lo.x * s;
    x[4 * i + 1] = lo.y * s;
    x[4 * i + 2] = hi.x * s;
    x[4 * i + 3] = hi.y * s;
  }
}

// Where lane j of the group `grp` of row m of batch z finds its two vectors of
// 8 columns: [at] and [at + 8] of a tensor of I columns, [gate], [gate + 8],
// [up], [up + 8] of one of 2 I columns (in vectors).
struct Place {
  int z, m, grp, lane8;
  size_t at, gate, up;
  __device__ __forceinline__ Place(int z_, int m_, int grp_, int j, int M, int I)
      : z(z_), m(m_), grp(grp_), lane8(j) {
    const size_t row = static_cast<size_t>(z) * M + m;
    at = row * (I >> 3) + grp * 16 + j;
    gate = row * (I >> 2) + grp * 16 + j;
    up = gate + (I >> 3);
  }
};

// One lane's share of a group, forward: v = {gate, gate + 8, up, up + 8}.
// Every lane of the warp takes part; `on`: this one's row is stored.
template <bool UE8M0>
__device__ __forceinline__ void forward_group(const SwigluFwd& a, const Place& p, const uint4 (&v)[4],
                                              bool on) {
  const int kb = a.I >> 7;
  float g[16], u[16], y[16];
  bf16x8_to_float(v[0], g);
  bf16x8_to_float(v[1], g + 8);
  bf16x8_to_float(v[2], u);
  bf16x8_to_float(v[3], u + 8);
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = g[i] * sigmoid(g[i]) * u[i];
  if (a.Y && on) {
    uint4* Y = static_cast<uint4*>(a.Y) + p.at;
    Y[0] = float_to_bf16x8(y);
    Y[8] = float_to_bf16x8(y + 8);
  }
  float f;
  uint32_t e8;
  if (a.Q) {
    const float amax = group_max(y);
    group_factor<UE8M0>(amax, f, e8);
    if (on) {
      uint2* Q = static_cast<uint2*>(a.Q) + p.at;
      Q[0] = quantise8(y, f);
      Q[8] = quantise8(y + 8, f);
      if (p.lane8 == 0)
        store_scale<UE8M0>(static_cast<float*>(a.sa), p.z, kb, a.ld, p.grp, p.m, amax, e8);
    }
  }
  if (a.CQ) {
    const float ag = group_max(g), au = group_max(u);
    uint2* CQ = static_cast<uint2*>(a.CQ);
    if (on) {
      group_factor<false>(ag, f, e8);
      CQ[p.gate] = quantise8(g, f);
      CQ[p.gate + 8] = quantise8(g + 8, f);
      group_factor<false>(au, f, e8);
      CQ[p.up] = quantise8(u, f);
      CQ[p.up + 8] = quantise8(u + 8, f);
      if (p.lane8 == 0) {
        store_scale<false>(a.csa, p.z, 2 * kb, a.ld, p.grp, p.m, ag, 0);
        store_scale<false>(a.csa, p.z, 2 * kb, a.ld, kb + p.grp, p.m, au, 0);
      }
    }
  }
}

// The same backward: c = codes of {gate, gate + 8, up, up + 8}, their scales
// sg and su, d = the gradient's two vectors.
__device__ __forceinline__ void backward_group(const SwigluBwd& a, const Place& p,
                                               const uint2 (&c)[4], float sg, float su,
                                               const uint4 (&dv)[2]) {
  uint4* dGU = static_cast<uint4*>(a.dGU);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float g[8], u[8], d[8], y[8];
    dequantise8(c[h], sg, g);
    dequantise8(c[2 + h], su, u);
    bf16x8_to_float(dv[h], d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(g[i]), gs = g[i] * s;
      y[i] = gs * u[i];
      // s (1 + g (1 - s)) = s + g s (1 - s)
      g[i] = d[i] * u[i] * fmaf(gs, 1.0f - s, s);
      u[i] = d[i] * gs;
    }
    dGU[p.gate + 8 * h] = float_to_bf16x8(g);
    dGU[p.up + 8 * h] = float_to_bf16x8(u);
    if (a.Y) static_cast<uint4*>(a.Y)[p.at + 8 * h] = float_to_bf16x8(y);
  }
}

template <bool UE8M0>
__global__ void __launch_bounds__(SG_THREADS) swiglu_kernel(const SwigluFwd a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int m = blockIdx.x * 32 + (threadIdx.x >> 3), z = blockIdx.z;
  const int rows = valid_rows(a.masked_m, z, a.M, a.status);
  if (static_cast<int>(blockIdx.x) * 32 >= rows) return;
  const Place p(z, m, blockIdx.y, threadIdx.x & 7, a.M, a.I);
  const bool on = m < rows;
  uint4 v[4] = {};
  if (on) {
    const uint4* GU = static_cast<const uint4*>(a.GU);
    v[0] = ld_stream_v4(GU + p.gate);
    v[1] = ld_stream_v4(GU + p.gate + 8);
    v[2] = ld_stream_v4(GU + p.up);
    v[3] = ld_stream_v4(GU + p.up + 8);
  }
  forward_group<UE8M0>(a, p, v, on);
}

__global__ void __launch_bounds__(SG_THREADS) swiglu_backward_kernel(const SwigluBwd a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int m = blockIdx.x * 32 + (threadIdx.x >> 3), z = blockIdx.z, kb = a.I >> 7;
  if (m >= valid_rows(a.masked_m, z, a.M, a.status)) return;
  const Place p(z, m, blockIdx.y, threadIdx.x & 7, a.M, a.I);
  const uint2* CQ = static_cast<const uint2*>(a.CQ);
  const uint4* dY = static_cast<const uint4*>(a.dY);
  const uint2 c[4] = {__ldg(CQ + p.gate), __ldg(CQ + p.gate + 8), __ldg(CQ + p.up),
                      __ldg(CQ + p.up + 8)};
  const uint4 d[2] = {ld_stream_v4(dY + p.at), ld_stream_v4(dY + p.at + 8)};
  const float* cs = a.csa + static_cast<size_t>(z) * (2 * kb) * a.ld + m;
  backward_group(a, p, c, __ldg(cs + static_cast<size_t>(p.grp) * a.ld),
                 __ldg(cs + static_cast<size_t>(kb + p.grp) * a.ld), d);
}

// Ring form: a chunk is `rows` whole rows, of which a thread takes one lane's
// share of a group at a time.
template <bool UE8M0>
__global__ void __launch_bounds__(SG_THREADS) swiglu_ring_kernel(const SwigluFwd a, int rows,
                                                                 int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kMaxRing];
  __shared__ uint32_t aborted;
  volatile uint32_t* abort_flag = &aborted;
  const int lanes = a.I >> 4, total = a.G * a.M;   // lanes per row, rows
  ChunkRing ring{{a.GU, nullptr, nullptr}, smem, full, stages, 1, rows * a.I * 4, 0, 0};
  auto fill = [&](int c, int s) { ring.fill(c, s, min(rows, total - c * rows) * a.I * 4); };
  const int chunks = (total + rows - 1) / rows;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(full + s), 1);
    aborted = 0;
    fence_mbarrier_init();
  }
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && blockIdx.x + s * gridDim.x < chunks; ++s)
      fill(blockIdx.x + s * gridDim.x, s);
  __syncthreads();
  int s = 0;
  uint32_t ph = 0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const bool ok = wait_bar(smem_u32(full + s), ph, abort_flag, a);
    const int n = ok ? min(rows, total - c * rows) * lanes : 0;
    const uint4* x = reinterpret_cast<const uint4*>(ring.slot(s));
    for (int u0 = threadIdx.x & ~31; u0 < n; u0 += SG_THREADS) {
      const int u = u0 + (threadIdx.x & 31), r = u / lanes, q = u - r * lanes;
      const int row = c * rows + r, z = row / a.M;
      const Place p(z, row - z * a.M, q >> 3, q & 7, a.M, a.I);
      const uint4* g = x + r * (a.I >> 2) + p.grp * 16 + p.lane8;
      const bool on = u < n;
      uint4 v[4] = {};
      if (on) {
        v[0] = g[0];
        v[1] = g[8];
        v[2] = g[a.I >> 3];
        v[3] = g[(a.I >> 3) + 8];
      }
      forward_group<UE8M0>(a, p, v, on);
    }
    __syncthreads();   // the slot has been read
    const long long next = c + static_cast<long long>(stages) * gridDim.x;
    if (threadIdx.x == 0 && next < chunks && *abort_flag == 0) fill(static_cast<int>(next), s);
    if (++s == stages) { s = 0; ph ^= 1; }
  }
  if (threadIdx.x == 0 && *abort_flag) ring.drain(a);
}

// (the codes are a row of 2 I bytes, and so is the gradient's row: two operands
// of equal chunks)
__global__ void __launch_bounds__(SG_THREADS) swiglu_backward_ring_kernel(const SwigluBwd a, int rows,
                                                                          int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kMaxRing];
  __shared__ uint32_t aborted;
  volatile uint32_t* abort_flag = &aborted;
  const int lanes = a.I >> 4, total = a.G * a.M, kb = a.I >> 7;
  ChunkRing ring{{a.CQ, a.dY, nullptr}, smem, full, stages, 2, rows * a.I * 2, 0, 0};
  auto fill = [&](int c, int s) { ring.fill(c, s, min(rows, total - c * rows) * a.I * 2); };
  const int chunks = (total + rows - 1) / rows;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(full + s), 1);
    aborted = 0;
    fence_mbarrier_init();
  }
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && blockIdx.x + s * gridDim.x < chunks; ++s)
      fill(blockIdx.x + s * gridDim.x, s);
  __syncthreads();
  int s = 0;
  uint32_t ph = 0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const bool ok = wait_bar(smem_u32(full + s), ph, abort_flag, a);
    const int n = ok ? min(rows, total - c * rows) * lanes : 0;
    const uint2* x = reinterpret_cast<const uint2*>(ring.slot(s));
    const uint4* y = reinterpret_cast<const uint4*>(ring.slot(s) + ring.bytes);
    for (int u = threadIdx.x; u < n; u += SG_THREADS) {
      const int r = u / lanes, q = u - r * lanes;
      const int row = c * rows + r, z = row / a.M;
      const Place p(z, row - z * a.M, q >> 3, q & 7, a.M, a.I);
      const float* cs = a.csa + static_cast<size_t>(z) * (2 * kb) * a.ld + p.m;
      const float sg = __ldg(cs + static_cast<size_t>(p.grp) * a.ld);
      const float su = __ldg(cs + static_cast<size_t>(kb + p.grp) * a.ld);
      const uint2* g = x + r * (a.I >> 2) + p.grp * 16 + p.lane8;
      const uint4* dy = y + r * (a.I >> 3) + p.grp * 16 + p.lane8;
      const uint2 cd[4] = {g[0], g[8], g[a.I >> 3], g[(a.I >> 3) + 8]};
      const uint4 d[2] = {dy[0], dy[8]};
      backward_group(a, p, cd, sg, su, d);
    }
    __syncthreads();   // the slot has been read
    const long long next = c + static_cast<long long>(stages) * gridDim.x;
    if (threadIdx.x == 0 && next < chunks && *abort_flag == 0) fill(static_cast<int>(next), s);
    if (++s == stages) { s = 0; ph ^= 1; }
  }
  if (threadIdx.x == 0 && *abort_flag) ring.drain(a);
}

dim3 grid_of(int G, int M, int I) { return dim3((M + 31) / 32, I / 128, G); }

struct RingShape {
  int rows, stages, smem, blocks;
};

// Chunks of about CHUNK bytes in rows of `row` bytes, PER_SM blocks per SM.
// Returns stages = 0 where a row is too long for a ring of two.
template <int PER_SM, int CHUNK>
RingShape ring_shape(long long total, int row, int num_sms) {
  RingShape r;
  r.rows = std::max(1, CHUNK / row);
  r.stages = std::min(kMaxRing, ring_bytes(PER_SM) / (r.rows * row));
  if (r.stages < 2) r.stages = 0;
  r.smem = r.stages * r.rows * row;
  r.blocks = static_cast<int>(std::min<long long>((total + r.rows - 1) / r.rows,
                                                  static_cast<long long>(PER_SM) * num_sms));
  return r;
}

constexpr int kFwdPerSm = 3, kBwdPerSm = 4, kChunk = 16384;

}  // namespace

cudaError_t swiglu_set_up() {
  cudaError_t e = cudaFuncSetAttribute(swiglu_ring_kernel<false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       ring_bytes(kFwdPerSm));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(swiglu_ring_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ring_bytes(kFwdPerSm));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(swiglu_backward_ring_kernel,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, ring_bytes(kBwdPerSm));
  return e;
}

cudaError_t launch_swiglu(const SwigluFwd& a, bool ue8m0, int num_sms, cudaStream_t stream) {
  const long long total = static_cast<long long>(a.G) * a.M;
  const RingShape r = ring_shape<kFwdPerSm, kChunk>(total, 4 * a.I, num_sms);
  if (!a.masked_m && r.stages && total < (1ll << 31) && r.blocks == kFwdPerSm * num_sms)
    return launch_dependent(ue8m0 ? swiglu_ring_kernel<true> : swiglu_ring_kernel<false>,
                            dim3(r.blocks), SG_THREADS, stream, r.smem, a, r.rows, r.stages);
  return launch_dependent(ue8m0 ? swiglu_kernel<true> : swiglu_kernel<false>,
                          grid_of(a.G, a.M, a.I), SG_THREADS, stream, 0, a);
}

cudaError_t launch_swiglu_backward(const SwigluBwd& a, int num_sms, cudaStream_t stream) {
  const long long total = static_cast<long long>(a.G) * a.M;
  const RingShape r = ring_shape<kBwdPerSm, kChunk>(total, 4 * a.I, num_sms);
  if (!a.masked_m && r.stages && total < (1ll << 31) && r.blocks == kBwdPerSm * num_sms)
    return launch_dependent(swiglu_backward_ring_kernel, dim3(r.blocks), SG_THREADS, stream, r.smem,
                            a, r.rows, r.stages);
  return launch_dependent(swiglu_backward_kernel, grid_of(a.G, a.M, a.I), SG_THREADS, stream, 0, a);
}

}  // namespace dgk
