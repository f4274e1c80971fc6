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
// Under a limit on the SMs either form has one block per SM, of the threads that
// otherwise share one (132 of the 152 SMs, 32647 rows, I = 2048, with checkpoint: 87
// us, with all 75; the gradient 118 and 104).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <utility>

#include "dg_fp8.cuh"
#include "dg_launch.h"
#include "dg_params.h"
#include "dg_ring.cuh"
#include "dg_swiglu.h"

namespace dgk {
namespace {

constexpr int SG_THREADS = 256;   // direct form: 32 rows of one 128-column group
constexpr int SG_WALK = 1024;     // under a limit on the SMs: 128 rows at a time

// 1 / (1 + exp(-g)) with the hardware's exponential and reciprocal; a gate whose
// exponential is not finite gives 0 (below -88) or 1.
__device__ __forceinline__ float2 sigmoid2(float2 g) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float2 t = mul2(g, make_float2(-kLog2e, -kLog2e));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = add2(e, make_float2(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
  return r;
}

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
  // Checked build: the places lie in tensors of G batches, the row in its scales'.
  template <class P>
  __device__ __forceinline__ bool inside(const P& a) const {
    const size_t rows = static_cast<size_t>(a.G) * a.M;
    return in_bounds(a, at, 9, rows * (a.I >> 3)) && in_bounds(a, gate, 9, rows * (a.I >> 2)) &&
           in_bounds(a, up, 9, rows * (a.I >> 2)) && in_bounds(a, grp, 1, a.I >> 7) &&
           in_bounds(a, z, 1, a.G) && in_bounds(a, m, 1, a.M);
  }
};

// One lane's share of a group, forward: v = {gate, gate + 8, up, up + 8}.
// Every lane of the warp takes part; `on`: this one's row is stored.
//
// The time goes to instructions as much as to memory (38.8 per element in a
// plain version, 28.8 so), so values are taken in pairs and the group's six
// quotients are shared out over its lanes: 448 / a for y, gate and up in lanes
// 0 to 2 (the others fetch them), a / 448 in lanes 3 to 5, which store them.
template <bool UE8M0>
__device__ __forceinline__ void forward_group(const SwigluFwd& a, const Place& p, const uint4 (&v)[4],
                                              bool on) {
  const int kb = a.I >> 7;
  Pairs g[2] = {bf16x8_to_pairs(v[0]), bf16x8_to_pairs(v[1])};
  Pairs u[2] = {bf16x8_to_pairs(v[2]), bf16x8_to_pairs(v[3])};
  Pairs y[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[h].v[i] = mul2(mul2(g[h].v[i], sigmoid2(g[h].v[i])), u[h].v[i]);
  on = on && p.inside(a);
  if (a.Y && on) {
    uint4* Y = static_cast<uint4*>(a.Y) + p.at;
    Y[0] = pairs_to_bf16x8(y[0]);
    Y[8] = pairs_to_bf16x8(y[1]);
  }
  float ay = kScaleFloor, ag = kScaleFloor, au = kScaleFloor;
  if (a.Q) ay = fminf(lanes_max(fmaxf(pairs_amax(y[0]), pairs_amax(y[1]))), kScaleTop);
  if (a.CQ) {
    ag = lanes_max(fmaxf(bf16x8_amax(v[0]), bf16x8_amax(v[1])));
    au = lanes_max(fmaxf(bf16x8_amax(v[2]), bf16x8_amax(v[3])));
  }
  const int j = p.lane8;
  const float mine = (j == 0 || j == 3) ? ay : (j == 1 || j == 4) ? ag : au;
  const float quot = j < 3 ? __fdiv_rn(448.0f, mine) : __fdiv_rn(mine, 448.0f);
  const int first = (threadIdx.x & 31) - j;
  if (a.Q) {
    float f;
    uint32_t e8;
    if constexpr (UE8M0) group_factor<true>(ay, f, e8);
    else f = __shfl_sync(0xffffffffu, quot, first);
    if (on) {
      uint2* Q = static_cast<uint2*>(a.Q) + p.at;
      Q[0] = pairs_to_e4m3x8(y[0], f);
      Q[8] = pairs_to_e4m3x8(y[1], f);
      if constexpr (UE8M0) {
        if (j == 3) store_scale<true>(static_cast<float*>(a.sa), p.z, kb, a.ld, p.grp, p.m, ay, e8);
      } else {
        if (j == 3)
          static_cast<float*>(a.sa)[(static_cast<size_t>(p.z) * kb + p.grp) * a.ld + p.m] = quot;
      }
    }
  }
  if (a.CQ) {
    const float fg = __shfl_sync(0xffffffffu, quot, first + 1);
    const float fu = __shfl_sync(0xffffffffu, quot, first + 2);
    if (on) {
      uint2* CQ = static_cast<uint2*>(a.CQ);
      CQ[p.gate] = pairs_to_e4m3x8(g[0], fg);
      CQ[p.gate + 8] = pairs_to_e4m3x8(g[1], fg);
      CQ[p.up] = pairs_to_e4m3x8(u[0], fu);
      CQ[p.up + 8] = pairs_to_e4m3x8(u[1], fu);
      if (j == 4 || j == 5)
        a.csa[(static_cast<size_t>(p.z) * (2 * kb) + (j - 4) * kb + p.grp) * a.ld + p.m] = quot;
    }
  }
}

// The same backward: c = codes of {gate, gate + 8, up, up + 8}, their scales
// sg and su, d = the gradient's two vectors.
__device__ __forceinline__ void backward_group(const SwigluBwd& a, const Place& p,
                                               const uint2 (&c)[4], float sg, float su,
                                               const uint4 (&dv)[2]) {
  if (!p.inside(a)) return;
  uint4* dGU = static_cast<uint4*>(a.dGU);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    Pairs g = e4m3x8_to_pairs(c[h], sg), u = e4m3x8_to_pairs(c[2 + h], su), y;
    const Pairs d = bf16x8_to_pairs(dv[h]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 s = sigmoid2(g.v[i]), gs = mul2(g.v[i], s);
      y.v[i] = mul2(gs, u.v[i]);
      // s (1 + g (1 - s)) = s + g s (1 - s)
      const float2 slope = fma2(gs, fma2(s, make_float2(-1.f, -1.f), make_float2(1.f, 1.f)), s);
      g.v[i] = mul2(mul2(d.v[i], u.v[i]), slope);
      u.v[i] = mul2(d.v[i], gs);
    }
    dGU[p.gate + 8 * h] = pairs_to_bf16x8(g);
    dGU[p.up + 8 * h] = pairs_to_bf16x8(u);
    if (a.Y) static_cast<uint4*>(a.Y)[p.at + 8 * h] = pairs_to_bf16x8(y);
  }
}

// Rows m0 .. of batch z, as many as eight threads each make; group `grp` of each.
template <bool UE8M0>
__device__ __forceinline__ void forward_block(const SwigluFwd& a, int m0, int grp, int z) {
  const int m = m0 + (threadIdx.x >> 3);
  const int rows = valid_rows(a.masked_m, z, a.M, a.status);
  if (m0 >= rows) return;
  const Place p(z, m, grp, threadIdx.x & 7, a.M, a.I);
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

__device__ __forceinline__ void backward_block(const SwigluBwd& a, int m0, int grp, int z) {
  const int m = m0 + (threadIdx.x >> 3), kb = a.I >> 7;
  if (m >= valid_rows(a.masked_m, z, a.M, a.status)) return;
  const Place p(z, m, grp, threadIdx.x & 7, a.M, a.I);
  const uint2* CQ = static_cast<const uint2*>(a.CQ);
  const uint4* dY = static_cast<const uint4*>(a.dY);
  const uint2 c[4] = {__ldg(CQ + p.gate), __ldg(CQ + p.gate + 8), __ldg(CQ + p.up),
                      __ldg(CQ + p.up + 8)};
  const uint4 d[2] = {ld_stream_v4(dY + p.at), ld_stream_v4(dY + p.at + 8)};
  const float* cs = a.csa + static_cast<size_t>(z) * (2 * kb) * a.ld + m;
  backward_group(a, p, c, __ldg(cs + static_cast<size_t>(p.grp) * a.ld),
                 __ldg(cs + static_cast<size_t>(kb + p.grp) * a.ld), d);
}

template <bool UE8M0>
__global__ void __launch_bounds__(SG_THREADS, 4) swiglu_kernel(const SwigluFwd a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  forward_block<UE8M0>(a, blockIdx.x * 32, blockIdx.y, blockIdx.z);
}

__global__ void __launch_bounds__(SG_THREADS) swiglu_backward_kernel(const SwigluBwd a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  backward_block(a, blockIdx.x * 32, blockIdx.y, blockIdx.z);
}

// Under a limit on the SMs: one block after the other of G x I / 128 x M / 128.
template <class F>
__device__ __forceinline__ void walk_blocks(int G, int M, int I, F f) {
  const int mb = (M + SG_WALK / 8 - 1) / (SG_WALK / 8), kb = I >> 7;
  for (long long u = blockIdx.x; u < static_cast<long long>(mb) * kb * G; u += gridDim.x) {
    const long long zg = u / mb;
    f(static_cast<int>(u - zg * mb) * (SG_WALK / 8), static_cast<int>(zg % kb), static_cast<int>(zg / kb));
  }
}

template <bool UE8M0>
__global__ void __launch_bounds__(SG_WALK) swiglu_walk_kernel(const SwigluFwd a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  walk_blocks(a.G, a.M, a.I, [&](int m0, int grp, int z) { forward_block<UE8M0>(a, m0, grp, z); });
}

__global__ void __launch_bounds__(SG_WALK) swiglu_backward_walk_kernel(const SwigluBwd a) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  walk_blocks(a.G, a.M, a.I, [&](int m0, int grp, int z) { backward_block(a, m0, grp, z); });
}

// Ring form: a chunk is `rows` whole rows, of which a thread takes one lane's
// share of a group at a time.
template <bool UE8M0, int THREADS>
__global__ void __launch_bounds__(THREADS) swiglu_ring_kernel(const SwigluFwd a, int rows,
                                                              int stages) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kMaxRing];
  __shared__ uint32_t aborted, fills[kDebugRing];
  volatile uint32_t* abort_flag = &aborted;
  const int lanes = a.I >> 4, total = a.G * a.M;   // lanes per row, rows
  ChunkRing ring{{a.GU, nullptr, nullptr}, smem, full, stages, 1, rows * a.I * 4,
                 {static_cast<size_t>(total) * a.I * 4, a.status, abort_flag, fills}, a.debug_flags, 0, 0};
  auto fill = [&](int c, int s) { ring.fill(c, s, min(rows, total - c * rows) * a.I * 4); };
  const int chunks = (total + rows - 1) / rows;
  if (threadIdx.x == 0) ring.init(abort_flag);
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && blockIdx.x + s * gridDim.x < chunks; ++s)
      fill(blockIdx.x + s * gridDim.x, s);
  __syncthreads();
  // this thread's first unit of a chunk (row, lane of the row), and the next
  const int r0 = threadIdx.x / lanes, q0 = threadIdx.x - r0 * lanes;
  const int dr = THREADS / lanes, dq = THREADS - dr * lanes;
  auto advance = [&](int& r, int& q) {
    r += dr;
    q += dq;
    if (q >= lanes) { q -= lanes; ++r; }
  };
  int s = 0;
  uint32_t ph = 0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    // the warp's lanes agree (forward_group exchanges values among all 32, and a
    // wait that gives up may do so in some lanes only); after a failed wait
    // nothing more is loaded or stored
    const bool ok = __all_sync(0xffffffffu, wait_bar(smem_u32(full + s), ph, abort_flag, a) &&
                                                *abort_flag == 0 &&
                                                ring.holds(s, (c - blockIdx.x) / gridDim.x / stages + 1));
    const int n = ok ? min(rows, total - c * rows) * lanes : 0;
    const uint4* x = reinterpret_cast<const uint4*>(ring.slot(s));
    int r = r0, q = q0;
    for (int u0 = threadIdx.x & ~31; u0 < n; u0 += THREADS, advance(r, q)) {
      const int row = c * rows + r, z = a.G > 1 ? row / a.M : 0;
      const Place p(z, row - z * a.M, q >> 3, q & 7, a.M, a.I);
      const uint4* g = x + r * (a.I >> 2) + p.grp * 16 + p.lane8;
      const bool on = u0 + static_cast<int>(threadIdx.x & 31) < n;
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

dim3 grid_of(int G, int M, int I) { return dim3((M + 31) / 32, I / 128, G); }
dim3 walk_grid(int G, int M, int I, int num_sms) {
  const long long blocks = static_cast<long long>(G) * (I / 128) * ((M + SG_WALK / 8 - 1) / (SG_WALK / 8));
  return dim3(static_cast<unsigned>(std::min<long long>(num_sms, blocks)));
}

// Ring: two blocks per SM (112 registers a thread; a third block, or a ring in
// smaller chunks, was slower), chunks of about 48 KB, which are three units of
// work per thread between two barriers.  32647 rows, I = 2048: 76 us, with
// chunks of 16 KB 83 us, three blocks of 85 registers each 91 us; loads straight
// to registers 90-101 us.  (The gradient, with two thirds of the instructions
// per byte, runs at 96% of the copy rate without a ring.)
// Under a limit on the SMs one block of twice the threads and chunks.
constexpr int kRingPerSm = 2, kChunk = 49152;

template <bool UE8M0>
cudaError_t launch_fwd(const SwigluFwd& a, int num_sms, bool limited, cudaStream_t stream) {
  const long long total = static_cast<long long>(a.G) * a.M;
  const int per_sm = limited ? 1 : kRingPerSm;
  const int row = 4 * a.I, rows = std::max(1, kRingPerSm / per_sm * kChunk / row);
  const int stages = std::min(kMaxRing, ring_bytes(per_sm) / (rows * row));
  const int blocks = per_sm * num_sms;
  // whole rows only (no masked layout), and enough chunks for every block to
  // make up for the ring's 2 us of start (measured both ways, I = 256 to 4096:
  // with a checkpoint the ring is ahead from about 6 chunks per block, 46 to 41
  // us at 16384 x 2048, without one from 14, 61 to 58 us at 32647 x 2048)
  if (!a.masked_m && stages >= 2 && total < (1ll << 31) &&
      total >= (a.CQ ? 6ll : 14ll) * blocks * rows)
    return launch_dependent(limited ? swiglu_ring_kernel<UE8M0, kRingPerSm * SG_THREADS>
                                    : swiglu_ring_kernel<UE8M0, SG_THREADS>,
                            dim3(blocks), kRingPerSm / per_sm * SG_THREADS, stream, stages * rows * row, a,
                            rows, stages);
  if (limited)
    return launch_dependent(swiglu_walk_kernel<UE8M0>, walk_grid(a.G, a.M, a.I, num_sms), SG_WALK, stream, 0,
                            a);
  return launch_dependent(swiglu_kernel<UE8M0>, grid_of(a.G, a.M, a.I), SG_THREADS, stream, 0, a);
}

}  // namespace

cudaError_t swiglu_set_up() {
  constexpr int two = kRingPerSm * SG_THREADS;
  const std::pair<const void*, int> kernels[] = {
      {reinterpret_cast<const void*>(swiglu_ring_kernel<false, SG_THREADS>), kRingPerSm},
      {reinterpret_cast<const void*>(swiglu_ring_kernel<true, SG_THREADS>), kRingPerSm},
      {reinterpret_cast<const void*>(swiglu_ring_kernel<false, two>), 1},
      {reinterpret_cast<const void*>(swiglu_ring_kernel<true, two>), 1}};
  for (const auto& [k, per_sm] : kernels) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ring_bytes(per_sm));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_swiglu(const SwigluFwd& a, bool ue8m0, int num_sms, bool limited,
                          cudaStream_t stream) {
  return ue8m0 ? launch_fwd<true>(a, num_sms, limited, stream)
               : launch_fwd<false>(a, num_sms, limited, stream);
}

cudaError_t launch_swiglu_backward(const SwigluBwd& a, int num_sms, bool limited,
                                   cudaStream_t stream) {
  if (limited)
    return launch_dependent(swiglu_backward_walk_kernel, walk_grid(a.G, a.M, a.I, num_sms), SG_WALK, stream,
                            0, a);
  return launch_dependent(swiglu_backward_kernel, grid_of(a.G, a.M, a.I), SG_THREADS, stream, 0, a);
}

}  // namespace dgk
