// Rows between tokens and experts: where each (token, choice) pair's row lies in
// the experts' operands, the rows copied there, and the weighted sum back.
//
//   rows[t][j]   a stable counting sort of the pairs by their expert, in one of the
//                grouped products' layouts
//   D[rows[t][j]] = X[t]                         (with the 1x128 scales of 8-bit rows)
//   out[t] = R[t] + sum_j w[t][j] Y[rows[t][j]]  (w = 1, no R: the gradient of the
//                                                 copy above)
//   dY[rows[t][j]] = w[t][j] dO[t];  dw[t][j] = <dO[t], Y[rows[t][j]]>
//
// The copies and sums are memory-bound; the sort is bound by latency.
#include <algorithm>

#include "dg_fp8.cuh"
#include "dg_launch.h"
#include "dg_rows.h"
#include "dg_wait.cuh"
#include "ptx.cuh"

namespace dgk {
namespace {

constexpr unsigned ALL = 0xffffffffu;

// ------------------------------------------------------------ the sort ----
constexpr int SORT_THREADS = 1024, SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_CLUSTER = 8;
constexpr int kSegment = 128;   // contiguous layout: an expert's segment in whole blocks

// Shared memory of a block: a count per warp and expert; the block's count, all
// blocks' count and the first row of each expert; the totals of the scan's warps.
int sort_smem(int G) { return (SORT_WARPS * G + 3 * G + 1 + 32) * 4; }

__device__ __forceinline__ int expert_of(const RowsCall& a, int pair, bool& bad) {
  const int e = __ldg(a.experts + pair);
  if (e >= a.G || e < -1) bad = true;
  return e >= 0 && e < a.G ? e : -1;
}

// One cluster sorts.  The blocks share the pairs in order, a block's warps its
// share; a warp takes 32 pairs at a time, where __match_any gives each lane the
// lanes of the same expert.  Two passes: each warp's counts, from which follow
// (over the warps, over the blocks, over the experts) the first row of each warp's
// pairs of each expert; then the rows themselves.
template <int LAYOUT>
__global__ void __launch_bounds__(SORT_THREADS)
expert_rows_kernel(const RowsCall a, int cluster, int chunk) {
  extern __shared__ int sort_mem[];
  int* count = sort_mem;                      // [warp][expert]
  int* total = count + SORT_WARPS * a.G;      // [expert], read by the cluster
  int* have = total + a.G;                    // [expert]
  int* first = have + a.G;                    // [expert + 1]
  int* part = first + a.G + 1;                // [32]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  for (int i = tid; i < SORT_WARPS * a.G; i += SORT_THREADS) count[i] = 0;
  grid_dep_wait();
  grid_dep_launch_dependents();
  __syncthreads();

  // `chunk` pairs a warp (a multiple of 32)
  const long long from = (static_cast<long long>(rank) * SORT_WARPS + warp) * chunk;
  const int begin = static_cast<int>(min(from, static_cast<long long>(a.pairs)));
  const int end = static_cast<int>(min(from + chunk, static_cast<long long>(a.pairs)));
  int* mine = count + warp * a.G;
  bool bad = false;
  for (int p = begin; p < end; p += 32) {
    const int e = p + lane < end ? expert_of(a, p + lane, bad) : -1;
    const unsigned same = __match_any_sync(ALL, e);
    if (e >= 0 && (same & ((1u << lane) - 1)) == 0) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // counts of the warps before, of the block, of the blocks before, of all
  int sum = 0, before = 0, all = 0;
  if (tid < a.G) {
#pragma unroll 8
    for (int w = 0; w < SORT_WARPS; ++w) {
      const int n = count[w * a.G + tid];
      count[w * a.G + tid] = sum;
      sum += n;
    }
    total[tid] = sum;
  }
  if (cluster > 1) {
    cluster_sync();
    if (tid < a.G)
#pragma unroll
      for (int r = 0; r < SORT_CLUSTER; ++r)
        if (r < cluster) {
          const int n = static_cast<int>(ld_cluster_u32(map_cluster(smem_u32(total + tid), r)));
          if (r < rank) before += n;
          all += n;
        }
  } else {
    all = sum;
  }
  // first rows: a scan over the experts
  int room = LAYOUT == kRowsContiguous ? (all + kSegment - 1) / kSegment * kSegment : all;
  int x = room;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(ALL, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(ALL, y, o);
      if (lane >= o) y += z;
    }
    part[lane] = y;
  }
  __syncthreads();
  x += warp > 0 ? part[warp - 1] : 0;
  if (tid < a.G) {
    first[tid + 1] = x;
    if (tid == 0) first[0] = 0;
    have[tid] = all;
    const int start = (LAYOUT == kRowsMasked ? 0 : x - room) + before;
#pragma unroll 8
    for (int w = 0; w < SORT_WARPS; ++w) count[w * a.G + tid] += start;
    if (rank == 0) {
      int n = all;
      if (LAYOUT == kRowsMasked && n > a.room) {
        raise_status(a, ST_MASK_RANGE);
        n = a.room;
      }
      if (LAYOUT == kRowsContiguous && x - room + all > a.room) raise_status(a, ST_KS_RANGE);
      a.sizes[tid] = n;
    }
  }
  __syncthreads();
  for (int p = begin; p < end; p += 32) {
    const bool on = p + lane < end;
    const int e = on ? expert_of(a, p + lane, bad) : -1;
    const unsigned same = __match_any_sync(ALL, e);
    int row = -1;
    if (e >= 0) row = mine[e] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (e >= 0 && (same & ((1u << lane) - 1)) == 0) mine[e] += __popc(same);
    __syncwarp();
    if (LAYOUT != kRowsRagged && row >= a.room) row = -1;
    if (LAYOUT == kRowsMasked && row >= 0) row += e * a.room;
    if (on) a.rows[p + lane] = row;
  }
  if (bad) raise_status(a, ST_EXPERT_RANGE);
  if (LAYOUT == kRowsContiguous) {
    // the expert of each row: the last that starts at or before it, where it has
    // that many rows
    for (long long r = rank * SORT_THREADS + tid; r < a.room; r += cluster * SORT_THREADS) {
      int lo = 0, hi = a.G;   // first[lo] <= r < first[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= r) lo = mid;
        else hi = mid;
      }
      a.m_indices[r] = r - first[lo] < have[lo] ? lo : -1;
    }
  }
  // (a peer may still read this block's counts)
  __syncwarp();
  if (cluster > 1) cluster_sync();
}

// ------------------------------------------------------- rows of experts ----
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_VECS = 4;      // 16-byte vectors of a lane: 2 KB of a row a warp

// The row of a lane's choice; one outside the operand is left out and reported.
__device__ __forceinline__ int row_of(const int32_t* rows, size_t at, bool on, int num_rows,
                                      unsigned int* status) {
  const int r = on ? __ldg(rows + at) : -1;
  if (r >= num_rows || r < -1) atomicCAS(status, 0u, ST_EXPERT_RANGE);
  return r >= 0 && r < num_rows ? r : -1;
}

// A warp takes 2 KB of a token's row, read once, and stores it into the rows of all
// its choices.  The scales are a second kind of work: a warp takes 32 tokens (a
// lane each) of 8 groups; what it stores lies in 4-byte pieces that fill whole
// sectors in L2 with those of the expert's other tokens.
__global__ void __launch_bounds__(MOVE_THREADS)
dispatch_kernel(const DispatchCall a) {
  constexpr int GROUPS = 8;
  const int lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int pieces = (a.vecs + 32 * MOVE_VECS - 1) / (32 * MOVE_VECS);
  const long long moves = static_cast<long long>(a.T) * pieces;
  const int bands = (a.T + 31) / 32, steps = a.sa ? (a.kb + GROUPS - 1) / GROUPS : 0;
  const long long units = moves + static_cast<long long>(bands) * steps;
  const uint4* X = static_cast<const uint4*>(a.X);
  uint4* D = static_cast<uint4*>(a.D);
  const long long stride = static_cast<long long>(gridDim.x) * (MOVE_THREADS / 32);
  for (long long u = static_cast<long long>(blockIdx.x) * (MOVE_THREADS / 32) + (threadIdx.x >> 5);
       u < units; u += stride) {
    if (u < moves) {
      const int t = static_cast<int>(u / pieces);
      const int v0 = static_cast<int>(u - static_cast<long long>(t) * pieces) * (32 * MOVE_VECS) + lane;
      uint4 x[MOVE_VECS];
      const uint4* src = X + static_cast<size_t>(t) * a.vecs + v0;
#pragma unroll
      for (int i = 0; i < MOVE_VECS; ++i)
        if (v0 + 32 * i < a.vecs) x[i] = ld_stream_v4(src + 32 * i);
      const int mine = row_of(a.rows, static_cast<size_t>(t) * a.k + lane, lane < a.k, a.num_rows, a.status);
      for (int j = 0; j < a.k; ++j) {
        const int r = __shfl_sync(ALL, mine, j);
        if (r < 0) continue;
        uint4* dst = D + static_cast<size_t>(r) * a.vecs + v0;
#pragma unroll
        for (int i = 0; i < MOVE_VECS; ++i)
          if (v0 + 32 * i < a.vecs) dst[32 * i] = x[i];
      }
    } else {
      const long long w = u - moves;
      const int band = static_cast<int>(w / steps), g0 = static_cast<int>(w - static_cast<long long>(band) * steps) * GROUPS;
      const int t = band * 32 + lane;
      if (t >= a.T) continue;   // (no exchange between the lanes below)
      uint32_t s[GROUPS];
#pragma unroll
      for (int i = 0; i < GROUPS; ++i)
        if (g0 + i < a.kb) s[i] = __ldg(a.sa + static_cast<size_t>(g0 + i) * a.ld + t);
      for (int j = 0; j < a.k; ++j) {
        const int r = row_of(a.rows, static_cast<size_t>(t) * a.k + j, true, a.num_rows, a.status);
        if (r < 0) continue;
        const int z = r / a.per, m = r - z * a.per;
        uint32_t* dst = a.sa_out + (static_cast<size_t>(z) * a.kb + g0) * a.ld_out + m;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i)
          if (g0 + i < a.kb) dst[static_cast<size_t>(i) * a.ld_out] = s[i];
      }
    }
  }
}

// ---------------------------------------------------------- weighted sum ----
constexpr int SUM_THREADS = 256;
constexpr int SUM_ROWS = 8;   // rows of a token in flight at a time

// A warp takes 256 columns of a token, a lane eight of them, of all its rows:
// products and sum in fp32 in the order of the choices, the residual added first.
__global__ void __launch_bounds__(SUM_THREADS)
combine_kernel(const CombineCall a) {
  const int lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int vecs = a.K >> 3, pieces = (vecs + 31) / 32;
  const long long units = static_cast<long long>(a.T) * pieces;
  const uint4* Y = static_cast<const uint4*>(a.Y);
  const long long stride = static_cast<long long>(gridDim.x) * (SUM_THREADS / 32);
  for (long long u = static_cast<long long>(blockIdx.x) * (SUM_THREADS / 32) + (threadIdx.x >> 5);
       u < units; u += stride) {
    const int t = static_cast<int>(u / pieces);
    const int v = static_cast<int>(u - static_cast<long long>(t) * pieces) * 32 + lane;
    const bool on = v < vecs;
    const size_t at = static_cast<size_t>(t) * vecs + v;
    uint4 r = make_uint4(0, 0, 0, 0);
    if (a.R && on) r = static_cast<const uint4*>(a.R)[at];   // (may be `out`)
    const size_t pair = static_cast<size_t>(t) * a.k + lane;
    const int mine = row_of(a.rows, pair, lane < a.k, a.num_rows, a.status);
    const float weight = mine < 0 ? 0.f : a.weights ? __ldg(a.weights + pair) : 1.f;
    float sum[8];
    bf16x8_to_float(r, sum);
    for (int j0 = 0; j0 < a.k; j0 += SUM_ROWS) {
      uint4 y[SUM_ROWS];
#pragma unroll
      for (int j = 0; j < SUM_ROWS; ++j) {
        const int row = __shfl_sync(ALL, mine, (j0 + j) & 31);
        y[j] = make_uint4(0, 0, 0, 0);
        if (j0 + j < a.k && row >= 0 && on) y[j] = ld_stream_v4(Y + static_cast<size_t>(row) * vecs + v);
      }
#pragma unroll
      for (int j = 0; j < SUM_ROWS; ++j) {
        const float w = __shfl_sync(ALL, weight, (j0 + j) & 31);
        float x[8];
        bf16x8_to_float(y[j], x);
        // (a choice without a row adds nothing, also to an infinite sum)
        if (j0 + j < a.k)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = fmaf(w, x[i], sum[i]);
      }
    }
    if (on) static_cast<uint4*>(a.out)[at] = float_to_bf16x8(sum);
  }
}

// A block takes a token: a thread eight columns at a time of the gradient and of
// all its rows; the dot products are summed over the block in a fixed order.
template <int THREADS>
__global__ void __launch_bounds__(THREADS)
combine_backward_kernel(const CombineBwd a) {
  __shared__ float part[SUM_ROWS][THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int vecs = a.K >> 3;
  const uint4* Y = static_cast<const uint4*>(a.Y);
  uint4* dY = static_cast<uint4*>(a.dY);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const uint4* dO = static_cast<const uint4*>(a.dO) + static_cast<size_t>(t) * vecs;
    const size_t pair = static_cast<size_t>(t) * a.k + lane;
    const int mine = row_of(a.rows, pair, lane < a.k, a.num_rows, a.status);
    const float weight = mine < 0 ? 0.f : a.weights ? __ldg(a.weights + pair) : 1.f;
    for (int j0 = 0; j0 < a.k; j0 += SUM_ROWS) {
      float dot[SUM_ROWS] = {};
      for (int v = threadIdx.x; v < (vecs + 31) / 32 * 32; v += THREADS) {
        const bool on = v < vecs;
        uint4 d = make_uint4(0, 0, 0, 0);
        if (on) d = __ldg(dO + v);
        uint4 y[SUM_ROWS];
        if (a.dw) {
#pragma unroll
          for (int j = 0; j < SUM_ROWS; ++j) {
            const int row = __shfl_sync(ALL, mine, (j0 + j) & 31);
            y[j] = make_uint4(0, 0, 0, 0);
            if (j0 + j < a.k && row >= 0 && on) y[j] = ld_stream_v4(Y + static_cast<size_t>(row) * vecs + v);
          }
        }
        float g[8];
        bf16x8_to_float(d, g);
#pragma unroll
        for (int j = 0; j < SUM_ROWS; ++j) {
          const int row = __shfl_sync(ALL, mine, (j0 + j) & 31);
          const float w = __shfl_sync(ALL, weight, (j0 + j) & 31);
          if (a.dw) {
            float x[8];
            bf16x8_to_float(y[j], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], x[i], dot[j]);
          }
          if (j0 + j < a.k && row >= 0 && on) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = w * g[i];
            dY[static_cast<size_t>(row) * vecs + v] = float_to_bf16x8(x);
          }
        }
      }
      if (a.dw) {
#pragma unroll
        for (int j = 0; j < SUM_ROWS; ++j) {
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) dot[j] += __shfl_xor_sync(ALL, dot[j], o);
          if (lane == 0) part[j][warp] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < SUM_ROWS && j0 + static_cast<int>(threadIdx.x) < a.k) {
          float s = 0.f;
#pragma unroll
          for (int w = 0; w < THREADS / 32; ++w) s += part[threadIdx.x][w];
          const size_t at = static_cast<size_t>(t) * a.k + j0 + threadIdx.x;
          const int row = __ldg(a.rows + at);
          a.dw[at] = row >= 0 && row < a.num_rows ? s : 0.f;
        }
        __syncthreads();
      }
    }
  }
}

int move_grid(long long units, int per_block, int per_sm, int num_sms, bool limited) {
  const long long blocks = (units + per_block - 1) / per_block;
  return static_cast<int>(std::max(1ll, std::min<long long>(blocks, limited ? num_sms : per_sm * num_sms)));
}

}  // namespace

cudaError_t rows_set_up() {
  const void* kernels[] = {reinterpret_cast<const void*>(expert_rows_kernel<kRowsRagged>),
                           reinterpret_cast<const void*>(expert_rows_kernel<kRowsContiguous>),
                           reinterpret_cast<const void*>(expert_rows_kernel<kRowsMasked>)};
  for (const void* k : kernels) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               sort_smem(kRowsMaxExperts));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_rows(const RowsCall& a, RowsLayout layout, int num_sms, cudaStream_t stream) {
  // a block sorts 4096 pairs in less time than a second one takes to join
  int cluster = 1;
  while (cluster < SORT_CLUSTER && 2 * cluster <= num_sms && a.pairs > 4096 * cluster) cluster *= 2;
  const int per = SORT_WARPS * cluster;
  const int chunk = ((a.pairs + per - 1) / per + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster, 1, 1);
  cfg.blockDim = dim3(SORT_THREADS, 1, 1);
  cfg.dynamicSmemBytes = sort_smem(a.G);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  switch (layout) {
    case kRowsRagged: return cudaLaunchKernelEx(&cfg, expert_rows_kernel<kRowsRagged>, a, cluster, chunk);
    case kRowsContiguous:
      return cudaLaunchKernelEx(&cfg, expert_rows_kernel<kRowsContiguous>, a, cluster, chunk);
    default: return cudaLaunchKernelEx(&cfg, expert_rows_kernel<kRowsMasked>, a, cluster, chunk);
  }
}

cudaError_t launch_dispatch(const DispatchCall& a, int num_sms, bool limited, cudaStream_t stream) {
  const int pieces = (a.vecs + 32 * MOVE_VECS - 1) / (32 * MOVE_VECS);
  const long long units = static_cast<long long>(a.T) * pieces +
                          (a.sa ? static_cast<long long>((a.T + 31) / 32) * ((a.kb + 7) / 8) : 0);
  return launch_dependent(dispatch_kernel, dim3(move_grid(units, MOVE_THREADS / 32, 8, num_sms, limited)),
                          MOVE_THREADS, stream, 0, a);
}

cudaError_t launch_combine(const CombineCall& a, int num_sms, bool limited, cudaStream_t stream) {
  const long long units = static_cast<long long>(a.T) * (((a.K >> 3) + 31) / 32);
  return launch_dependent(combine_kernel, dim3(move_grid(units, SUM_THREADS / 32, 8, num_sms, limited)),
                          SUM_THREADS, stream, 0, a);
}

cudaError_t launch_combine_backward(const CombineBwd& a, int num_sms, bool limited,
                                    cudaStream_t stream) {
  return launch_dependent(combine_backward_kernel<256>, dim3(move_grid(a.T, 1, 8, num_sms, limited)), 256,
                          stream, 0, a);
}

}  // namespace dgk
