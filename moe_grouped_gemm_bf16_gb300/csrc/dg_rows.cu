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
constexpr int SORT_CLUSTER = 8;
constexpr int SORT_BATCH = 8;   // pairs of a lane asked for at a time
constexpr int kSegment = 128;   // contiguous layout: an expert's segment in whole blocks

// Shared memory of a block: a count per warp and expert (rows of an odd length: the
// warps' counts of an expert lie in different banks); the block's count, all blocks'
// count, the block's first row and the first row of each expert; the totals of the
// scan's warps.
int sort_smem(int warps, int G) { return (warps * (G | 1) + 4 * G + 1 + 32) * 4; }

__device__ __forceinline__ int expert_of(const RowsCall& a, int pair, bool& bad) {
  const int e = __ldg(a.experts + pair);
  if (e >= a.G || e < -1) bad = true;
  return e >= 0 && e < a.G ? e : -1;
}

// The lanes with the same expert (of `bits` bits; -1: none) as the lane's own: by a
// ballot for each bit (__match_any_sync, on the SM's one unit for it, made up most of a
// sort of 16384 pairs).
__device__ __forceinline__ unsigned peers(int e, int bits) {
  unsigned m = __ballot_sync(ALL, e >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool set = (e >> b) & 1;
    const unsigned v = __ballot_sync(ALL, set);
    m &= set ? v : ~v;
  }
  return m;
}

// Inclusive sum over the warp's lanes up to each.
__device__ __forceinline__ int scan(int x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(ALL, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// One cluster sorts.  The blocks share the pairs in order, a block's warps its
// share; a warp takes 32 pairs at a time, of which each lane finds those of the same
// expert.  Two passes: each warp's counts, from which follow
// (over the warps, over the blocks, over the experts) the first row of each warp's
// pairs of each expert; then the rows themselves.
template <int LAYOUT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS)
expert_rows_kernel(const RowsCall a, int cluster, int chunk, int bits) {
  constexpr int THREADS = 32 * WARPS;
  extern __shared__ int sort_mem[];
  const int pitch = a.G | 1;
  int* count = sort_mem;                      // [warp][expert]
  int* total = count + WARPS * pitch;         // [expert], read by the cluster
  int* have = total + a.G;                    // [expert]
  int* start = have + a.G;                    // [expert]
  int* first = start + a.G;                   // [expert + 1]
  int* part = first + a.G + 1;                // [32]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  for (int i = tid; i < WARPS * pitch; i += THREADS) count[i] = 0;
  grid_dep_wait();
  grid_dep_launch_dependents();

  // `chunk` pairs a warp (a multiple of 32)
  const long long from = (static_cast<long long>(rank) * WARPS + warp) * chunk;
  const int begin = static_cast<int>(min(from, static_cast<long long>(a.pairs)));
  const int end = static_cast<int>(min(from + chunk, static_cast<long long>(a.pairs)));
  int* mine = count + warp * pitch;
  bool bad = false;
  int e[SORT_BATCH];
  unsigned same[SORT_BATCH];   // of the first batch, for the second pass
  auto ask = [&](int p) {
#pragma unroll
    for (int i = 0; i < SORT_BATCH; ++i) e[i] = p + 32 * i + lane < end ? expert_of(a, p + 32 * i + lane, bad) : -1;
  };
  ask(begin);
  __syncthreads();
  for (int p = begin; p < end; p += 32 * SORT_BATCH) {
    if (p != begin) ask(p);
#pragma unroll
    for (int i = 0; i < SORT_BATCH; ++i) {
      if (p + 32 * i >= end) break;
      same[i] = peers(e[i], bits);
      if (e[i] >= 0 && (same[i] & ((1u << lane) - 1)) == 0) mine[e[i]] += __popc(same[i]);
      __syncwarp();
    }
  }
  __syncthreads();
  // each expert's counts of the warps before (a warp an expert, a lane a warp)
  for (int x = warp; x < a.G; x += WARPS) {
    const int n = lane < WARPS ? count[lane * pitch + x] : 0;
    const int sum = scan(n);
    if (lane < WARPS) count[lane * pitch + x] = sum - n;
    if (lane == 31) total[x] = sum;
  }
  if (cluster > 1) {
    __syncwarp();
    cluster_sync();
  } else {
    __syncthreads();
  }
  // of the blocks before, and of all; then the experts' first rows
  int base = 0;   // rows of the experts up to those of this round
  for (int x0 = 0; x0 < a.G; x0 += THREADS) {
    const int x = x0 + tid;
    int before = 0, all = 0;
    if (x < a.G) {
      if (cluster > 1) {
#pragma unroll
        for (int r = 0; r < SORT_CLUSTER; ++r)
          if (r < cluster) {
            const int n = static_cast<int>(ld_cluster_u32(map_cluster(smem_u32(total + x), r)));
            if (r < rank) before += n;
            all += n;
          }
      } else {
        all = total[x];
      }
    }
    const int room = LAYOUT == kRowsContiguous ? (all + kSegment - 1) / kSegment * kSegment : all;
    int end_row = scan(room);
    if (lane == 31) part[warp] = end_row;
    __syncthreads();
    if (warp == 0) {
      const int n = lane < WARPS ? part[lane] : 0;
      const int sum = scan(n);
      if (lane < WARPS) part[lane] = sum;
    }
    __syncthreads();
    end_row += base + (warp > 0 ? part[warp - 1] : 0);
    base += part[WARPS - 1];
    if (x < a.G) {
      const int first_row = end_row - room;
      first[x] = first_row;
      have[x] = all;
      start[x] = (LAYOUT == kRowsMasked ? 0 : first_row) + before;
      if (rank == 0) {
        int n = all;
        if (LAYOUT == kRowsMasked && n > a.room) {
          raise_status(a, ST_MASK_RANGE);
          n = a.room;
        }
        if (LAYOUT == kRowsContiguous && first_row + all > a.room) raise_status(a, ST_KS_RANGE);
        if (in_bounds(a, x, 1, a.G)) a.sizes[x] = n;
      }
    }
    if (tid == 0) first[a.G] = base;   // (the last round's)
    __syncthreads();
  }
  // This block has used all that it read of its peers; none leaves before they all
  // have (a relaxed arrival: there is nothing to publish, and a release would wait for
  // the stores below).
  if (cluster > 1) cluster_arrive_relaxed();
  for (int p = begin; p < end; p += 32 * SORT_BATCH) {
    const bool again = chunk > 32 * SORT_BATCH;
    if (again) ask(p);
#pragma unroll
    for (int i = 0; i < SORT_BATCH; ++i) {
      const int at = p + 32 * i + lane;
      if (p + 32 * i >= end) break;
      const int x = e[i];
      const unsigned all_same = again ? peers(x, bits) : same[i], less = all_same & ((1u << lane) - 1);
      int row = -1;
      if (x >= 0) row = start[x] + mine[x] + __popc(less);
      __syncwarp();
      if (x >= 0 && less == 0) mine[x] += __popc(all_same);
      __syncwarp();
      if (LAYOUT != kRowsRagged && row >= a.room) row = -1;
      if (LAYOUT == kRowsContiguous && row >= 0 && in_bounds(a, row, 1, a.room)) a.m_indices[row] = x;
      if (LAYOUT == kRowsMasked && row >= 0) row += x * a.room;
      if (at < end && in_bounds(a, at, 1, a.pairs)) a.rows[at] = row;
    }
  }
  if (bad) raise_status(a, ST_EXPERT_RANGE);
  if (LAYOUT == kRowsContiguous) {
    // -1 behind each expert's rows (a warp an expert), and behind the last expert
    for (int x = rank * WARPS + warp; x < a.G; x += cluster * WARPS)
      for (int r = first[x] + have[x] + lane; r < min(first[x + 1], a.room); r += 32)
        if (in_bounds(a, r, 1, a.room)) a.m_indices[r] = -1;
    for (long long r = static_cast<long long>(first[a.G]) + rank * THREADS + tid; r < a.room;
         r += cluster * THREADS)
      if (in_bounds(a, r, 1, a.room)) a.m_indices[r] = -1;
  }
  if (cluster > 1) cluster_wait();
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
          if (v0 + 32 * i < a.vecs && in_bounds(a, static_cast<size_t>(r) * a.vecs + v0 + 32 * i, 1,
                                                static_cast<size_t>(a.num_rows) * a.vecs))
            dst[32 * i] = x[i];
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
          if (g0 + i < a.kb && in_bounds(a, m, 1, a.ld_out) && in_bounds(a, z, 1, a.num_rows / a.per))
            dst[static_cast<size_t>(i) * a.ld_out] = s[i];
      }
    }
  }
}

// ---------------------------------------------------------- weighted sum ----
// (blocks per SM: with 2, 3 and 4, 4096 tokens of 8 rows of 7168 take 127, 102 and 107 us,
// their gradient 209, 174 and 192.  Of 80 registers a thread some spill, 28 to 84 bytes, in
// every instance but those of 8 rows at a time in combine and in its gradient by warps.)
constexpr int SUM_THREADS = kSumThreads, SUM_PER_SM = kSumPerSm;
// 16-byte vectors that a thread has in flight: of ROWS rows, VECS of each.  Few choices
// take more of each row (3393 tokens of one row of 5016: 35 us with one vector of it).
constexpr int SUM_LOADS = kSumLoads;

// A warp takes 256 VECS columns of a token, a lane eight of each 256, of all its rows:
// products and sum in fp32 in the order of the choices, the residual added first.
// The next token's rows and weights are on their way meanwhile.
template <int ROWS>
__global__ void __launch_bounds__(SUM_THREADS, SUM_PER_SM)
combine_kernel(const CombineCall a) {
  constexpr int VECS = SUM_LOADS / ROWS;
  const int lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int vecs = a.K >> 3, pieces = (vecs + 32 * VECS - 1) / (32 * VECS);
  const uint4* Y = static_cast<const uint4*>(a.Y);
  const unsigned warps = gridDim.x * (SUM_THREADS / 32), w0 = blockIdx.x * (SUM_THREADS / 32) + (threadIdx.x >> 5);
  // (the warp's first unit, and the step from one to the next, without a division each)
  int t = w0 / pieces, piece = w0 - t * pieces;
  const int step_t = warps / pieces, step_p = warps - step_t * pieces;
  int mine = -1;
  float weight = 0.f;
  auto ask = [&](int t, int& mine, float& weight) {
    const size_t pair = static_cast<size_t>(t) * a.k + lane;
    const bool on = t < a.T && lane < a.k;
    mine = row_of(a.rows, pair, on, a.num_rows, a.status);
    weight = !on ? 0.f : a.weights ? __ldg(a.weights + pair) : 1.f;
    if (mine < 0) weight = 0.f;
  };
  ask(t, mine, weight);
  while (t < a.T) {
    const int v = piece * (32 * VECS) + lane;
    const size_t at = static_cast<size_t>(t) * vecs + v;
    uint4 r[VECS];
#pragma unroll
    for (int h = 0; h < VECS; ++h) {
      r[h] = make_uint4(0, 0, 0, 0);
      if (a.R && v + 32 * h < vecs) r[h] = static_cast<const uint4*>(a.R)[at + 32 * h];   // (may be `out`)
    }
    t += step_t;
    piece += step_p;
    if (piece >= pieces) {
      piece -= pieces;
      ++t;
    }
    int next_row;
    float next_weight;
    ask(t, next_row, next_weight);
    float sum[VECS][8];
#pragma unroll
    for (int h = 0; h < VECS; ++h) bf16x8_to_float(r[h], sum[h]);
    for (int j0 = 0; j0 < a.k; j0 += ROWS) {
      uint4 y[ROWS][VECS];
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const int row = __shfl_sync(ALL, mine, (j0 + j) & 31);
#pragma unroll
        for (int h = 0; h < VECS; ++h) {
          y[j][h] = make_uint4(0, 0, 0, 0);
          if (j0 + j < a.k && row >= 0 && v + 32 * h < vecs)
            y[j][h] = ld_stream_v4(Y + static_cast<size_t>(row) * vecs + v + 32 * h);
        }
      }
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const float w = __shfl_sync(ALL, weight, (j0 + j) & 31);
        // (a choice without a row adds nothing, also to an infinite sum)
        if (j0 + j < a.k)
#pragma unroll
          for (int h = 0; h < VECS; ++h) {
            float x[8];
            bf16x8_to_float(y[j][h], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[h][i] = fmaf(w, x[i], sum[h][i]);
          }
      }
    }
#pragma unroll
    for (int h = 0; h < VECS; ++h)
      if (v + 32 * h < vecs && in_bounds(a, at + 32 * h, 1, static_cast<size_t>(a.T) * vecs))
        static_cast<uint4*>(a.out)[at + 32 * h] = float_to_bf16x8(sum[h]);
    mine = next_row;
    weight = next_weight;
  }
}

// A team of threads (32 to 256) takes a token: a thread eight columns at a time (VECS
// times) of the gradient and of all its rows; the dot products are summed over the team
// in a fixed order.
template <int TEAM, int ROWS>
__global__ void __launch_bounds__(SUM_THREADS, SUM_PER_SM)
combine_backward_kernel(const CombineBwd a) {
  constexpr int TEAMS = SUM_THREADS / TEAM, VECS = SUM_LOADS / ROWS;
  __shared__ float part[ROWS][SUM_THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, member = threadIdx.x % TEAM;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int vecs = a.K >> 3;
  const uint4* Y = static_cast<const uint4*>(a.Y);
  uint4* dY = static_cast<uint4*>(a.dY);
  const long long step = static_cast<long long>(gridDim.x) * TEAMS;
  int next_row = -1;
  float next_weight = 0.f;
  auto ask = [&](long long t) {
    const size_t pair = static_cast<size_t>(t) * a.k + lane;
    const bool on = t < a.T && lane < a.k;
    next_row = row_of(a.rows, pair, on, a.num_rows, a.status);
    next_weight = !on ? 0.f : a.weights ? __ldg(a.weights + pair) : 1.f;
  };
  long long t = static_cast<long long>(blockIdx.x) * TEAMS + threadIdx.x / TEAM;
  ask(t);
  for (; t < a.T; t += step) {
    const uint4* dO = static_cast<const uint4*>(a.dO) + static_cast<size_t>(t) * vecs;
    const int mine = next_row;
    const float weight = mine < 0 ? 0.f : next_weight;
    ask(t + step);   // (on its way meanwhile)
    for (int j0 = 0; j0 < a.k; j0 += ROWS) {
      float dot[ROWS] = {};
      // (the bound a whole number of warps: the shuffles below)
      for (int v = member; v < (vecs + 31) / 32 * 32; v += TEAM * VECS) {
        uint4 d[VECS], y[ROWS][VECS];
#pragma unroll
        for (int h = 0; h < VECS; ++h) {
          d[h] = make_uint4(0, 0, 0, 0);
          if (v + h * TEAM < vecs) d[h] = __ldg(dO + v + h * TEAM);
        }
        if (a.dw) {
#pragma unroll
          for (int j = 0; j < ROWS; ++j) {
            const int row = __shfl_sync(ALL, mine, (j0 + j) & 31);
#pragma unroll
            for (int h = 0; h < VECS; ++h) {
              y[j][h] = make_uint4(0, 0, 0, 0);
              if (j0 + j < a.k && row >= 0 && v + h * TEAM < vecs)
                y[j][h] = ld_stream_v4(Y + static_cast<size_t>(row) * vecs + v + h * TEAM);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < VECS; ++h) {
          float g[8];
          bf16x8_to_float(d[h], g);
#pragma unroll
          for (int j = 0; j < ROWS; ++j) {
            const int row = __shfl_sync(ALL, mine, (j0 + j) & 31);
            const float w = __shfl_sync(ALL, weight, (j0 + j) & 31);
            if (a.dw) {
              float x[8];
              bf16x8_to_float(y[j][h], x);
#pragma unroll
              for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], x[i], dot[j]);
            }
            const size_t at = static_cast<size_t>(max(row, 0)) * vecs + v + h * TEAM;
            if (j0 + j < a.k && row >= 0 && v + h * TEAM < vecs &&
                in_bounds(a, at, 1, static_cast<size_t>(a.num_rows) * vecs)) {
              float x[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = w * g[i];
              dY[at] = float_to_bf16x8(x);
            }
          }
        }
      }
      if (a.dw) {
        // lane j of each warp: the warp's sum of row j
        float mine_dot = 0.f;
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) dot[j] += __shfl_xor_sync(ALL, dot[j], o);
          if (lane == j) mine_dot = dot[j];
        }
        const int j = j0 + lane;
        const int row = __shfl_sync(ALL, mine, j & 31);
        if (TEAM > 32) {
          const int team = threadIdx.x / TEAM;
          if (lane < ROWS) part[lane][warp] = mine_dot;
          named_bar_sync(1 + team, TEAM);
          mine_dot = 0.f;
          if (lane < ROWS)
#pragma unroll
            for (int w = 0; w < TEAM / 32; ++w) mine_dot += part[lane][team * (TEAM / 32) + w];
          named_bar_sync(1 + team, TEAM);
        }
        if (lane < ROWS && j < a.k && member < 32 &&
            in_bounds(a, static_cast<size_t>(t) * a.k + j, 1, static_cast<size_t>(a.T) * a.k))
          a.dw[static_cast<size_t>(t) * a.k + j] = row >= 0 ? mine_dot : 0.f;
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
  auto opt_in = [](auto kernel, int warps) {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                sort_smem(warps, kRowsMaxExperts));
  };
  const cudaError_t set[] = {
      opt_in(expert_rows_kernel<kRowsRagged, 8>, 8),      opt_in(expert_rows_kernel<kRowsRagged, 32>, 32),
      opt_in(expert_rows_kernel<kRowsContiguous, 8>, 8),  opt_in(expert_rows_kernel<kRowsContiguous, 32>, 32),
      opt_in(expert_rows_kernel<kRowsMasked, 8>, 8),      opt_in(expert_rows_kernel<kRowsMasked, 32>, 32)};
  for (const cudaError_t e : set)
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

cudaError_t launch_rows(const RowsCall& a, RowsLayout layout, int num_sms, cudaStream_t stream) {
  // a block for every 2048 pairs (16384 pairs of 32 experts with their rows of 7168 in 8
  // bits: 36.6 us so and with 1024, 38.7 with 4096, 42.2 with 8192)
  int cluster = 1;
  // and for every 4096 rows to mark (28 choices of 184 experts, 23552 rows: 10.2 us with one
  // block, dispatch included, 8.5 with eight)
  const int room = layout == kRowsContiguous ? a.room : 0;
  while (cluster < SORT_CLUSTER && 2 * cluster <= num_sms && (a.pairs > 2048 * cluster || room > 4096 * cluster))
    cluster *= 2;
  const int warps = a.pairs <= 1024 ? 8 : 32, per = warps * cluster;
  const int chunk = ((a.pairs + per - 1) / per + 31) / 32 * 32;
  int bits = 1;
  while ((1 << bits) < a.G) ++bits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster, 1, 1);
  cfg.blockDim = dim3(32 * warps, 1, 1);
  cfg.dynamicSmemBytes = sort_smem(warps, a.G);
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
  auto go = [&](auto few, auto many) { return cudaLaunchKernelEx(&cfg, warps == 8 ? few : many, a, cluster, chunk, bits); };
  switch (layout) {
    case kRowsRagged: return go(expert_rows_kernel<kRowsRagged, 8>, expert_rows_kernel<kRowsRagged, 32>);
    case kRowsContiguous:
      return go(expert_rows_kernel<kRowsContiguous, 8>, expert_rows_kernel<kRowsContiguous, 32>);
    default: return go(expert_rows_kernel<kRowsMasked, 8>, expert_rows_kernel<kRowsMasked, 32>);
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
  const int rows = a.k <= 2 ? 2 : a.k <= 4 ? 4 : 8, wide = 32 * SUM_LOADS / rows;
  const long long units = static_cast<long long>(a.T) * (((a.K >> 3) + wide - 1) / wide);
  const dim3 grid(move_grid(units, SUM_THREADS / 32, SUM_PER_SM, num_sms, limited));
  return launch_dependent(rows == 2 ? combine_kernel<2> : rows == 4 ? combine_kernel<4> : combine_kernel<8>, grid,
                          SUM_THREADS, stream, 0, a);
}

cudaError_t launch_combine_backward(const CombineBwd& a, int num_sms, int device_sms,
                                    cudaStream_t stream) {
  const int rows = a.k <= 2 ? 2 : a.k <= 4 ? 4 : 8;
  const int team = combine_team(a.T, a.K >> 3, a.k, rows, device_sms);
  const dim3 grid(move_grid(a.T, SUM_THREADS / team, SUM_PER_SM, num_sms, num_sms < device_sms));
  auto go = [&](auto two, auto four, auto eight) {
    return launch_dependent(rows == 2 ? two : rows == 4 ? four : eight, grid, SUM_THREADS, stream, 0, a);
  };
  return team == 32    ? go(combine_backward_kernel<32, 2>, combine_backward_kernel<32, 4>, combine_backward_kernel<32, 8>)
         : team == 64  ? go(combine_backward_kernel<64, 2>, combine_backward_kernel<64, 4>, combine_backward_kernel<64, 8>)
         : team == 128 ? go(combine_backward_kernel<128, 2>, combine_backward_kernel<128, 4>, combine_backward_kernel<128, 8>)
                       : go(combine_backward_kernel<256, 2>, combine_backward_kernel<256, 4>, combine_backward_kernel<256, 8>);
}

}  // namespace dgk
