// The ragged bf16 products (dg_bf16.cu) of a few rows in all: a decoding step's
// tokens, where the tensor cores have next to nothing to do and their kernel's
// start (tensor memory, tensor maps, a ring's first loads) and a split
// reduction's cluster barriers take longer than reading the weights does.
//
//   nt  D[t][n]    = sum_k A[t][k] B[e][n][k]
//   nn  D[t][n]    = sum_k A[t][k] B[e][k][n]
//   tn  D[e][m][n] = C[e][m][n] + sum_{t in e} A[t][m] B[t][n]
//
// Plain loads of 16 bytes straight to registers, fp32 products in pairs, the
// sums joined in a fixed order by shuffles and through shared memory.  What
// bounds them is one round of loads and the launch; a block therefore takes so
// little that its loads are all in flight at once, or nearly.  A block of nt and
// nn has one group's weights, up to FEW_ROWS rows at a time (a group of more reads
// them again, out of L2); of tn one tile of a group's D.
//
// Measured (us; the tensor cores' kernel takes): nt 1 row, 920 x 1352 3.3 (7.6),
// nn 2 rows in two groups, 312 x 1320 3.2 (9.7), 5 rows in 7 groups, 3808 x 5672 34
// (38; 6.4 TB/s), tn 3 rows in 44 groups, 696 x 7856 71 (77; the copy rate).  A
// launch alone is 2.2.
#include <algorithm>

#include "dg_bf16.h"
#include "dg_fp8.cuh"
#include "dg_launch.h"
#include "dg_params.h"
#include "dg_wait.cuh"
#include "ptx.cuh"

namespace dgk {
namespace {

constexpr int FEW_ROWS = 4;
// nt: columns of D per warp; three blocks per SM (80 registers; without the limit
// 134 and one block, 2 rows of 4760 x 5480: 27.5 us, so 21.7)
constexpr int NT_THREADS = 256, NT_COLS = 4, NT_PER_SM = 3;
constexpr int NN_THREADS = 512;                // two blocks per SM, for the same reason
constexpr int TN_THREADS = 256, TN_M = 8;      // tn: rows of D per warp, 256 columns

struct FewParams {
  const uint16_t* A;
  const uint16_t* B;
  const uint16_t* C;
  uint16_t* D;
  const int32_t* sizes;
  int G, rows, M, N, K;
  unsigned int* status;
};

struct FewGroup {
  int g, first, n;   // group, its first row, its rows (0: there is none)
};

// The z-th group that has rows or, with ANY, group z; the whole warp calls.  A
// negative size counts as zero and the running total stops at `rows`; `report`:
// this block looks at every group for either.
template <bool ANY>
__device__ __forceinline__ FewGroup few_group(const FewParams& p, int z, bool report) {
  const int lane = threadIdx.x & 31;
  FewGroup f{0, 0, 0};
  bool bad = false, found = false;
  int row = 0, seen = 0;
  for (int base = 0; base < p.G && (report || !found); base += 32) {
    const int given = base + lane < p.G ? __ldg(p.sizes + base + lane) : 0;
    const int v = min(max(given, 0), p.rows);   // (rows is small: 32 of them fit 32 bits)
    int end = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    end += row;
    bad = bad || v != given || end > p.rows;
    end = min(end, p.rows);
    int from = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) from = row;
    const uint32_t have = ANY ? 0xffffffffu : __ballot_sync(0xffffffffu, end > from);
    const bool mine = (ANY || end > from) && seen + __popc(have & ((1u << lane) - 1)) == z;
    const uint32_t at = __ballot_sync(0xffffffffu, mine);
    if (at) {
      const int src = __ffs(at) - 1;
      found = true;
      f.g = base + src;
      f.first = __shfl_sync(0xffffffffu, from, src);
      f.n = __shfl_sync(0xffffffffu, end - from, src);
    }
    seen += __popc(have);
    row = __shfl_sync(0xffffffffu, end, 31);
  }
  if (report && bad) raise_status(p, ST_KS_RANGE);
  return f;
}

// nt, nn: a value of D.
__device__ __forceinline__ void store_one(const FewParams& p, int t, int n, float sum) {
  const size_t at = static_cast<size_t>(t) * p.N + n;
  if (in_bounds(p, at, 1, static_cast<size_t>(p.rows) * p.N))
    p.D[at] = static_cast<uint16_t>(pack_bf16x2(sum, 0.f));
}

// One step of adding up V values over the lanes of a warp: with V > 1 the lanes of
// a pair (`o` apart) keep half of the values each, the upper lane the upper half;
// `at`: index of the first value kept.
template <int V>
__device__ __forceinline__ void fold(float (&v)[V], int o, int& at) {
  static_assert(V > 1, "");
  const bool up = threadIdx.x & o;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const float keep = up ? v[i + V / 2] : v[i], give = up ? v[i] : v[i + V / 2];
    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
  }
  at += up ? V / 2 : 0;
}

// Sums V values (a power of two) over the lanes that differ in the bits LO to 16;
// returns how many values a lane is left with, from index `at` (several lanes
// may hold the same).
template <int V, int LO, int O = 16>
__device__ __forceinline__ int fold_warp(float* v, int& at) {
  if constexpr (O < LO) {
    return V;
  } else if constexpr (V == 1) {
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], O);
    return fold_warp<1, LO, O / 2>(v, at);
  } else {
    fold<V>(*reinterpret_cast<float(*)[V]>(v), O, at);
    return fold_warp<V / 2, LO, O / 2>(v, at);
  }
}

// ---------------------------------------------------------------------- nt --
// A warp takes NT_COLS columns of D and every split-th run of 256 of K, a lane 8
// consecutive ones; U runs' loads at a time.
template <int R, int U>
__device__ __forceinline__ void nt_rows(const FewParams& p, const uint16_t* A, const uint16_t* B,
                                        int rows, int part, int split, bool on, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, step = split * 256;
  float2 acc[R * NT_COLS] = {};
  if (on) {
    for (int k0 = (part * 32 + lane) * 8; k0 < p.K; k0 += U * step) {
      uint4 b[U][NT_COLS], a[U][R];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * step;
#pragma unroll
        for (int c = 0; c < NT_COLS; ++c)
          b[u][c] = k < p.K ? ld_stream_v4(reinterpret_cast<const uint4*>(B + static_cast<size_t>(c) * p.K + k))
                            : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < R; ++r)
          a[u][r] = k < p.K && r < rows
                        ? __ldg(reinterpret_cast<const uint4*>(A + static_cast<size_t>(r) * p.K + k))
                        : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const Pairs ap = bf16x8_to_pairs(a[u][r]);
#pragma unroll
          for (int c = 0; c < NT_COLS; ++c) {
            const Pairs bp = bf16x8_to_pairs(b[u][c]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[r * NT_COLS + c] = fma2(ap.v[j], bp.v[j], acc[r * NT_COLS + c]);
          }
        }
    }
  }
  float v[R * NT_COLS];
#pragma unroll
  for (int i = 0; i < R * NT_COLS; ++i) v[i] = acc[i].x + acc[i].y;
  int at = 0;
  const int left = fold_warp<R * NT_COLS, 1>(v, at);
  static_assert(R * NT_COLS <= 32, "one value per lane");
  if (left == 1) red[warp * (FEW_ROWS * NT_COLS) + at] = v[0];
}

__global__ void __launch_bounds__(NT_THREADS, NT_PER_SM) few_nt_kernel(const FewParams p, int split) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float red[2][NT_THREADS / 32 * FEW_ROWS * NT_COLS];
  const FewGroup f = few_group<false>(p, blockIdx.y, blockIdx.x == 0 && blockIdx.y == 0);
  const int warp = threadIdx.x >> 5, part = warp % split, slot = warp / split;
  const int slots = NT_THREADS / 32 / split;
  const int n0 = (blockIdx.x * slots + slot) * NT_COLS;   // (N is a multiple of NT_COLS)
  const uint16_t* B = p.B + (static_cast<size_t>(f.g) * p.N + n0) * p.K;
  for (int r0 = 0, turn = 0; r0 < f.n; r0 += FEW_ROWS, turn ^= 1) {
    const int rows = min(FEW_ROWS, f.n - r0);
    const uint16_t* A = p.A + static_cast<size_t>(f.first + r0) * p.K;
    if (rows == 1) nt_rows<1, 2>(p, A, B, 1, part, split, n0 < p.N, red[turn]);
    else if (rows == 2) nt_rows<2, 1>(p, A, B, 2, part, split, n0 < p.N, red[turn]);
    else nt_rows<FEW_ROWS, 1>(p, A, B, rows, part, split, n0 < p.N, red[turn]);
    __syncthreads();
    for (int u = threadIdx.x; u < slots * rows * NT_COLS; u += NT_THREADS) {
      const int c = u % (slots * NT_COLS), r = u / (slots * NT_COLS);
      const int n = blockIdx.x * slots * NT_COLS + c;
      if (n >= p.N) continue;
      float sum = 0.f;
      for (int w = 0; w < split; ++w)
        sum += red[turn][((c / NT_COLS) * split + w) * (FEW_ROWS * NT_COLS) + r * NT_COLS + c % NT_COLS];
      store_one(p, f.first + r0 + r, n, sum);
    }
  }
}

// ---------------------------------------------------------------------- nn --
// A block takes COLS columns of D, a lane 8 of them; the COLS / 8 lanes of a row
// of B aside, lanes and warps share K, KB consecutive rows at a time.
template <int COLS, int R, int KB>
__device__ __forceinline__ void nn_rows(const FewParams& p, const uint16_t* A, const uint16_t* B,
                                        int rows, int n0, float* red) {
  constexpr int LN = COLS / 8, CHAINS = NN_THREADS / LN;
  const int ln = threadIdx.x % LN, n = n0 + 8 * ln;
  float2 acc[R][4] = {};
  if (n < p.N) {   // (N and K are multiples of 8)
    for (int k = KB * (threadIdx.x / LN); k < p.K; k += KB * CHAINS) {
      uint4 b[KB];
      uint32_t a[R][KB / 2];
#pragma unroll
      for (int i = 0; i < KB; ++i)
        b[i] = ld_stream_v4(reinterpret_cast<const uint4*>(B + static_cast<size_t>(k + i) * p.N + n));
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < KB / 2; ++i)
          a[r][i] = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(A + static_cast<size_t>(r) * p.K + k) + i)
                             : 0u;
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        const Pairs bp = bf16x8_to_pairs(b[i]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float x = i & 1 ? bf16_hi(a[r][i / 2]) : bf16_lo(a[r][i / 2]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[r][j] = fma2(make_float2(x, x), bp.v[j], acc[r][j]);
        }
      }
    }
  }
  float v[R * 8];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[r * 8 + 2 * j] = acc[r][j].x;
      v[r * 8 + 2 * j + 1] = acc[r][j].y;
    }
  int at = 0;   // of the lane's first value left: row at / 8, column at % 8
  const int left = fold_warp<R * 8, LN>(v, at);
#pragma unroll
  for (int i = 0; i < R * 8; ++i)
    if (i < left)
      red[((threadIdx.x >> 5) * FEW_ROWS + (at + i) / 8) * COLS + ln * 8 + (at + i) % 8] = v[i];
}

template <int COLS>
__global__ void __launch_bounds__(NN_THREADS, 2) few_nn_kernel(const FewParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  constexpr int WARPS = NN_THREADS / 32;
  __shared__ float red[WARPS * FEW_ROWS * COLS];
  const FewGroup f = few_group<false>(p, blockIdx.y, blockIdx.x == 0 && blockIdx.y == 0);
  const int n0 = blockIdx.x * COLS;
  const uint16_t* B = p.B + static_cast<size_t>(f.g) * p.K * p.N;
  for (int r0 = 0; r0 < f.n; r0 += FEW_ROWS) {
    const int rows = min(FEW_ROWS, f.n - r0);
    const uint16_t* A = p.A + static_cast<size_t>(f.first + r0) * p.K;
    if (r0 > 0) __syncthreads();   // the last sums have been read
    if (rows == 1) nn_rows<COLS, 1, 8>(p, A, B, 1, n0, red);
    else if (rows == 2) nn_rows<COLS, 2, 4>(p, A, B, 2, n0, red);
    else nn_rows<COLS, FEW_ROWS, 2>(p, A, B, rows, n0, red);
    __syncthreads();
    for (int u = threadIdx.x; u < rows * COLS; u += NN_THREADS) {
      const int r = u / COLS, c = u % COLS;
      if (n0 + c >= p.N) continue;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) sum += red[(w * FEW_ROWS + r) * COLS + c];
      store_one(p, f.first + r0 + r, n0 + c, sum);
    }
  }
}

// ---------------------------------------------------------------------- tn --
// A warp takes TN_M rows of a group's D, a lane 8 columns of each: writing D
// bounds it.
__global__ void __launch_bounds__(TN_THREADS) few_tn_kernel(const FewParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int g = blockIdx.z;
  const FewGroup f =
      few_group<true>(p, g, blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0);
  const int n = blockIdx.x * 256 + (threadIdx.x & 31) * 8;
  const int m = (blockIdx.y * (TN_THREADS / 32) + (threadIdx.x >> 5)) * TN_M;
  if (n >= p.N || m >= p.M) return;   // (M and N are multiples of 8)
  Pairs acc[TN_M] = {};
  const uint16_t* A = p.A + static_cast<size_t>(f.first) * p.M + m;
  const uint16_t* B = p.B + static_cast<size_t>(f.first) * p.N + n;
#pragma unroll 2
  for (int t = 0; t < f.n; ++t, A += p.M, B += p.N) {
    const uint4 av = __ldg(reinterpret_cast<const uint4*>(A));
    const Pairs b = bf16x8_to_pairs(__ldg(reinterpret_cast<const uint4*>(B)));
    float a[8];
    bf16x8_to_float(av, a);
#pragma unroll
    for (int i = 0; i < TN_M; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i].v[j] = fma2(make_float2(a[i], a[i]), b.v[j], acc[i].v[j]);
  }
  const size_t at = (static_cast<size_t>(g) * p.M + m) * p.N + n;
#pragma unroll
  for (int i = 0; i < TN_M; ++i) {
    if (p.C) {
      const Pairs c = bf16x8_to_pairs(*reinterpret_cast<const uint4*>(p.C + at + static_cast<size_t>(i) * p.N));
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i].v[j] = add2(acc[i].v[j], c.v[j]);
    }
    if (in_bounds(p, at + static_cast<size_t>(i) * p.N, 8, static_cast<size_t>(p.G) * p.M * p.N))
      *reinterpret_cast<uint4*>(p.D + at + static_cast<size_t>(i) * p.N) = pairs_to_bf16x8(acc[i]);
  }
}

}  // namespace

// Which form is ahead goes by the rows of the fullest group, of which the host
// knows the total only: nt and nn up to the FEW_ROWS that one pass over the
// weights takes (in us, the tensor cores' kernel and this one: nt 1 row of 3496 x
// 1392 7.7, 3.6; 4 rows in one group, 7792 x 872 7.1, 7.2, in two of 784 x 4592
// 10.0, 5.2; 8 in 19 groups, 944 x 7400 25, 25; two passes over weights of a few
// MB, 5 rows of 424 x 5144 13.2, 4.9, 7 of 2744 x 720 6.0, 5.3, but 6 of 3120 x 5216
// 21.7, 24.6; nn 2 rows in 46 groups, 648 x 2128
// 9.6, 4.9, in one of 8136 x 1024 7.3, 4.9; with 5 in one group of 5640 x 7880 24,
// 78), more where many groups share them.  tn reads each row once: 3 rows in one
// group, 6496 x 568 7.6, 4.3; 5 in 30 groups, 1872 x 5320 115, 90 (88 at the copy
// rate); 8 in one of two, 6816 x 576 8.7, 7.4; 21 in one of two, 304 x 5488 6.1,
// 7.6.  At most 32 in all, should one group have them.
bool bf16_few_rows(const BfCall& c) {
  const bool twice = c.form == kBfNT && static_cast<long long>(c.N) * c.K <= 4 << 20;
  const int most = c.form == kBfTN ? 8 + c.G / 2 : (twice ? 2 : 1) * FEW_ROWS + c.G / 4;
  return c.forced.lanes == 0 && c.rows <= std::min(32, most) && c.M <= 64 * 65535;
}

cudaError_t launch_bf16_few(const BfCall& c, int num_sms, cudaStream_t stream) {
  const FewParams p{static_cast<const uint16_t*>(c.A), static_cast<const uint16_t*>(c.B),
                    static_cast<const uint16_t*>(c.C), static_cast<uint16_t*>(c.D),
                    c.sizes, c.G, c.rows, c.M, c.N, c.K, c.status};
  const int groups = std::min(c.G, c.rows);   // that can have rows
  if (c.form == kBfTN)
    return launch_dependent(few_tn_kernel,
                            dim3((c.N + 255) / 256, (c.M + TN_M * 8 - 1) / (TN_M * 8), c.G), TN_THREADS,
                            stream, 0, p);
  if (c.form == kBfNT) {
    // K is split over the block's warps until there are two blocks per SM or a
    // warp has one run of 256
    int split = 1;
    auto blocks = [&] { return (c.N + 32 / split - 1) / (32 / split); };
    while (split < 8 && static_cast<long long>(blocks()) * groups < 2 * num_sms && c.K > 256 * split)
      split *= 2;
    return launch_dependent(few_nt_kernel, dim3(blocks(), groups), NT_THREADS, stream, 0, p, split);
  }
  // the widest rows of B (128 bytes down to 32) that still make enough blocks
  auto blocks = [&](int cols) { return (c.N + cols - 1) / cols; };
  auto enough = [&](int cols) { return static_cast<long long>(blocks(cols)) * groups >= num_sms; };
  return enough(64)   ? launch_dependent(few_nn_kernel<64>, dim3(blocks(64), groups), NN_THREADS, stream, 0, p)
         : enough(32) ? launch_dependent(few_nn_kernel<32>, dim3(blocks(32), groups), NN_THREADS, stream, 0, p)
                      : launch_dependent(few_nn_kernel<16>, dim3(blocks(16), groups), NN_THREADS, stream, 0, p);
}

}  // namespace dgk
