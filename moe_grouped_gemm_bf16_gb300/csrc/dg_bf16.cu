// bf16 products grouped by expert with ragged sizes, for sm_103a.  The groups'
// rows lie one after the other in A (group e owns sizes[e] rows, any number,
// read on the device):
//
//   nt  D[t][n]    = sum_k A[t][k] B[e][n][k]     forward, t in group e
//   nn  D[t][n]    = sum_k A[t][k] B[e][k][n]     gradient of the activations
//   tn  D[e][m][n] = C[e][m][n] + sum_{t in e} A[t][m] B[t][n]   gradient of the weights
//
// Every form is one computation: a tile of D with `lanes` consecutive columns
// of D on the tensor memory's lanes (B is the MMA's first operand) and up to
// `bc` rows of D on its columns (A is the second operand).  The ragged dimension
// of nt and nn is then the MMA's N, which the instruction takes in steps of
// 16 or 32: a group of 20 rows costs 32 columns, not 128 lanes, and a weight
// tile is always full.
//
// Two kernels:
//  * PAIR: a persistent CTA pair per 256 x 256 tile (cta_group::2: each CTA
//    holds 128 lanes of B and half of A's rows), for groups of many rows;
//  * single: one persistent CTA per tile of up to 256 lanes x 128 rows, for
//    groups of few rows, where the time is that of reading the weights.
// Where there are too few tiles for the SMs, either splits the reduction over
// the CTAs (pairs) of a cluster, one tile per cluster: each leaves its fp32
// partial in shared memory, and each then adds up a share of the rows in the
// order of the ranks.  The host estimates each tiling's time and takes the
// least (bf_cost).
//
// Warps 0 and 2 load by TMA (B's tile and A's) into a ring of slots, BK deep in
// the reduction: 64 for the pair (six or seven slots of 32 KB a CTA: with three
// of 64 KB the memory-bound nn case took 168 us, so 156), 128 for the single form
// (half the loads to issue).  Warp 1 (of the pair's leader) issues tcgen05.mma
// kind::f16 into one of two fp32 accumulators in tensor memory, warps 4-11
// round the other one to bf16 and store it.  tn's reduction ends at a group's
// last row, which need not end a slot: warp 3 zeroes the rows behind it, up to
// the next multiple of the MMA's 16, in both operands (the next group's rows
// may hold anything).
//
// Measured: nt 32647 rows in 4 groups, 4096 x 7168: 1135-1170 us (1640-1690
// TFLOP/s under the power cap, 1.43 GHz; the tensor pipe 94% active), tn 16391
// rows 2048 x 7168: 251 us alone, 290 us in a loop (with an addend, read four bytes
// at a time between the stores, 445 us; 8192 rows in 8 groups, 2048 x 2048: 43 us, with
// one 263); nn 5003 rows in 29 of 32 groups: 156 us (6.0 TB/s); nt 61 rows on 6 of 8
// groups, 4096 x 7168: 58 us (6.1 TB/s).  Far from these where groups are uneven or
// empty, or a width is a little above whole tiles (tn 12818 rows in one of two groups,
// 1816 x 352: 51 us, the floor 9).
//
// Every wait is bounded, as in the FP8 kernels.  Calls of a few rows in all take
// dg_bf16_few.cu instead.
#include <algorithm>
#include <cmath>

#include "dg_bf16.h"
#include "dg_params.h"
#include "dg_wait.cuh"
#include "ptx.cuh"

namespace dgk {
namespace {

constexpr int BF_EPI = 8;       // epilogue warps
constexpr int BF_THREADS = 128 + 32 * BF_EPI;
constexpr int BF_BAND = 8;      // column blocks (rows of D) per raster band
constexpr int BF_MAX_STAGES = 10;
constexpr int kBfMaxSmem = 232448;
constexpr int kBfMaxCluster = 8;

struct BfParams {
  int G;
  int rows;        // rows of A over all groups
  int M;           // tn: rows of each D[e]
  int N;           // columns of D
  int K;           // nt, nn: the reduction
  int lanes;       // columns of D per tile (pair: 256)
  int nl;          // lane blocks: ceil(N / lanes)
  int bc;          // rows of D per tile (pair: 256)
  int nc;          // tn: column blocks of each group: ceil(M / bc)
  int split;       // CTAs (pairs) of a cluster that share a tile's reduction
  unsigned long long inv_nl, inv_band, inv_per;   // Divisor of nl, BF_BAND nl, nc nl (tn)
  int stages;
  int p_bytes;     // bytes of a slot's lane operand (per CTA)
  int q_bytes;     // bytes of a slot's column operand (per CTA)
  int p_whole;     // extent of the operands' whole 64-wide pieces (see `operand` below)
  int q_whole;
  const int32_t* sizes;
  uint16_t* D;
  const uint16_t* C;
  unsigned int* status;
  unsigned long long timeout_ns;
  unsigned int debug_flags;
};

// Tensor maps of the lane and the column operand: [0] takes a slot's 64-wide
// pieces in one load, [1] one piece.
struct BfMaps {
  CUtensorMap p[2], q[2];
};

// Shared memory behind the ring: barriers, TMEM base and abort flag, then the
// groups' first rows and first column blocks.
struct BfSmem {
  static constexpr int FULL = 0, EMPTY = BF_MAX_STAGES, TAIL = 2 * BF_MAX_STAGES,
                       T_FULL = 3 * BF_MAX_STAGES, T_EMPTY = T_FULL + 2, MMA_DONE = T_EMPTY + 2,
                       NUM_BARS = MMA_DONE + 1;
  static constexpr int MISC = NUM_BARS * 8;
  // (checked build: fill counters of the lane and the column operand's slots)
  static constexpr int FILLS = MISC + 8;
  static constexpr int TAB = (FILLS + (kDebug ? 2 * BF_MAX_STAGES * 4 : 0) + 15) / 16 * 16;
  __host__ __device__ static constexpr int fixed(int G) { return 1024 + TAB + 2 * (G + 1) * 4; }
};

// Reduction depth of a slot.
__host__ __device__ constexpr int bf_bk(bool pair) { return pair ? 64 : 128; }

struct BfTile {
  int g;          // group
  int l0;         // first column of D
  int cols;       // rows of D in this tile
  int q0;         // first row of the column operand (nt, nn: row of A; tn: m)
  int k0;         // tn: first row of the group
  int kn;         // reduction length
  int nk;         // slots of it
  int kbeg, kend; // this CTA's (pair's) slots
};

// x / d for any 32-bit x with inv = floor(2^64 / d) + 1 (d > 1), 0 for d = 1
// (Lemire, Kaser and Kurz, "Faster remainder by direct computation", 2019).  The
// roles decode a tile each, on their critical path: with five integer divisions
// and a binary search that took 1000 to 1450 cycles a tile.
__host__ __device__ constexpr unsigned long long bf_inverse(unsigned d) {
  return d <= 1 ? 0 : ~0ull / d + 1;
}
__device__ __forceinline__ int bf_div(int x, unsigned long long inv) {
  return inv == 0 ? x : static_cast<int>(__umul64hi(static_cast<unsigned>(x), inv));
}

// Tile t; `from`: a group at or before the tile's (a role's tiles come in
// rising order), replaced by the tile's.  (350 to 500 cycles so.)
template <int BK, int FORM>
__device__ __forceinline__ BfTile bf_tile(int t, const BfParams& p, const int* first,
                                          const int* blk, int krank, int& from) {
  BfTile T;
  int nc;
  if (FORM == kBfTN) {
    T.g = bf_div(t, p.inv_per);
    t -= T.g * (p.nc * p.nl);
    nc = p.nc;
  } else {
    // largest g with blk[g] <= b
    const int b = bf_div(t, p.inv_nl);
    while (blk[from + 1] <= b) ++from;
    T.g = from;
    t -= blk[from] * p.nl;
    nc = blk[from + 1] - blk[from];
  }
  // bands of BF_BAND column blocks; within a band first along the column
  // blocks, then along the lanes, so that concurrent tiles share operands in L2
  const int band = bf_div(t, p.inv_band);
  const int r = t - band * (BF_BAND * p.nl);
  const int h = min(BF_BAND, nc - band * BF_BAND);
  // r / h with h <= 8: exact below 2^20 (r + 0.5 is half a unit or more from any
  // multiple of h, the product off by less than 2^-22 of itself)
  const int q = static_cast<int>((static_cast<float>(r) + 0.5f) * __frcp_rn(static_cast<float>(h)));
  T.l0 = q * p.lanes;
  const int c0 = (band * BF_BAND + r - q * h) * p.bc;
  const int n = first[T.g + 1] - first[T.g];
  if (FORM == kBfTN) {
    T.cols = min(p.bc, p.M - c0);
    T.q0 = c0;
    T.k0 = first[T.g];
    T.kn = n;
  } else {
    T.cols = min(p.bc, n - c0);
    T.q0 = first[T.g] + c0;
    T.k0 = 0;
    T.kn = p.K;
  }
  T.nk = (T.kn + BK - 1) / BK;
  T.kbeg = 0;
  T.kend = T.nk;
  if (p.split > 1) {
    T.kbeg = static_cast<int>(static_cast<long long>(T.nk) * krank / p.split);
    T.kend = static_cast<int>(static_cast<long long>(T.nk) * (krank + 1) / p.split);
  }
  return T;
}

__device__ __forceinline__ size_t bf_elements(const BfParams& p, bool tn) {
  return (tn ? static_cast<size_t>(p.G) * p.M : static_cast<size_t>(p.rows)) * p.N;
}

// Four columns of a row of D: the addend in fp32, then one rounding.
__device__ __forceinline__ void store_four(const BfParams& p, bool tn, size_t at, float4 v) {
  if (!in_bounds(p, at, 4, bf_elements(p, tn))) return;
  if (p.C) {
    const uint2 c = *reinterpret_cast<const uint2*>(p.C + at);
    v.x += __uint_as_float(c.x << 16);
    v.y += __uint_as_float(c.x & 0xFFFF0000u);
    v.z += __uint_as_float(c.y << 16);
    v.w += __uint_as_float(c.y & 0xFFFF0000u);
  }
  *reinterpret_cast<uint2*>(p.D + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// A CTA's share of a split tile's rows: the ranks' partials added up in the order
// of the ranks (`has`: those that have one).  A warp takes 8 / S rows at a time,
// a lane four columns of each, and asks for all S partials of them before it adds
// (rank by rank, with the ranks' flags before, 13 rows split in 8 took 3.8 us, so
// 1.0).  Nothing is stored where a rank gave up a wait (`ok`: this thread knows of
// none; lane r asks rank r's `flag`, while the partials are on their way).
template <bool PAIR, int BC, bool TN, int S>
__device__ __forceinline__ void add_partials(const BfParams& p, const BfTile& T, uint32_t sbase,
                                             uint32_t has, uint32_t flag, bool ok, int krank,
                                             uint32_t side, int halves) {
  constexpr int U = 8 / S;
  const int lane = threadIdx.x & 31, warp = static_cast<int>(threadIdx.x >> 5) - 4;
  const int l_end = min(p.N, T.l0 + p.lanes);
  const int c0 = U * (p.split * warp + krank);
  if (c0 >= T.cols) return;
  uint32_t gave_up = 0;
  if (lane < p.split) gave_up = ld_cluster_u32(map_cluster(flag, PAIR ? 2 * lane + side : lane));
  for (int a = 0; a < halves; ++a) {
    const int l = T.l0 + (PAIR ? static_cast<int>(side) : a) * 128 + 4 * lane;
    for (int c = c0; c < T.cols; c += U * BF_EPI * p.split) {
      const int rows = l < l_end ? min(U, T.cols - c) : 0;   // (l_end is a multiple of 8)
      float4 x[S][U];
      const uint32_t at = sbase + ((a * BC + c) * 128 + 4 * lane) * 4;
#pragma unroll
      for (int r = 0; r < S; ++r) {
        const int n = (has >> r) & 1u ? rows : 0;
        const int rank = min(r, p.split - 1);
        const uint32_t from = map_cluster(at, PAIR ? 2 * rank + side : rank);
#pragma unroll
        for (int j = 0; j < U; ++j) x[r][j] = ld_cluster_v4_if(from + j * 512, j < n);
      }
      if (!__all_sync(0xffffffffu, ok && gave_up == 0)) return;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < S; ++r) {
          sum.x += x[r][j].x; sum.y += x[r][j].y; sum.z += x[r][j].z; sum.w += x[r][j].w;
        }
        if (j < rows)
          store_four(p, TN, ((TN ? static_cast<size_t>(T.g) * p.M : 0) + T.q0 + c + j) * p.N + l, sum);
      }
    }
  }
}

// BC: capacity of an accumulator in rows of D (`bc` at most).
template <bool PAIR, int BC, int FORM>
__global__ void __launch_bounds__(BF_THREADS, 1)
bf16_grouped_kernel(const __grid_constant__ BfMaps maps, const BfParams p) {
  using L = BfSmem;
  constexpr int BK = bf_bk(PAIR);
  constexpr bool TN = FORM == kBfTN, P_MN = FORM != kBfNT;
  // columns of one accumulator: two M = 128 halves side by side, or the pair's
  constexpr int ACC = PAIR ? BC : 2 * BC;
  static_assert(2 * ACC <= 512, "two accumulators");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t q_off = p.stages * p.p_bytes;
  const int ring = p.stages * (p.p_bytes + p.q_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sbase + ring + 8 * i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + ring + L::MISC);
  volatile uint32_t* abort_flag = misc + 1;
  volatile uint32_t* fills = reinterpret_cast<uint32_t*>(smem + ring + L::FILLS);
  int* first = reinterpret_cast<int*>(smem + ring + L::TAB);
  int* blk = first + p.G + 1;
  const int cluster = (PAIR ? 2 : 1) * p.split;
  const uint32_t crank = cluster > 1 ? cluster_ctarank() : 0;
  const uint32_t side = PAIR ? crank & 1 : 0;    // CTA of the pair
  const uint32_t leader = crank - side;          // its leader's rank
  const int krank = static_cast<int>(PAIR ? crank >> 1 : crank);   // share of the reduction
  const int unit = blockIdx.x / cluster, units = gridDim.x / cluster;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      // the two producers (pair: the leader's, for both CTAs' bytes)
      mbar_init(bar(L::FULL + s), 2);
      mbar_init(bar(L::EMPTY + s), 1);
      mbar_init(bar(L::TAIL + s), 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(L::T_FULL + b), 1);
      mbar_init(bar(L::T_EMPTY + b), (PAIR ? 2 : 1) * BF_EPI);
    }
    mbar_init(bar(L::MMA_DONE), 1);
    misc[1] = 0;
    if constexpr (kDebug)
      for (int i = 0; i < 2 * BF_MAX_STAGES; ++i) fills[i] = 0;
    fence_mbarrier_init();
    prefetch_tmap(&maps.p[0]);
    prefetch_tmap(&maps.q[0]);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(sbase + ring + L::MISC, 2 * ACC);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(sbase + ring + L::MISC, 2 * ACC);
      tmem_relinquish();
    }
  }
  grid_dep_wait();
  grid_dep_launch_dependents();
  if (warp == 2) {
    // first row and first column block of every group; a negative size counts
    // as zero and the running total stops at `rows` (both reported)
    int row = 0, nb = 0;
    bool bad = false;
    for (int base = 0; base < p.G; base += 32) {
      const int g = base + lane;
      int v = g < p.G ? __ldg(p.sizes + g) : 0;
      if (v < 0) { bad = true; v = 0; }
      if (v > p.rows) { bad = true; v = p.rows; }
      // the running total in 64 bits: 32 sizes may pass 2^31
      long long x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (row + x > p.rows) bad = true;
      const int end = static_cast<int>(min(row + x, static_cast<long long>(p.rows)));
      const int prev = __shfl_up_sync(0xffffffffu, end, 1);
      const int mine = end - (lane == 0 ? row : prev);
      int c = (mine + p.bc - 1) / p.bc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += y;
      }
      if (g < p.G) {
        first[g + 1] = end;
        blk[g + 1] = nb + c;
      }
      row = __shfl_sync(0xffffffffu, end, 31);
      nb += __shfl_sync(0xffffffffu, c, 31);
    }
    if (lane == 0) first[0] = blk[0] = 0;
    if (bad && blockIdx.x == 0) raise_status(p, ST_KS_RANGE);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // a pair's CTAs signal each other's barriers from here on (their initialisation
  // was made visible to the cluster by thread 0's fence)
  if constexpr (PAIR) {
    cluster_arrive_relaxed();
    cluster_wait();
  }
  const uint32_t tmem = misc[0];
  const int tiles = TN ? p.G * p.nc * p.nl : blk[p.G] * p.nl;
  // the MMA's N: whole instruction steps; a pair's CTA holds half of the
  // columns each (tn: in whole 64-wide boxes)
  auto mma_n = [&](int cols) {
    return PAIR ? (TN ? (cols + 127) & ~127 : (cols + 31) & ~31) : (cols + 15) & ~15;
  };
  int group = 0;   // this thread's place in the groups (bf_tile)
  // the tile's last slot needs zeroed rows, and is this CTA's
  auto ragged = [&](const BfTile& T) {
    return TN && (T.kn & 15) != 0 && T.kend == T.nk && T.kbeg < T.kend;
  };

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------- TMA producers --
    // warp 0: the lane operand (B), warp 2: the column operand (A); one load
    // each per slot (a thread that issues one stalls for ~250 cycles)
    if (lane == 0 && !(p.debug_flags & DBG_SKIP_PRODUCER)) {
      const bool lanes_op = warp == 0;
      const CUtensorMap* wide = lanes_op ? &maps.p[0] : &maps.q[0];
      const CUtensorMap* piece = lanes_op ? &maps.p[1] : &maps.q[1];
      const bool mn = lanes_op ? P_MN : TN;
      const int whole = lanes_op ? p.p_whole : p.q_whole;
      const uint32_t bytes = lanes_op ? p.p_bytes : p.q_bytes;
      // 64-wide pieces of a slot, and the bytes of those that an MN-major operand
      // has at column x (what lies wholly past its edge is neither loaded nor
      // stored)
      const int pieces = mn ? static_cast<int>(bytes / (BK * 128)) : BK / 64;
      const int extent = lanes_op ? p.N : p.M;
      auto there = [&](int x) { return mn ? min(pieces, max(0, (extent - x + 63) >> 6)) : pieces; };
      const uint32_t base = sbase + (lanes_op ? 0 : q_off);
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0, tails = 0, tail_par = 0;
      for (int t = unit; t < tiles; t += units) {
        const BfTile T = bf_tile<BK, FORM>(t, p, first, blk, krank, group);
        const int half = lanes_op ? 128 : mma_n(T.cols) / 2;   // from one CTA of a pair to the other
        const int at = (lanes_op ? T.l0 : T.q0) + static_cast<int>(side) * half;
        const uint32_t piece_bytes = bytes / pieces;
        const uint32_t mine = there(at) * piece_bytes;
        const uint32_t both = mine + (PAIR ? there(at + half) * piece_bytes : 0);   // (the leader's)
        const int g = (lanes_op && !TN) ? T.g : 0;
        const bool rag = ragged(T);
        for (int n = T.kend - T.kbeg, j = 0; j < n; ++j) {
          // a ragged last slot is loaded first
          const int i = !rag ? T.kbeg + j : j == 0 ? T.kend - 1 : T.kbeg + j - 1;
          bool go = wait_bar(bar(L::EMPTY + s), ph ^ 1, abort_flag, p);
          const int k = T.k0 + i * BK;
          if constexpr (kDebug) {
            const int rows = lanes_op ? p.N : (TN ? p.M : p.rows);
            // (a pair's second CTA may start past the tensor: zero-filled)
            if (go && (T.g >= p.G || at < 0 || at >= rows + (PAIR ? 128 : 0) || k < 0 ||
                       k >= (TN ? p.rows : p.K))) {
              dbg_fail(p, ST_DEBUG_BOUNDS, abort_flag);
              go = false;
            }
            const int slot = lanes_op ? s : BF_MAX_STAGES + s;
            if (go) fills[slot] = fills[slot] + 1;
          }
          if (go) {
            const uint32_t dst = base + s * bytes;
            // a slot whose rows warp 3 completes arrives on its own CTA's TAIL
            const bool to_tail = rag && j == 0;
            const uint32_t b = to_tail ? bar(L::TAIL + s)
                               : PAIR  ? map_cluster(bar(L::FULL + s), leader)
                                       : bar(L::FULL + s);
            // the leader expects both CTAs' bytes (a remote arrival of the peer
            // at cluster scope would cost it a microsecond per slot)
            if (to_tail || side == 0)
              mbar_arrive_expect_tx(to_tail ? b : bar(L::FULL + s), to_tail ? mine : both);
            auto load = [&](const CUtensorMap* m, uint32_t d, int x, int y, int z) {
              if (PAIR && !to_tail) tma_load_4d_pair(map_cluster(d, crank), m, b, x, y, z, g);
              else tma_load_4d(d, m, b, x, y, z, g);
            };
            // one load where all the slot's 64-wide pieces are whole, else one
            // per piece (a piece's part past the tensor's edge is filled with zeros)
            if ((mn ? at : k) + 64 * pieces <= whole) {
              if (mn) load(wide, dst, 0, k, at >> 6);
              else load(wide, dst, 0, at, k >> 6);
            } else {
              for (int j = 0; j < there(at); ++j) {
                const uint32_t d = dst + j * piece_bytes;
                if (mn) load(piece, d, at + 64 * j, k, 0);
                else load(piece, d, k + 64 * j, at, 0);
              }
            }
            // (the slot's latest load, for the drain below: on one barrier or
            // the other)
            if (to_tail) {
              tails |= 1u << s;
              tail_par ^= 1u << s;
              issued &= ~(1u << s);
            } else {
              issued |= 1u << s;
              issued_par = (issued_par & ~(1u << s)) | (ph << s);
            }
          }
          if (++s == p.stages) { s = 0; ph ^= 1; }
        }
      }
      // after an abort the latest load into a slot may still be in flight
      // (pair: both CTAs' loads count on the leader's barriers; the CTAs leave
      // together)
      for (int q = 0; q < p.stages; ++q) {
        if (((issued >> q) & 1u) && side == 0)
          drain_wait(bar(L::FULL + q), (issued_par >> q) & 1u, p);
        if ((tails >> q) & 1u) drain_wait(bar(L::TAIL + q), ((tail_par >> q) & 1u) ^ 1u, p);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer --
    // The whole warp walks the loop, converged, and one elected thread issues:
    // with a single thread in the loop the descriptors of every instruction
    // cost the issue more than the instruction takes to run (nt, 32647 rows, N =
    // 4096, K = 7168, the loads switched off: 1092 us; so 830 us, the tensor
    // cores' rate).
    if (side == 0) {
      const bool issuer = elect_one();
      // a K step of 16: 32 bytes inside a K-major row, whose 64-wide pieces lie
      // `half` bytes apart; two 8-row atoms (2 KB) of an MN-major slot, whose
      // 64-wide atoms of 128 rows lie 16 KB apart
      constexpr uint32_t ATOM = BK * 128;
      const uint32_t p_half = P_MN ? 0 : p.p_bytes / 2, q_half = TN ? 0 : p.q_bytes / 2;
      const bool two = !PAIR && p.lanes > 128;
      // (desc units of 16 bytes) the second 128 lanes
      constexpr uint32_t P_SECOND = (P_MN ? 2 * ATOM : 16384) >> 4;
      const uint16_t mask = static_cast<uint16_t>(PAIR ? 0x3u << leader : 0x1u);
      int s = 0, b = 0;
      uint32_t ph = 0, bph = 0;
      uint32_t turn = 1;   // checked build: the fill that a slot has to hold
      for (int t = unit; t < tiles; t += units) {
        const BfTile T = bf_tile<BK, FORM>(t, p, first, blk, krank, group);
        if (T.kbeg == T.kend) continue;
        const uint32_t idesc = idesc_bf16_f32(PAIR ? 256 : 128, mma_n(T.cols), P_MN, TN);
        const uint32_t d = tmem + static_cast<uint32_t>(b * ACC);
        bool ok = wait_bar(bar(L::T_EMPTY + b), bph ^ 1, abort_flag, p);
        tc_fence_after();
        const bool rag = ragged(T);
        const int n = T.kend - T.kbeg;
        for (int j = 0; j < n; ++j) {
          // a ragged last slot comes first, when warp 3 has had the time of the
          // previous tile for it (8192 rows in 16 groups, 2048 x 7168: 189 us with
          // it last, 179 so, 166 without any zeroing)
          const bool tail = rag && j == 0;
          const int i = !rag ? T.kbeg + j : tail ? T.kend - 1 : T.kbeg + j - 1;
          // (the peer's warp 3 wrote the zeros of its own half)
          ok = (PAIR && tail ? wait_bar<true>(bar(L::FULL + s), ph, abort_flag, p)
                             : wait_bar(bar(L::FULL + s), ph, abort_flag, p)) && ok;
          tc_fence_after();
          if constexpr (kDebug) {
            if (ok && (fills[s] != turn || fills[BF_MAX_STAGES + s] != turn)) {
              dbg_fail(p, ST_DEBUG_PHASE, abort_flag);
              ok = false;
            }
          }
          if (issuer && ok) {
            const uint32_t ps = sbase + s * p.p_bytes, qs = sbase + q_off + s * p.q_bytes;
            const uint64_t pd = P_MN ? smem_desc_sw128_mnmajor(ps, ATOM) : smem_desc_sw128_kmajor(ps);
            const uint64_t qd = TN ? smem_desc_sw128_mnmajor(qs, ATOM) : smem_desc_sw128_kmajor(qs);
            auto step = [&](int kk, uint32_t acc) {
              const uint64_t pk = pd + (P_MN ? kk * (2048 >> 4)
                                             : (kk >> 2) * (p_half >> 4) + (kk & 3) * (32 >> 4));
              const uint64_t qk = qd + (TN ? kk * (2048 >> 4)
                                           : (kk >> 2) * (q_half >> 4) + (kk & 3) * (32 >> 4));
              if constexpr (PAIR) {
                mma_bf16_pair(d, pk, qk, idesc, acc);
              } else {
                mma_bf16(d, pk, qk, idesc, acc);
                // (the rows past `lanes` are not stored)
                if (two) mma_bf16(d + BC, pk + P_SECOND, qk, idesc, acc);
              }
            };
            const int left = T.kn - i * BK;
            if (left >= BK) {
              step(0, j > 0);
#pragma unroll
              for (int kk = 1; kk < BK / 16; ++kk) step(kk, 1);
            } else {
              for (int kk = 0; 16 * kk < left; ++kk) step(kk, j > 0 || kk > 0);
            }
            if constexpr (PAIR) mma_commit_pair_multicast(bar(L::EMPTY + s), mask);
            else mma_commit(bar(L::EMPTY + s));
            if (j == n - 1) {
              if constexpr (PAIR) mma_commit_pair_multicast(bar(L::T_FULL + b), mask);
              else mma_commit(bar(L::T_FULL + b));
            }
          }
          __syncwarp();
          if (++s == p.stages) {
            s = 0;
            ph ^= 1;
            if constexpr (kDebug) ++turn;
          }
        }
        b ^= 1;
        if (b == 0) bph ^= 1;
      }
      if (issuer) {
        if constexpr (PAIR) mma_commit_pair_multicast(bar(L::MMA_DONE), static_cast<uint16_t>(1u << leader));
        else mma_commit(bar(L::MMA_DONE));
        drain_wait(bar(L::MMA_DONE), 0, p);
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------ tn's last rows --
    if (TN) {
      int s = 0;
      uint32_t par = 0;
      for (int t = unit; t < tiles; t += units) {
        const BfTile T = bf_tile<BK, FORM>(t, p, first, blk, krank, group);
        if (ragged(T)) {
          // all 32 lanes: wait for this CTA's two loads, then zero the rows
          // behind the group's last one, up to the next multiple of 16 (a row
          // is one 128-byte line of each 64-wide atom)
          const bool ok = wait_bar(bar(L::TAIL + s), (par >> s) & 1u, abort_flag, p);
          par ^= 1u << s;
          if (ok) {
            const int left = T.kn - (T.nk - 1) * BK, end = (left + 15) & ~15;
            constexpr int ATOM = BK * 128;
            // a lane takes 16 bytes of every fourth row, in each atom
            const uint32_t off = (left + (lane >> 3)) * 128 + (lane & 7) * 16;
            auto zero = [&](uint32_t base, int atoms) {
              for (int i = 0; i < atoms; ++i)
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                  if (left + (lane >> 3) + r < end)
                    st_shared_v4(base + i * ATOM + off + r * 128, 0, 0, 0, 0);
            };
            zero(sbase + s * p.p_bytes, p.p_bytes / ATOM);
            zero(sbase + q_off + s * p.q_bytes, p.q_bytes / ATOM);
          }
          fence_proxy_async_smem();
          __syncwarp();
          // in place of the two producers' arrivals: one per CTA of a pair, or two
          if constexpr (PAIR) {
            if (lane == 0) mbar_arrive_remote_release(bar(L::FULL + s), leader);
          } else {
            if (lane < 2) mbar_arrive(bar(L::FULL + s));
          }
        }
        s = (s + T.kend - T.kbeg) % p.stages;
      }
    }
    __syncwarp();
  }

  // -------------------------------------------------------------- epilogue --
  const int q = warp & 3, eh = (warp >> 2) - 1;   // lane quarter; which of the warps on it
  const int halves = PAIR ? 1 : (p.lanes + 127) / 128;
  // Rows c .. c + 31 of the tile from a lane's 32 values of one column of D:
  // rounded in pairs of rows, then exchanged with the neighbouring lane, so that
  // the even lane stores two columns of the even row and the odd one those of
  // the odd row.  With an addend the exchange is of fp32 values: one rounding,
  // after the sum.
  auto store_rows = [&](const BfTile& T, int l, int c, const uint32_t (&v)[32]) {
    const int odd = lane & 1;
    const size_t row = (TN ? static_cast<size_t>(T.g) * p.M : 0) + T.q0 + c + odd;
    // rows this lane may store: those of its parity below the tile's end
    int n = l < min(p.N, T.l0 + p.lanes) ? min(16, (T.cols - c - odd + 1) >> 1) : 0;
    if constexpr (kDebug) {
      const size_t end = TN ? static_cast<size_t>(p.G) * p.M : static_cast<size_t>(p.rows);
      if (n > 0 && row + 2 * (n - 1) >= end) {
        raise_status(p, ST_DEBUG_BOUNDS);
        n = 0;
      }
    }
    const size_t step = 2 * static_cast<size_t>(p.N);
    uint16_t* d = p.D + row * p.N + l;
    if (p.C == nullptr) {
      // all exchanges first: between predicated stores they would run one by one
      const uint32_t sel = odd ? 0x3276u : 0x5410u;
      uint32_t o[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        o[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = __byte_perm(o[j], __shfl_xor_sync(0xffffffffu, o[j], 1), sel);
      if (n == 16) {
#pragma unroll
        for (int j = 0; j < 16; ++j, d += step) *reinterpret_cast<uint32_t*>(d) = o[j];
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j, d += step)
          if (j < n) *reinterpret_cast<uint32_t*>(d) = o[j];
      }
    } else {
      const uint16_t* cp = p.C + row * p.N + l;
#pragma unroll
      for (int j = 0; j < 16; ++j, d += step, cp += step) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[2 * j] : v[2 * j + 1], 1);
        if (j < n) {
          const uint32_t cw = *reinterpret_cast<const uint32_t*>(cp);
          const float lo = __uint_as_float(odd ? got : v[2 * j]) + __uint_as_float(cw << 16);
          const float hi =
              __uint_as_float(odd ? v[2 * j + 1] : got) + __uint_as_float(cw & 0xFFFF0000u);
          *reinterpret_cast<uint32_t*>(d) = pack_bf16x2(lo, hi);
        }
      }
    }
  };
  // first column of the thread's pair of columns of D, in half `a` of the lanes
  auto column = [&](const BfTile& T, int a) {
    return T.l0 + (PAIR ? static_cast<int>(side) : a) * 128 + q * 32 + (lane & ~1);
  };
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(q * 32) << 16);
  if (p.split == 1) {
    if (warp >= 4) {
      int b = 0;
      uint32_t bph = 0;
      for (int t = unit; t < tiles; t += units) {
        const BfTile T = bf_tile<BK, FORM>(t, p, first, blk, 0, group);
        const int l_end = min(p.N, T.l0 + p.lanes);
        if (T.nk == 0) {
          // tn, a group without rows: its block of D is C, or zero
          const int l0 = T.l0 + static_cast<int>(side) * 128;
          const int per = PAIR ? 16 : p.lanes >> 3;   // 8 columns each
          for (int u = static_cast<int>(threadIdx.x) - 128; u < per * T.cols; u += 32 * BF_EPI) {
            const int r = u / per, l = l0 + 8 * (u - r * per);
            if (l >= l_end) continue;
            const size_t at = (static_cast<size_t>(T.g) * p.M + T.q0 + r) * p.N + l;
            if (!in_bounds(p, at, 8, bf_elements(p, TN))) continue;
            *reinterpret_cast<uint4*>(p.D + at) =
                p.C ? *reinterpret_cast<const uint4*>(p.C + at) : make_uint4(0, 0, 0, 0);
          }
          continue;
        }
        // (the warp's lanes agree, for the exchange)
        const bool ok =
            __all_sync(0xffffffffu, wait_bar(bar(L::T_FULL + b), bph, abort_flag, p));
        tc_fence_after();
        for (int a = 0; a < halves; ++a) {
          const int l = column(T, a);
          // two chunks of 32 rows at a time, for one wait on tensor memory
          for (int c = 32 * eh; c < T.cols; c += 128) {
            uint32_t v[32], w[32];
            const bool more = c + 64 < T.cols;
            const uint32_t at = t_lane + static_cast<uint32_t>(b * ACC + a * BC + c);
            tmem_ld_32x32b_x32(at, v);
            if (more) tmem_ld_32x32b_x32(at + 64, w);
            tmem_wait_ld(v);
            if (more) tmem_wait_ld(w);
            if (ok) {
              store_rows(T, l, c, v);
              if (more) store_rows(T, l, c + 64, w);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR && side != 0) mbar_arrive_remote_relaxed(bar(L::T_EMPTY + b), leader);
          else mbar_arrive(bar(L::T_EMPTY + b));
        }
        b ^= 1;
        if (b == 0) bph ^= 1;
      }
    }
  } else {
    // One tile per cluster.  Its MMAs and loads are done once the accumulator
    // is complete: the ring now holds the partial [half][row][128] in fp32.
    const bool mine = unit < tiles;
    BfTile T{};
    if (mine) T = bf_tile<BK, FORM>(unit, p, first, blk, krank, group);
    float* part = reinterpret_cast<float*>(smem);
    bool ok = true;
    if (warp >= 4 && mine && T.kbeg < T.kend) {
      ok = wait_bar(bar(L::T_FULL), 0, abort_flag, p);
      tc_fence_after();
      for (int a = 0; a < halves; ++a)
        for (int c = 32 * eh; c < T.cols; c += 64) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(t_lane + static_cast<uint32_t>(a * BC + c), v);
          tmem_wait_ld(v);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            part[(a * BC + c + j) * 128 + q * 32 + lane] = __uint_as_float(v[j]);
        }
    }
    __syncwarp();
    cluster_sync();
    if (warp >= 4 && mine) {
      // ranks that had slots of the reduction
      const long long nk = T.nk;
      const uint32_t has = __ballot_sync(
          0xffffffffu, lane < p.split && nk * lane / p.split < nk * (lane + 1) / p.split);
      const uint32_t flag = smem_u32(misc + 1);
      if (p.split <= 2) add_partials<PAIR, BC, TN, 2>(p, T, sbase, has, flag, ok, krank, side, halves);
      else if (p.split <= 4) add_partials<PAIR, BC, TN, 4>(p, T, sbase, has, flag, ok, krank, side, halves);
      else add_partials<PAIR, BC, TN, 8>(p, T, sbase, has, flag, ok, krank, side, halves);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, 2 * ACC);
    else tmem_dealloc(tmem, 2 * ACC);
  }
  // no CTA leaves while a peer may still signal it or read its shared memory: the
  // arrival is a release, which a read of a peer's partial or flag comes before
  // even where nothing has used its value yet
  if (cluster > 1) {
    __syncwarp();
    cluster_sync();
  }
}

// Estimated time of a plan beyond the launch (us), for the choice between
// plans only.  The groups' sizes are on the device: one group stands for all, at
// 1.3 times the average rows (some get none).  Constants fitted to timings of
// every plan below on 3700 shapes drawn over 1 to 64 groups, 1 to 32647 rows and
// widths of 256 to 8192, all forms: the choice is 3.6% slower than the best plan
// on average, on as many others too (splits of 3, 5 and 6 as well would gain 0.2%).
//  * a slot costs a pair 0.33 us (64 deep), the single form (128 deep) 0.08 us, 2.6
//    ns per lane and 2 ns per row of A: what they take to load;
//  * a tile's epilogue 3.7 ns per row of D and 128 lanes, hidden behind the next
//    tile but for the last one;
//  * a split adds 2.2 us (partials written, a cluster barrier, a round of reads)
//    and 0.2 ns per partial that a CTA reads from the others, and large clusters
//    leave SMs empty;
//  * memory 8.3 TB/s over what is read and written once (weights in L2 count in).
double bf_cost(const BfCall& c, const BfPlan& f, int num_sms) {
  const bool tn = c.form == kBfTN;
  const double groups = tn ? c.G : std::min(c.G, c.rows), fill = groups > 1 ? 1.3 : 1.0;
  const double per = tn ? c.M : fill * c.rows / groups;       // rows of D in a group
  const double depth = tn ? fill * c.rows / c.G : c.K;
  const int cluster = (f.pair ? 2 : 1) * f.split;
  const double room = std::max(
      1.0, std::floor(num_sms * (cluster >= 8 ? 0.55 : cluster >= 4 ? 0.8 : 1.0) / cluster));
  const double tiles = groups * std::ceil(per / f.bc) * ((c.N + f.lanes - 1) / f.lanes);
  const double waves = std::max(1.0, std::ceil(tiles / room));
  const int halves = f.pair ? 1 : (f.lanes + 127) / 128;
  const double cols = std::min<double>(f.bc, per);
  const double slots = std::max(1.0, std::ceil(depth / bf_bk(f.pair) / f.split));
  const double main = slots * (f.pair ? 0.33 : 0.08 + 0.0026 * f.lanes + 0.002 * f.bc);
  const double epilogue = 0.0037 * cols * halves;
  const double run = main + epilogue + (waves - 1) * std::max(main, epilogue);
  const double N = c.N, K = c.K, M = c.M, T = c.rows;
  const double memory =
      2 * (tn ? c.G * M * N + T * (M + N) : groups * N * K + T * (N + K)) / 8.3e6;
  return std::max(run, memory) + 0.12 * std::min(run, memory) +
         (f.split > 1 ? 2.2 + 2e-4 * 128 * halves * cols * (f.split - 1) / f.split : 0.0);
}

// Tiles of `lanes` columns and `bc` rows of D that the call can have at most.
long long bf_most_tiles(const BfCall& c, int lanes, int bc) {
  const long long nl = (c.N + lanes - 1) / lanes;
  return nl * (c.form == kBfTN ? static_cast<long long>(c.G) * ((c.M + bc - 1) / bc)
                               : std::min<long long>(c.G, c.rows) + c.rows / bc);
}

BfPlan bf_plan(const BfCall& c, int num_sms) {
  const bool tn = c.form == kBfTN;
  const int per = tn ? c.M : (c.rows + std::min(c.G, c.rows) - 1) / std::max(1, std::min(c.G, c.rows));
  const int depth = tn ? c.rows / c.G : c.K;
  BfPlan best{false, 128, 64, 1};
  double least = 1e300;
  auto consider = [&](bool pair, int lanes, int bc) {
    const int width = pair ? 2 : 1;
    for (int split = 1; split * width <= kBfMaxCluster && (split == 1 || depth >= 128 * split); split *= 2) {
      if (split * width > num_sms) break;   // (a limit on the SMs may leave fewer)
      const BfPlan f{pair, lanes, bc, split};
      if (c.limited && bf16_grid(c, f, num_sms) > num_sms) break;   // (a cluster per tile)
      const double t = bf_cost(c, f, num_sms);
      if (t < least) {
        least = t;
        best = f;
      }
    }
  };
  if (per > 32) consider(true, 256, 256);
  // rows of D per tile near the average group's (tn: whole 64-wide boxes)
  for (int bc = tn ? 64 : 16; bc <= 128; bc *= 2) {
    if (!tn && (per > 4 * bc || (bc > 16 && per < bc / 4))) continue;
    for (int lanes = 128; lanes <= 256 && lanes - 64 < c.N; lanes += 64) consider(false, lanes, bc);
  }
  return best;
}

template <bool PAIR, int BC, int FORM>
cudaError_t launch_tiles(const BfCall& c, PFN_cuTensorMapEncodeTiled_v12000 encode,
                         const BfPlan& plan, int num_sms, cudaStream_t stream) {
  constexpr bool tn = FORM == kBfTN;
  const int lanes = plan.lanes, bc = plan.bc, split = plan.split;
  constexpr int BK = bf_bk(PAIR);
  BfParams p{};
  p.G = c.G;
  p.rows = c.rows;
  p.M = c.M;
  p.N = c.N;
  p.K = c.K;
  p.lanes = lanes;
  p.nl = (c.N + lanes - 1) / lanes;
  p.bc = bc;
  p.nc = tn ? (c.M + bc - 1) / bc : 0;
  p.split = split;
  p.inv_nl = bf_inverse(p.nl);
  p.inv_band = bf_inverse(BF_BAND * p.nl);
  p.inv_per = tn ? bf_inverse(p.nc * p.nl) : 0;
  const int p_rows = PAIR ? 128 : lanes, q_rows = PAIR ? bc / 2 : bc;
  p.p_bytes = p_rows * BK * 2;
  p.q_bytes = q_rows * BK * 2;
  p.stages = std::min(BF_MAX_STAGES, (kBfMaxSmem - BfSmem::fixed(c.G)) / (p.p_bytes + p.q_bytes));
  p.sizes = c.sizes;
  p.D = static_cast<uint16_t*>(c.D);
  p.C = static_cast<const uint16_t*>(c.C);
  p.status = c.status;
  p.timeout_ns = c.timeout_ns;
  p.debug_flags = c.debug_flags;

  // bf16 tensor map of four dimensions (innermost first), 128-byte swizzle
  auto map = [&](CUtensorMap* m, const void* x, const cuuint64_t (&dims)[4],
                 const cuuint64_t (&strides)[3], const cuuint32_t (&box)[4]) {
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x), dims, strides, box,
                  one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  // A slot of a K-major operand [z][rows][K] is BK / 64 pieces of 64 (K) x box
  // rows, one of an MN-major operand [z][K][width] is box / 64 pieces of 64
  // (width) x BK rows of K.  One load takes them all, with the pieces as the third
  // dimension of a map of the whole pieces; where the extent is no multiple of
  // 64, its edge needs the other map, a load per piece.
  auto operand = [&](CUtensorMap* m, int* whole, const void* x, bool mn, uint64_t z, uint64_t rows,
                     uint64_t k, uint32_t box) {
    const uint64_t wide = mn ? rows : k, deep = mn ? k : rows, all = 2 * wide * deep;
    const uint32_t pieces = mn ? box / 64 : BK / 64, height = mn ? BK : box;
    *whole = static_cast<int>(wide / 64 * 64);
    if (!map(m + 1, x, {wide, deep, 1, z}, {2 * wide, all, all}, {64, height, 1, 1})) return false;
    if (*whole == 0) {
      m[0] = m[1];   // (never used)
      return true;
    }
    return map(m, x, {64, deep, wide / 64, z}, {2 * wide, 128, all}, {64, height, pieces, 1});
  };
  BfMaps maps;
  // (a reduction without rows loads nothing; its maps still need an extent)
  const uint64_t rows = std::max(c.rows, 1);
  const bool good =
      (tn ? operand(maps.p, &p.p_whole, c.B, true, 1, c.N, rows, p_rows)
          : operand(maps.p, &p.p_whole, c.B, FORM == kBfNN, c.G, c.N, c.K, p_rows)) &&
      (tn ? operand(maps.q, &p.q_whole, c.A, true, 1, c.M, rows, q_rows)
          : operand(maps.q, &p.q_whole, c.A, false, 1, rows, c.K, q_rows));
  if (!good) return cudaErrorInvalidValue;

  const int cluster = (PAIR ? 2 : 1) * split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(bf16_grid(c, plan, num_sms)), 1, 1);
  cfg.blockDim = dim3(BF_THREADS, 1, 1);
  cfg.dynamicSmemBytes = p.stages * (p.p_bytes + p.q_bytes) + BfSmem::fixed(c.G);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, bf16_grouped_kernel<PAIR, BC, FORM>, maps, p);
}

template <int FORM>
cudaError_t set_up_form() {
  const void* kernels[] = {reinterpret_cast<const void*>(bf16_grouped_kernel<true, 256, FORM>),
                           reinterpret_cast<const void*>(bf16_grouped_kernel<false, 128, FORM>),
                           reinterpret_cast<const void*>(bf16_grouped_kernel<false, 64, FORM>)};
  for (const void* k : kernels) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kBfMaxSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int FORM>
cudaError_t launch_form(const BfCall& c, PFN_cuTensorMapEncodeTiled_v12000 encode, int num_sms,
                        cudaStream_t stream) {
  const BfPlan f = c.forced.lanes > 0 ? c.forced : bf_plan(c, num_sms);
  return f.pair       ? launch_tiles<true, 256, FORM>(c, encode, f, num_sms, stream)
         : f.bc <= 64 ? launch_tiles<false, 64, FORM>(c, encode, f, num_sms, stream)
                      : launch_tiles<false, 128, FORM>(c, encode, f, num_sms, stream);
}

}  // namespace

// As many CTAs (pairs) as there can be tiles, at most one per SM; with a split
// reduction a cluster for each of them.
long long bf16_grid(const BfCall& c, const BfPlan& f, int num_sms) {
  const long long most = bf_most_tiles(c, f.lanes, f.bc);
  const int width = f.pair ? 2 : 1;
  return std::max(1ll, f.split > 1 ? most : std::min<long long>(most, num_sms / width)) * width * f.split;
}

cudaError_t bf16_set_up() {
  cudaError_t e = set_up_form<kBfNT>();
  if (e == cudaSuccess) e = set_up_form<kBfNN>();
  if (e == cudaSuccess) e = set_up_form<kBfTN>();
  return e;
}

cudaError_t launch_bf16_grouped(const BfCall& c, PFN_cuTensorMapEncodeTiled_v12000 encode,
                                int num_sms, cudaStream_t stream) {
  switch (c.form) {
    case kBfNT: return launch_form<kBfNT>(c, encode, num_sms, stream);
    case kBfNN: return launch_form<kBfNN>(c, encode, num_sms, stream);
    default: return launch_form<kBfTN>(c, encode, num_sms, stream);
  }
}

}  // namespace dgk
