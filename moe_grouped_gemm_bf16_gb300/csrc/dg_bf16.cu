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
// BC rows of D on its columns (A is the second operand).  The ragged dimension
// of nt and nn is then the MMA's N, which the instruction takes in steps of
// 16 or 32: a group of 20 rows costs 32 columns, not 128 lanes, and a weight
// tile is always full.
//
// Two kernels:
//  * PAIR: a persistent CTA pair per 256 x 256 tile (cta_group::2: each CTA
//    holds 128 lanes of B and half of A's rows), for groups of many rows;
//  * single: one persistent CTA per tile of up to 256 lanes x BC rows, for
//    groups of few rows, where the time is that of reading the weights: the
//    host picks the lanes so that the tiles fill the SMs once (all of them
//    stream at HBM's rate and end together).
//
// Warps 0 and 2 load by TMA (B's tile and A's) into a ring of slots 64 deep in
// the reduction, warp 1 (of the pair's leader) issues tcgen05.mma kind::f16
// into one of two fp32 accumulators in tensor memory, warps 4-7 round the
// other one to bf16 and store it.  tn's reduction ends at a group's last row,
// which need not end a slot: warp 3 zeroes the rows behind it, up to the next
// multiple of the MMA's 16, in both operands (the next group's rows may hold
// anything).
//
// Every wait is bounded, as in the FP8 kernels.
#include <algorithm>

#include "dg_bf16.h"
#include "dg_params.h"
#include "dg_wait.cuh"
#include "ptx.cuh"

namespace dgk {
namespace {

constexpr int BK = 64;          // reduction depth per slot (128 bytes)
constexpr int BF_THREADS = 256;
constexpr int BF_BAND = 8;      // column blocks (rows of D) per raster band
constexpr int BF_MAX_STAGES = 12;
constexpr int kBfMaxSmem = 232448;

struct BfParams {
  int G;
  int rows;        // rows of A over all groups
  int M;           // tn: rows of each D[e]
  int N;           // columns of D
  int nk;          // nt, nn: 64-deep slots of the reduction
  int lanes;       // columns of D per tile (pair: 256)
  int nl;          // lane blocks: ceil(N / lanes)
  int nc;          // tn: column blocks of each group: ceil(M / BC)
  int stages;
  int p_bytes;     // bytes of a slot's lane operand (per CTA)
  int q_bytes;     // bytes of a slot's column operand (per CTA)
  int p_split;     // lane operand loaded in 64-wide boxes (N not a multiple of 64)
  int q_split;     // column operand (tn) loaded in 64-wide boxes (M not a multiple of 64)
  const int32_t* sizes;
  uint16_t* D;
  const uint16_t* C;
  unsigned int* status;
  unsigned long long timeout_ns;
  unsigned int debug_flags;
};

// Shared memory behind the ring: barriers, TMEM base and abort flag, then the
// groups' first rows and first column blocks.
struct BfSmem {
  static constexpr int FULL = 0, EMPTY = BF_MAX_STAGES, TAIL = 2 * BF_MAX_STAGES,
                       T_FULL = 3 * BF_MAX_STAGES, T_EMPTY = T_FULL + 2, MMA_DONE = T_EMPTY + 2,
                       NUM_BARS = MMA_DONE + 1;
  static constexpr int MISC = NUM_BARS * 8;
  static constexpr int TAB = (MISC + 8 + 15) / 16 * 16;
  __host__ __device__ static constexpr int fixed(int G) { return 1024 + TAB + 2 * (G + 1) * 4; }
};

struct BfTile {
  int g;       // group
  int l0;      // first column of D
  int cols;    // rows of D in this tile
  int q0;      // first row of the column operand (nt, nn: row of A; tn: m)
  int k0;      // tn: first row of the group
  int kn;      // reduction length (nt, nn: all of K, in whole slots)
  int nk;      // slots
};

template <int BC, int FORM>
__device__ __forceinline__ BfTile bf_tile(int t, const BfParams& p, const int* first,
                                          const int* blk) {
  BfTile T;
  int nc;
  if (FORM == kBfTN) {
    const int per = p.nc * p.nl;
    T.g = t / per;
    t -= T.g * per;
    nc = p.nc;
  } else {
    // largest g with blk[g] * nl <= t
    int lo = 0, hi = p.G - 1;
    const int b = t / p.nl;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (blk[mid] <= b) lo = mid; else hi = mid - 1;
    }
    T.g = lo;
    t -= blk[lo] * p.nl;
    nc = blk[lo + 1] - blk[lo];
  }
  // bands of BF_BAND column blocks; within a band first along the column
  // blocks, then along the lanes, so that concurrent tiles share operands in L2
  const int band = t / (BF_BAND * p.nl);
  const int r = t - band * BF_BAND * p.nl;
  const int h = min(BF_BAND, nc - band * BF_BAND);
  T.l0 = (r / h) * p.lanes;
  const int c0 = (band * BF_BAND + r % h) * BC;
  const int n = first[T.g + 1] - first[T.g];
  if (FORM == kBfTN) {
    T.cols = min(BC, p.M - c0);
    T.q0 = c0;
    T.k0 = first[T.g];
    T.kn = n;
    T.nk = (n + BK - 1) / BK;
  } else {
    T.cols = min(BC, n - c0);
    T.q0 = first[T.g] + c0;
    T.k0 = 0;
    T.kn = p.nk * BK;
    T.nk = p.nk;
  }
  return T;
}

template <bool PAIR, int BC, int FORM>
__global__ void __launch_bounds__(BF_THREADS, 1)
bf16_grouped_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                    const BfParams p) {
  using L = BfSmem;
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
  int* first = reinterpret_cast<int*>(smem + ring + L::TAB);
  int* blk = first + p.G + 1;
  const uint32_t crank = PAIR ? cluster_ctarank() : 0;
  const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x, units = PAIR ? gridDim.x >> 1 : gridDim.x;
  constexpr bool TN = FORM == kBfTN, P_MN = FORM != kBfNT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      // the two producers (pair: the leader's, for both CTAs' bytes)
      mbar_init(bar(L::FULL + s), 2);
      mbar_init(bar(L::EMPTY + s), 1);
      mbar_init(bar(L::TAIL + s), 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(L::T_FULL + b), 1);
      mbar_init(bar(L::T_EMPTY + b), PAIR ? 8 : 4);
    }
    mbar_init(bar(L::MMA_DONE), 1);
    misc[1] = 0;
    fence_mbarrier_init();
    prefetch_tmap(&tmP);
    prefetch_tmap(&tmQ);
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
      int c = (mine + BC - 1) / BC;
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
  // the peer signals this CTA's barriers from here on (their initialisation was
  // made visible to the cluster by thread 0's fence)
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
  // a tile's last slot needs zeroed rows (tn)
  auto ragged = [&](const BfTile& T) { return TN && (T.kn & 15) != 0; };

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------- TMA producers --
    // warp 0: the lane operand (B), warp 2: the column operand (A); one load
    // each per slot (a thread that issues one stalls for ~250 cycles)
    if (lane == 0 && !(p.debug_flags & DBG_SKIP_PRODUCER)) {
      const bool lanes_op = warp == 0;
      const CUtensorMap* tm = lanes_op ? &tmP : &tmQ;
      const bool mn = lanes_op ? P_MN : TN;
      const bool split = lanes_op ? p.p_split : p.q_split;
      const uint32_t bytes = lanes_op ? p.p_bytes : p.q_bytes;
      const uint32_t base = sbase + (lanes_op ? 0 : q_off);
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0, tails = 0, tail_par = 0;
      for (int t = unit; t < tiles; t += units) {
        const BfTile T = bf_tile<BC, FORM>(t, p, first, blk);
        const int at = lanes_op ? T.l0 + static_cast<int>(crank) * 128
                                : T.q0 + static_cast<int>(crank) * (mma_n(T.cols) / 2);
        const int g = (lanes_op && !TN) ? T.g : 0;
        const bool rag = ragged(T);
        for (int i = 0; i < T.nk; ++i) {
          bool go = wait_bar(bar(L::EMPTY + s), ph ^ 1, abort_flag, p);
          const int k = T.k0 + i * BK;
          if constexpr (kDebug) {
            const int rows = lanes_op ? p.N : (TN ? p.M : p.rows);
            // (a pair's second CTA may start past the tensor: zero-filled)
            if (go && (T.g >= p.G || at < 0 || at >= rows + (PAIR ? 128 : 0) || k < 0 ||
                       (TN && k >= p.rows))) {
              dbg_fail(p, ST_DEBUG_BOUNDS, abort_flag);
              go = false;
            }
          }
          if (go) {
            const uint32_t dst = base + s * bytes;
            // a slot whose rows warp 3 completes arrives on its own CTA's TAIL
            const bool to_tail = rag && i == T.nk - 1;
            const uint32_t b = to_tail ? bar(L::TAIL + s)
                               : PAIR  ? map_cluster(bar(L::FULL + s), 0)
                                       : bar(L::FULL + s);
            // the leader expects both CTAs' bytes (a remote arrival of the peer
            // at cluster scope would cost it a microsecond per slot)
            if (to_tail || crank == 0)
              mbar_arrive_expect_tx(to_tail ? b : bar(L::FULL + s), PAIR && !to_tail ? 2 * bytes : bytes);
            auto load = [&](uint32_t d, int x, int y, int z) {
              if (PAIR && !to_tail) tma_load_4d_pair(map_cluster(d, crank), tm, b, x, y, z, g);
              else tma_load_4d(d, tm, b, x, y, z, g);
            };
            if (!mn) {
              load(dst, k, at, 0);
            } else if (!split) {
              load(dst, 0, k, at >> 6);
            } else {
              for (uint32_t j = 0; j < bytes / 8192; ++j) load(dst + j * 8192, at + 64 * j, k, 0);
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
        if (((issued >> q) & 1u) && (!PAIR || crank == 0))
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
    if (crank == 0) {
      const bool issuer = elect_one();
      // a K step of 16: 32 bytes inside a K-major row, two 8-row atoms (2 KB) of
      // an MN-major slot, whose 64-wide atoms lie 64 rows x 128 bytes apart
      constexpr uint64_t P_STEP = (P_MN ? 2048 : 32) >> 4, Q_STEP = (TN ? 2048 : 32) >> 4;
      const bool two = !PAIR && p.lanes > 128;
      int s = 0, b = 0;
      uint32_t ph = 0, bph = 0;
      for (int t = unit; t < tiles; t += units) {
        const BfTile T = bf_tile<BC, FORM>(t, p, first, blk);
        if (T.nk == 0) continue;
        const uint32_t idesc = idesc_bf16_f32(PAIR ? 256 : 128, mma_n(T.cols), P_MN, TN);
        const uint32_t d = tmem + static_cast<uint32_t>(b * ACC);
        bool ok = wait_bar(bar(L::T_EMPTY + b), bph ^ 1, abort_flag, p);
        tc_fence_after();
        for (int i = 0; i < T.nk; ++i) {
          // (the peer's warp 3 wrote a ragged slot's zeros itself)
          const bool zeroed = PAIR && i == T.nk - 1 && ragged(T);
          ok = (zeroed ? wait_bar<true>(bar(L::FULL + s), ph, abort_flag, p)
                       : wait_bar(bar(L::FULL + s), ph, abort_flag, p)) && ok;
          tc_fence_after();
          if (issuer && ok) {
            const uint32_t ps = sbase + s * p.p_bytes, qs = sbase + q_off + s * p.q_bytes;
            const uint64_t pd = P_MN ? smem_desc_sw128_mnmajor(ps, 8192) : smem_desc_sw128_kmajor(ps);
            const uint64_t qd = TN ? smem_desc_sw128_mnmajor(qs, 8192) : smem_desc_sw128_kmajor(qs);
            auto step = [&](int kk, uint32_t acc) {
              if constexpr (PAIR) {
                mma_bf16_pair(d, pd + P_STEP * kk, qd + Q_STEP * kk, idesc, acc);
              } else {
                mma_bf16(d, pd + P_STEP * kk, qd + Q_STEP * kk, idesc, acc);
                // the second 128 lanes (the rows past `lanes` are not stored)
                if (two) mma_bf16(d + BC, pd + (16384 >> 4) + P_STEP * kk, qd + Q_STEP * kk, idesc, acc);
              }
            };
            const int left = T.kn - i * BK;
            if (!TN || left >= BK) {
              step(0, i > 0);
#pragma unroll
              for (int kk = 1; kk < BK / 16; ++kk) step(kk, 1);
            } else {
              for (int kk = 0; 16 * kk < left; ++kk) step(kk, i > 0 || kk > 0);
            }
            if constexpr (PAIR) mma_commit_pair_multicast(bar(L::EMPTY + s), 0x3);
            else mma_commit(bar(L::EMPTY + s));
            if (i == T.nk - 1) {
              if constexpr (PAIR) mma_commit_pair_multicast(bar(L::T_FULL + b), 0x3);
              else mma_commit(bar(L::T_FULL + b));
            }
          }
          __syncwarp();
          if (++s == p.stages) { s = 0; ph ^= 1; }
        }
        b ^= 1;
        if (b == 0) bph ^= 1;
      }
      if (issuer) {
        if constexpr (PAIR) mma_commit_pair_multicast(bar(L::MMA_DONE), 0x1);
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
        const BfTile T = bf_tile<BC, FORM>(t, p, first, blk);
        if (T.nk == 0) continue;
        s = (s + T.nk - 1) % p.stages;
        if (ragged(T)) {
          // all 32 lanes: wait for this CTA's two loads, then zero the rows
          // behind the group's last one, up to the next multiple of 16 (a row
          // is one 128-byte line of each 64-wide atom)
          const bool ok = wait_bar(bar(L::TAIL + s), (par >> s) & 1u, abort_flag, p);
          par ^= 1u << s;
          if (ok) {
            const int left = T.kn - (T.nk - 1) * BK, r = ((left + 15) & ~15) - left;
            const int pa = p.p_bytes / 8192, n = r * 8 * (pa + p.q_bytes / 8192);
            const uint32_t ps = sbase + s * p.p_bytes, qs = sbase + q_off + s * p.q_bytes;
            for (int u = lane; u < n; u += 32) {
              const int atom = u / (r * 8), w = u - atom * (r * 8);
              const uint32_t base = atom < pa ? ps + atom * 8192 : qs + (atom - pa) * 8192;
              st_shared_v4(base + (left + (w >> 3)) * 128 + (w & 7) * 16, 0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          // in place of the two producers' arrivals: one per CTA of a pair, or two
          if constexpr (PAIR) {
            if (lane == 0) mbar_arrive_remote_release(bar(L::FULL + s), 0);
          } else {
            if (lane < 2) mbar_arrive(bar(L::FULL + s));
          }
        }
        s = (s + 1) % p.stages;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue --
    const int q = warp & 3;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int halves = PAIR ? 1 : (p.lanes + 127) / 128;
    int b = 0;
    uint32_t bph = 0;
    for (int t = unit; t < tiles; t += units) {
      const BfTile T = bf_tile<BC, FORM>(t, p, first, blk);
      const bool have = T.nk > 0;
      const bool ok = !have || wait_bar(bar(L::T_FULL + b), bph, abort_flag, p);
      tc_fence_after();
      const size_t row0 = TN ? static_cast<size_t>(T.g) * p.M + T.q0 : static_cast<size_t>(T.q0);
      const int l_end = min(p.N, T.l0 + p.lanes);
      for (int a = 0; a < halves; ++a) {
        // this thread's pair of columns of D (lanes l and l ^ 1 share them)
        const int l = T.l0 + (PAIR ? static_cast<int>(crank) : a) * 128 + q * 32 + (lane & ~1);
        for (int c = 0; c < T.cols; c += 32) {
          uint32_t v[32];
          if (have) {
            tmem_ld_32x32b_x32(t_lane + static_cast<uint32_t>(b * ACC + a * BC + c), v);
            tmem_wait_ld(v);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
          }
          // a lane holds 32 rows of one column of D: exchange with the
          // neighbouring lane, so that the even lane stores two columns of row
          // j and the odd one those of row j + 1
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint32_t give = (lane & 1) ? v[j] : v[j + 1];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
            float lo = __uint_as_float((lane & 1) ? got : v[j]);
            float hi = __uint_as_float((lane & 1) ? v[j + 1] : got);
            const int r = c + j + (lane & 1);
            if (ok && r < T.cols && l < l_end) {
              const size_t at = (row0 + r) * p.N + l;
              if constexpr (kDebug) {
                if (row0 + r >= static_cast<size_t>(TN ? p.G * static_cast<long long>(p.M) : p.rows)) {
                  raise_status(p, ST_DEBUG_BOUNDS);
                  continue;
                }
              }
              if (p.C) {
                // the addend in fp32, then one rounding
                const uint32_t cw = *reinterpret_cast<const uint32_t*>(p.C + at);
                lo += __uint_as_float(cw << 16);
                hi += __uint_as_float(cw & 0xFFFF0000u);
              }
              *reinterpret_cast<uint32_t*>(p.D + at) = pack_bf16x2(lo, hi);
            }
          }
        }
      }
      if (have) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR && crank != 0) mbar_arrive_remote_relaxed(bar(L::T_EMPTY + b), 0);
          else mbar_arrive(bar(L::T_EMPTY + b));
        }
        b ^= 1;
        if (b == 0) bph ^= 1;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, 2 * ACC);
    else tmem_dealloc(tmem, 2 * ACC);
  }
  // no CTA leaves while its peer may still signal it or read its operands
  if constexpr (PAIR) cluster_sync_relaxed();
}

template <bool PAIR, int BC, int FORM>
cudaError_t launch_tiles(const BfCall& c, PFN_cuTensorMapEncodeTiled_v12000 encode, int lanes,
                         int num_sms, cudaStream_t stream) {
  constexpr bool tn = FORM == kBfTN;
  BfParams p{};
  p.G = c.G;
  p.rows = c.rows;
  p.M = c.M;
  p.N = c.N;
  p.nk = tn ? 0 : (c.K + BK - 1) / BK;
  p.lanes = lanes;
  p.nl = (c.N + lanes - 1) / lanes;
  p.nc = tn ? (c.M + BC - 1) / BC : 0;
  const int p_rows = PAIR ? 128 : lanes, q_rows = PAIR ? BC / 2 : BC;
  p.p_bytes = (p_rows * 128 + 1023) / 1024 * 1024;
  p.q_bytes = q_rows * 128;
  p.stages = std::min(BF_MAX_STAGES, (kBfMaxSmem - BfSmem::fixed(c.G)) / (p.p_bytes + p.q_bytes));
  p.p_split = c.N % 64 != 0;
  p.q_split = c.M % 64 != 0;
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
  // A K-major operand [z][rows][K] is read in boxes of 64 (K) x rows; an
  // MN-major one [z][K][width] in boxes of 64 (width) x 64 rows of K, several
  // side by side in one load where the width is a multiple of 64.
  auto k_major = [&](CUtensorMap* m, const void* x, uint64_t z, uint64_t rows, uint64_t k,
                     uint32_t box) {
    return map(m, x, {k, rows, 1, z}, {2 * k, 2 * k * rows, 2 * k * rows}, {BK, box, 1, 1});
  };
  auto mn_major = [&](CUtensorMap* m, const void* x, uint64_t z, uint64_t k, uint64_t width,
                      uint32_t box) {
    const uint64_t all = 2 * width * k;
    if (width % 64 != 0) return map(m, x, {width, k, 1, z}, {2 * width, all, all}, {64, BK, 1, 1});
    return map(m, x, {64, k, width / 64, z}, {2 * width, 128, all}, {64, BK, box / 64, 1});
  };
  CUtensorMap mp, mq;
  // (a reduction without rows loads nothing; its maps still need an extent)
  const uint64_t G = c.G, N = c.N, K = c.K, R = std::max(c.rows, 1);
  const bool good =
      (FORM == kBfNT   ? k_major(&mp, c.B, G, N, K, p_rows)
       : FORM == kBfNN ? mn_major(&mp, c.B, G, K, N, p_rows)
                         : mn_major(&mp, c.B, 1, R, N, p_rows)) &&
      (tn ? mn_major(&mq, c.A, 1, R, c.M, q_rows) : k_major(&mq, c.A, 1, R, K, q_rows));
  if (!good) return cudaErrorInvalidValue;

  // as many CTAs (pairs) as there can be tiles, at most one per SM
  const long long most = tn ? static_cast<long long>(c.G) * p.nc * p.nl
                            : (std::min<long long>(c.G, c.rows) + c.rows / BC) * p.nl;
  const long long fit = PAIR ? num_sms / 2 : num_sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::max(1ll, std::min(most, fit)) * (PAIR ? 2 : 1)), 1, 1);
  cfg.blockDim = dim3(BF_THREADS, 1, 1);
  cfg.dynamicSmemBytes = p.stages * (p.p_bytes + p.q_bytes) + BfSmem::fixed(c.G);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (PAIR) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, bf16_grouped_kernel<PAIR, BC, FORM>, mp, mq, p);
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
  constexpr bool tn = FORM == kBfTN;
  // rows of D that a group has: the average (nt, nn), M (tn)
  const long long per = tn ? c.M : (c.rows + c.G - 1) / c.G;
  const long long groups = tn ? c.G : std::min(c.G, c.rows);
  // (a limit on the SMs may leave a single one: no pair fits)
  if (per > 128 && num_sms >= 2)
    return launch_tiles<true, 256, FORM>(c, encode, 256, num_sms, stream);
  // lanes such that the tiles fill the SMs once, in whole MMA boxes: 64 where
  // the lane operand is MN-major, else 16
  const int bc = per > 64 ? 128 : 64, step = FORM == kBfNT ? 16 : 64;
  const long long cols = groups * ((per + bc - 1) / bc);
  const long long blocks = std::max(1ll, num_sms / cols);   // lane blocks per column block
  const long long want = ((c.N + blocks - 1) / blocks + step - 1) / step * step;
  const int lanes = static_cast<int>(std::min(256ll, std::max(64ll, want)));
  return bc == 128 ? launch_tiles<false, 128, FORM>(c, encode, lanes, num_sms, stream)
                   : launch_tiles<false, 64, FORM>(c, encode, lanes, num_sms, stream);
}

}  // namespace

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
