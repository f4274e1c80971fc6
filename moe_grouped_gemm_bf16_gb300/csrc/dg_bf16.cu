// bf16 products grouped by expert with ragged sizes, for sm_103a.  The groups'
// rows lie one after the other in A (group e owns sizes[e] rows, any number,
// read on the device):
//
//   nt  D[t][n]    = sum_k A[t][k] B[e][n][k]     forward, t in group e
//   nn  D[t][n]    = sum_k A[t][k] B[e][k][n]     gradient of the activations
//   tn  D[e][m][n] = C[e][m][n] + sum_{t in e} A[t][m] B[t][n]   gradient of the weights
//
// Every form is one computation: a tile of D with BL = 128 consecutive columns
// of a row of D on the tensor memory's lanes (B is the MMA's first operand)
// and up to BC rows of D on its columns (A is the second operand).  The ragged
// dimension of nt and nn is then the MMA's N, which the instruction takes in
// steps of 16: a group of 20 rows costs 32 columns, not 128 lanes, and a
// weight tile is always full.
//
// One persistent CTA per SM; warp 0 loads by TMA into a ring of STAGES slots
// (64 deep in the reduction), warp 1 issues tcgen05.mma kind::f16 into one of
// two fp32 accumulators in tensor memory, warps 4-7 round the other one to
// bf16 and store it.  tn's reduction ends at a group's last row, which need
// not end a 64-row slot: the rows behind it, up to the next multiple of the
// MMA's 16, are zeroed in shared memory (in both operands: the next group's
// rows may hold anything).
//
// Every wait is bounded, as in the FP8 kernels.
#include <algorithm>

#include "dg_bf16.h"
#include "dg_params.h"
#include "dg_wait.cuh"
#include "ptx.cuh"

namespace dgk {
namespace {

constexpr int BL = 128;      // lanes: columns of D per tile
constexpr int BK = 64;       // reduction depth per slot (128 bytes)
constexpr int BF_THREADS = 256;
constexpr int BF_BAND = 8;   // column blocks (rows of D) per raster band

struct BfParams {
  int form;
  int G;
  int rows;        // rows of A over all groups
  int M;           // tn: rows of each D[e]
  int N;           // columns of D
  int nk;          // nt, nn: 64-deep slots of the reduction
  int nl;          // lane blocks: ceil(N / BL)
  int nc;          // tn: column blocks of each group: ceil(M / BC)
  int p_split;     // lane operand loaded in 64-wide boxes (N not a multiple of 64)
  int q_split;     // column operand (tn) loaded in 64-wide boxes (M not a multiple of 64)
  const int32_t* sizes;
  uint16_t* D;
  const uint16_t* C;
  unsigned int* status;
  unsigned long long timeout_ns;
  unsigned int debug_flags;
};

template <int BC, int STAGES>
struct BfSmem {
  static constexpr int P_BYTES = BL * BK * 2;
  static constexpr int Q_BYTES = BC * BK * 2;
  static constexpr int P_OFF = 0;
  static constexpr int Q_OFF = STAGES * P_BYTES;
  static constexpr int BAR_OFF = Q_OFF + STAGES * Q_BYTES;
  static constexpr int FULL = 0, EMPTY = STAGES, T_FULL = 2 * STAGES, T_EMPTY = T_FULL + 2,
                       MMA_DONE = T_EMPTY + 2, NUM_BARS = MMA_DONE + 1;
  static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;   // TMEM base, abort flag
  static constexpr int TAB_OFF = (MISC_OFF + 8 + 15) / 16 * 16;
  // first row of each group, then first column block of each group
  static constexpr int bytes(int G) { return 1024 + TAB_OFF + 2 * (G + 1) * 4; }
  static constexpr int TMEM_COLS = 2 * BC < 32 ? 32 : 2 * BC;
};

struct BfTile {
  int g;       // group
  int l0;      // first column of D
  int c0;      // first row of D within the group (nt, nn: row of the group; tn: m)
  int cols;    // rows of D in this tile
  int q0;      // first row of the column operand (nt, nn: row of A; tn: m)
  int k0;      // tn: first row of the group
  int kn;      // reduction length (nt, nn: all of K, in whole slots)
  int nk;      // slots
};

template <int BC>
__device__ __forceinline__ BfTile bf_tile(int t, const BfParams& p, const int* first,
                                          const int* blk) {
  BfTile T;
  int nc;
  if (p.form == kBfTN) {
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
  T.l0 = (r / h) * BL;
  T.c0 = (band * BF_BAND + r % h) * BC;
  const int n = first[T.g + 1] - first[T.g];
  if (p.form == kBfTN) {
    T.cols = min(BC, p.M - T.c0);
    T.q0 = T.c0;
    T.k0 = first[T.g];
    T.kn = n;
    T.nk = (n + BK - 1) / BK;
  } else {
    T.cols = min(BC, n - T.c0);
    T.q0 = first[T.g] + T.c0;
    T.k0 = 0;
    T.kn = p.nk * BK;
    T.nk = p.nk;
  }
  return T;
}

template <int BC, int STAGES>
__global__ void __launch_bounds__(BF_THREADS, 1)
bf16_grouped_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                    const BfParams p) {
  using L = BfSmem<BC, STAGES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sbase + L::BAR_OFF + 8 * i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  volatile uint32_t* abort_flag = misc + 1;
  int* first = reinterpret_cast<int*>(smem + L::TAB_OFF);
  int* blk = first + p.G + 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar(L::FULL + s), 1);
      mbar_init(bar(L::EMPTY + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(L::T_FULL + b), 1);
      mbar_init(bar(L::T_EMPTY + b), 4);
    }
    mbar_init(bar(L::MMA_DONE), 1);
    misc[1] = 0;
    fence_mbarrier_init();
    prefetch_tmap(&tmP);
    prefetch_tmap(&tmQ);
  }
  if (warp == 1) {
    tmem_alloc(sbase + L::MISC_OFF, L::TMEM_COLS);
    tmem_relinquish();
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
  const uint32_t tmem = misc[0];
  const bool tn = p.form == kBfTN;
  const int tiles = tn ? p.G * p.nc * p.nl : blk[p.G] * p.nl;

  if (warp == 0) {
    if (lane == 0 && !(p.debug_flags & DBG_SKIP_PRODUCER)) {
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;
      for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        const BfTile T = bf_tile<BC>(t, p, first, blk);
        for (int i = 0; i < T.nk; ++i) {
          bool go = wait_bar(bar(L::EMPTY + s), ph ^ 1, abort_flag, p);
          if constexpr (kDebug) {
            const int qmax = tn ? p.M : p.rows;
            if (go && (T.l0 >= p.N || T.g >= p.G || T.q0 < 0 || T.q0 >= qmax || T.k0 < 0 ||
                       (tn && T.k0 + i * BK >= p.rows))) {
              dbg_fail(p, ST_DEBUG_BOUNDS, abort_flag);
              go = false;
            }
          }
          if (go) {
            const uint32_t full = bar(L::FULL + s);
            const uint32_t pd = sbase + L::P_OFF + s * L::P_BYTES;
            const uint32_t qd = sbase + L::Q_OFF + s * L::Q_BYTES;
            mbar_arrive_expect_tx(full, L::P_BYTES + L::Q_BYTES);
            if (p.form == kBfNT) {
              tma_load_4d(pd, &tmP, full, i * BK, T.l0, 0, T.g);
            } else {
              const int k = T.k0 + i * BK, g = tn ? 0 : T.g;
              if (p.p_split) {
                for (int j = 0; j < BL / 64; ++j)
                  tma_load_4d(pd + j * 64 * 128, &tmP, full, T.l0 + 64 * j, k, 0, g);
              } else {
                tma_load_4d(pd, &tmP, full, 0, k, T.l0 / 64, g);
              }
            }
            if (!tn) {
              tma_load_4d(qd, &tmQ, full, i * BK, T.q0, 0, 0);
            } else {
              const int k = T.k0 + i * BK;
              if (p.q_split) {
                for (int j = 0; j < BC / 64; ++j)
                  tma_load_4d(qd + j * 64 * 128, &tmQ, full, T.q0 + 64 * j, k, 0, 0);
              } else {
                tma_load_4d(qd, &tmQ, full, 0, k, T.q0 / 64, 0);
              }
            }
            issued |= 1u << s;
            issued_par = (issued_par & ~(1u << s)) | (ph << s);
          }
          if (++s == STAGES) { s = 0; ph ^= 1; }
        }
      }
      // after an abort the latest load into a slot may still be in flight
      for (int q = 0; q < STAGES; ++q)
        if ((issued >> q) & 1u) drain_wait(bar(L::FULL + q), (issued_par >> q) & 1u, p);
    }
    __syncwarp();
  } else if (warp == 1) {
    const bool p_mn = p.form != kBfNT, q_mn = tn;
    // a K step of 16: 32 bytes inside a K-major row, two 8-row atoms (2 KB) of
    // an MN-major slot, whose 64-wide atoms lie 64 rows x 128 bytes apart
    const uint64_t p_step = (p_mn ? 2048 : 32) >> 4, q_step = (q_mn ? 2048 : 32) >> 4;
    int s = 0, b = 0;
    uint32_t ph = 0, bph = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const BfTile T = bf_tile<BC>(t, p, first, blk);
      if (T.nk == 0) continue;
      const uint32_t idesc = idesc_bf16_f32(BL, (T.cols + 15) & ~15, p_mn, q_mn);
      const uint32_t d = tmem + static_cast<uint32_t>(b * BC);
      bool ok = wait_bar(bar(L::T_EMPTY + b), bph ^ 1, abort_flag, p);
      tc_fence_after();
      for (int i = 0; i < T.nk; ++i) {
        ok = wait_bar(bar(L::FULL + s), ph, abort_flag, p) && ok;
        tc_fence_after();
        const uint32_t ps = sbase + L::P_OFF + s * L::P_BYTES;
        const uint32_t qs = sbase + L::Q_OFF + s * L::Q_BYTES;
        const int left = min(BK, T.kn - i * BK), steps = (left + 15) >> 4;
        if (tn && (left & 15)) {
          // zero rows left .. 16 steps - 1 of both operands (a row is one
          // 128-byte line of each 64-wide atom)
          const int r = 16 * steps - left;
          for (int u = lane; u < r * 8 * (BL + BC) / 64; u += 32) {
            const int atom = u / (r * 8), w = u - atom * (r * 8);
            const uint32_t base = atom < BL / 64 ? ps + atom * 8192 : qs + (atom - BL / 64) * 8192;
            st_shared_v4(base + (left + (w >> 3)) * 128 + (w & 7) * 16, 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0 && ok) {
          const uint64_t pd = p_mn ? smem_desc_sw128_mnmajor(ps, 8192) : smem_desc_sw128_kmajor(ps);
          const uint64_t qd = q_mn ? smem_desc_sw128_mnmajor(qs, 8192) : smem_desc_sw128_kmajor(qs);
          for (int kk = 0; kk < steps; ++kk)
            mma_bf16(d, pd + p_step * kk, qd + q_step * kk, idesc, (i | kk) ? 1u : 0u);
          mma_commit(bar(L::EMPTY + s));
          if (i == T.nk - 1) mma_commit(bar(L::T_FULL + b));
        }
        __syncwarp();
        if (++s == STAGES) { s = 0; ph ^= 1; }
      }
      b ^= 1;
      if (b == 0) bph ^= 1;
    }
    if (lane == 0) {
      mma_commit(bar(L::MMA_DONE));
      drain_wait(bar(L::MMA_DONE), 0, p);
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int q = warp & 3;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(q * 32) << 16);
    int b = 0;
    uint32_t bph = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const BfTile T = bf_tile<BC>(t, p, first, blk);
      const bool have = T.nk > 0;
      const bool ok = !have || wait_bar(bar(L::T_FULL + b), bph, abort_flag, p);
      tc_fence_after();
      // this thread's pair of columns of D (lanes l and l ^ 1 share them)
      const int l = T.l0 + q * 32 + (lane & ~1);
      const size_t row0 = tn ? static_cast<size_t>(T.g) * p.M + T.c0 : static_cast<size_t>(T.q0);
      for (int c = 0; c < T.cols; c += 32) {
        uint32_t v[32];
        if (have) {
          tmem_ld_32x32b_x32(t_lane + static_cast<uint32_t>(b * BC + c), v);
          tmem_wait_ld(v);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
        // a lane holds 32 rows of one column of D: exchange with the
        // neighbouring lane, so that the even lane stores two columns of row j
        // and the odd one those of row j + 1
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const uint32_t give = (lane & 1) ? v[j] : v[j + 1];
          const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
          float lo = __uint_as_float((lane & 1) ? got : v[j]);
          float hi = __uint_as_float((lane & 1) ? v[j + 1] : got);
          const int r = c + j + (lane & 1);
          if (ok && r < T.cols && l < p.N) {
            const size_t at = (row0 + r) * p.N + l;
            if constexpr (kDebug) {
              if (row0 + r >= static_cast<size_t>(tn ? p.G * static_cast<long long>(p.M) : p.rows)) {
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
      if (have) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::T_EMPTY + b));
        b ^= 1;
        if (b == 0) bph ^= 1;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

constexpr int STAGES_WIDE = 4, STAGES_NARROW = 8;
constexpr int BC_WIDE = 256, BC_NARROW = 64;
constexpr int kBfMaxSmem = 232448;

template <int BC, int STAGES>
cudaError_t launch_tiles(const BfCall& c, PFN_cuTensorMapEncodeTiled_v12000 encode, int num_sms, cudaStream_t stream) {
  using L = BfSmem<BC, STAGES>;
  const bool tn = c.form == kBfTN;
  BfParams p{};
  p.form = c.form;
  p.G = c.G;
  p.rows = c.rows;
  p.M = c.M;
  p.N = c.N;
  p.nk = tn ? 0 : (c.K + BK - 1) / BK;
  p.nl = (c.N + BL - 1) / BL;
  p.nc = tn ? (c.M + BC - 1) / BC : 0;
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
      (c.form == kBfNT   ? k_major(&mp, c.B, G, N, K, BL)
       : c.form == kBfNN ? mn_major(&mp, c.B, G, K, N, BL)
                         : mn_major(&mp, c.B, 1, R, N, BL)) &&
      (tn ? mn_major(&mq, c.A, 1, R, c.M, BC) : k_major(&mq, c.A, 1, R, K, BC));
  if (!good) return cudaErrorInvalidValue;

  // as many CTAs as there can be tiles, at most one per SM
  const long long most = tn ? static_cast<long long>(c.G) * p.nc * p.nl
                            : (std::min<long long>(c.G, c.rows) + c.rows / BC) * p.nl;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::max(1ll, std::min<long long>(most, num_sms))), 1, 1);
  cfg.blockDim = dim3(BF_THREADS, 1, 1);
  cfg.dynamicSmemBytes = L::bytes(c.G);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, bf16_grouped_kernel<BC, STAGES>, mp, mq, p);
}

}  // namespace

cudaError_t bf16_set_up() {
  static_assert(BfSmem<BC_WIDE, STAGES_WIDE>::bytes(kBfMaxGroups) <= kBfMaxSmem, "shared memory");
  static_assert(BfSmem<BC_NARROW, STAGES_NARROW>::bytes(kBfMaxGroups) <= kBfMaxSmem, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(bf16_grouped_kernel<BC_WIDE, STAGES_WIDE>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kBfMaxSmem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(bf16_grouped_kernel<BC_NARROW, STAGES_NARROW>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, kBfMaxSmem);
}

cudaError_t launch_bf16_grouped(const BfCall& c, PFN_cuTensorMapEncodeTiled_v12000 encode, int num_sms, cudaStream_t stream) {
  // rows of D that a tile holds: the average group's (nt, nn), M (tn)
  const long long per = c.form == kBfTN ? c.M : (c.rows + c.G - 1) / c.G;
  return per <= BC_NARROW ? launch_tiles<BC_NARROW, STAGES_NARROW>(c, encode, num_sms, stream)
                          : launch_tiles<BC_WIDE, STAGES_WIDE>(c, encode, num_sms, stream);
}

}  // namespace dgk
