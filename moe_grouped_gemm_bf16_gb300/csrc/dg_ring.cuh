// A ring of chunks in shared memory, filled with bulk copies: what the
// memory-bound kernels read their inputs through when there are many rows.
#pragma once
#include <cstdint>

#include "dg_wait.cuh"
#include "ptx.cuh"

namespace dgk {

constexpr int kMaxRing = 8;   // slots of a ring
constexpr int kDebugRing = kDebug ? kMaxRing : 1;   // (their fill counters)

// Bytes of ring a block may take when `per_sm` blocks share an SM (228 KB, of
// which the system keeps 1 KB per block and the kernels use up to 512 bytes).
__host__ __device__ constexpr int ring_bytes(int per_sm) {
  return ((227 * 1024) / per_sm - 1536) / 128 * 128;
}

// What the checked build checks a ring with (nothing in the regular one: the fields
// alone cost the norm's gradient of 8192 x 7168 79 to 81 us).
template <bool DEBUG>
struct RingChecks {
  size_t extent;           // bytes of each operand
  unsigned int* status;
  volatile uint32_t* abort_flag;
  volatile uint32_t* fills;   // each slot's fills so far
};
template <>
struct RingChecks<false> {
  __device__ __forceinline__ RingChecks(size_t, unsigned int*, volatile uint32_t*, volatile uint32_t*) {}
};

// A slot holds a chunk of each of up to three operands, one after the other; a
// chunk is the i-th run of `bytes` bytes of its operand.  One thread fills.
template <bool DEBUG>
struct ChunkRingT {
  const void* op[3];
  uint8_t* smem;
  uint64_t* full;          // a barrier per slot
  int stages, ops, bytes;
  RingChecks<DEBUG> checks;
  uint32_t debug_flags;
  uint32_t issued, phase;  // filling thread: slots with a load, and that load's phase

  // Filling thread, before the first fill (and a barrier of the block).
  __device__ __forceinline__ void init(volatile uint32_t* abort_flag) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(full + s), 1);
    if constexpr (DEBUG)
      for (int s = 0; s < stages; ++s) checks.fills[s] = 0;
    *abort_flag = 0;
    fence_mbarrier_init();
  }

  __device__ __forceinline__ uint8_t* slot(int s) const { return smem + s * ops * bytes; }

  // Chunk i into slot s; `part` bytes of it, where it is the operands' last and
  // shorter (16-byte multiples).
  __device__ __forceinline__ void fill(int i, int s, int part) {
    if (debug_flags & DBG_SKIP_PRODUCER) return;
    if constexpr (DEBUG) {
      if (i < 0 || part < 0 || part > bytes || static_cast<size_t>(i) * bytes + part > checks.extent) {
        dbg_fail(checks, ST_DEBUG_BOUNDS, checks.abort_flag);
        return;
      }
      checks.fills[s] = checks.fills[s] + 1;
    }
    const uint32_t dst = smem_u32(slot(s)), bar = smem_u32(full + s);
    mbar_arrive_expect_tx(bar, ops * part);
    for (int j = 0; j < ops; ++j)
      bulk_load_g2s(dst + j * bytes,
                    static_cast<const uint8_t*>(op[j]) + static_cast<size_t>(i) * bytes, part, bar);
    phase = (issued >> s) & 1u ? phase ^ (1u << s) : phase;
    issued |= 1u << s;
  }
  __device__ __forceinline__ void fill(int i, int s) { fill(i, s, bytes); }

  // Checked build, after a wait: slot s holds its n-th fill.
  __device__ __forceinline__ bool holds(int s, long long n) const {
    if constexpr (DEBUG) {
      if (checks.fills[s] != n) {
        dbg_fail(checks, ST_DEBUG_PHASE, checks.abort_flag);
        return false;
      }
    }
    return true;
  }

  // Filling thread, before the block ends after an abort: loads may be in flight.
  template <class P>
  __device__ __forceinline__ void drain(const P& p) {
    for (int s = 0; s < stages; ++s)
      if ((issued >> s) & 1u) drain_wait(smem_u32(full + s), (phase >> s) & 1u, p);
  }
};
using ChunkRing = ChunkRingT<kDebug>;

}  // namespace dgk
