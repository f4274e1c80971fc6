// A ring of chunks in shared memory, filled with bulk copies: what the
// memory-bound kernels read their inputs through when there are many rows.
#pragma once
#include <cstdint>

#include "dg_wait.cuh"
#include "ptx.cuh"

namespace dgk {

constexpr int kMaxRing = 8;   // slots of a ring

// Bytes of ring a block may take when `per_sm` blocks share an SM (228 KB, of
// which the system keeps 1 KB per block and the kernels use up to 512 bytes).
__host__ __device__ constexpr int ring_bytes(int per_sm) {
  return ((227 * 1024) / per_sm - 1536) / 128 * 128;
}

// A slot holds a chunk of each of up to three operands, one after the other; a
// chunk is the i-th run of `bytes` bytes of its operand.  One thread fills.
struct ChunkRing {
  const void* op[3];
  uint8_t* smem;
  uint64_t* full;          // a barrier per slot
  int stages, ops, bytes;
  uint32_t debug_flags;
  uint32_t issued, phase;  // filling thread: slots with a load, and that load's phase

  __device__ __forceinline__ uint8_t* slot(int s) const { return smem + s * ops * bytes; }

  // Chunk i into slot s; `part` bytes of it, where it is the operands' last and
  // shorter (16-byte multiples).
  __device__ __forceinline__ void fill(int i, int s, int part) {
    if (debug_flags & DBG_SKIP_PRODUCER) return;
    const uint32_t dst = smem_u32(slot(s)), bar = smem_u32(full + s);
    mbar_arrive_expect_tx(bar, ops * part);
    for (int j = 0; j < ops; ++j)
      bulk_load_g2s(dst + j * bytes,
                    static_cast<const uint8_t*>(op[j]) + static_cast<size_t>(i) * bytes, part, bar);
    phase = (issued >> s) & 1u ? phase ^ (1u << s) : phase;
    issued |= 1u << s;
  }
  __device__ __forceinline__ void fill(int i, int s) { fill(i, s, bytes); }

  // Filling thread, before the block ends after an abort: loads may be in flight.
  template <class P>
  __device__ __forceinline__ void drain(const P& p) {
    for (int s = 0; s < stages; ++s)
      if ((issued >> s) & 1u) drain_wait(smem_u32(full + s), (phase >> s) & 1u, p);
  }
};

}  // namespace dgk
