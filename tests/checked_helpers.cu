// The checks that the checked build adds to the operators around the GEMMs, one by
// one: what they let pass, what they skip, and what they report.  Every address
// that is handed out lies in its buffer, whatever a check says.
#include <cstdint>
#include <cstdio>

#include "dg_ring.cuh"

using namespace dgk;

struct Word {
  unsigned int* status;
  unsigned long long timeout_ns;
};

__global__ void run(const uint8_t* src, Word w, int* out) {
  __shared__ __align__(128) uint8_t slots[2 * 256];
  __shared__ __align__(8) uint64_t full[2];
  __shared__ uint32_t aborted, fills[kMaxRing];
  int n = 0;
  auto note = [&](int v) { out[n++] = v; };
  auto status = [&]() {   // read and clear, with the abort flag
    note(static_cast<int>(atomicExch(w.status, 0u)));
    note(static_cast<int>(*static_cast<volatile uint32_t*>(&aborted)));
    aborted = 0;
  };
  // an operand of 1008 bytes (in a buffer of 2048), chunks of 256
  ChunkRing ring{{src, nullptr, nullptr}, slots, full, 2, 1, 256, {1008, w.status, &aborted, fills}, 0, 0, 0};
  ring.init(&aborted);
  note(in_bounds(w, 4, 4, 8));
  status();
  note(in_bounds(w, 5, 4, 8));
  status();
  note(in_bounds(w, 9, 0, 8));
  status();
  note(in_bounds(w, ~size_t{0}, 2, 8));
  status();
  ring.fill(0, 0);
  note(wait_bar(smem_u32(full), 0, &aborted, w));
  note(ring.holds(0, 1));
  status();
  note(ring.holds(0, 2));
  status();
  ring.fill(3, 1);   // bytes 768 .. 1023
  note(static_cast<int>(ring.issued));
  status();
  ring.fill(3, 1, 240);
  note(static_cast<int>(ring.issued));
  note(wait_bar(smem_u32(full + 1), 0, &aborted, w));
  note(ring.holds(1, 1));
  status();
  ring.fill(-1, 0);
  status();
  ring.drain(w);
}

int main() {
  uint8_t* src;
  Word w{nullptr, 1000000000ull};
  int *out, host[64] = {};
  if (cudaMalloc(&src, 2048) || cudaMalloc(&w.status, 4) || cudaMalloc(&out, sizeof(host))) return 2;
  if (cudaMemset(src, 0, 2048) || cudaMemset(w.status, 0, 4) || cudaMemset(out, 0xFF, sizeof(host))) return 2;
  run<<<1, 1>>>(src, w, out);
  if (cudaDeviceSynchronize() || cudaMemcpy(host, out, sizeof(host), cudaMemcpyDeviceToHost)) return 3;
  for (int v : host)
    if (v != -1) std::printf("%d ", v);
  std::printf("\n");
  return 0;
}
