// Routing of tokens to experts, and its gradient.  Per token, of its G logits x
// and the experts' bias b:
//
//   s_e = 1 / (1 + exp(-x_e)), or softmax(x)_e;   c_e = s_e + b_e
//   of n groups of consecutive experts the m with the largest value stay, a
//   group's value the sum of its (one or two) largest c
//   the k largest c among them are chosen, equal ones by their index
//   w_j = scale s_j, or scale s_j / (sum of the chosen s)
//
// A warp takes a token (or several of few experts), a lane NPL consecutive experts: the
// k largest are k rounds of a maximum over the lanes, on the values' order as unsigned
// integers, which the first lane that holds it takes out.
//
// The choice is that of the formulas in 64 bits, whatever the rounding here: where all
// biases are equal, experts are chosen by the logits themselves (both scores rise with
// them), else by c in fp32.  A token with two values nearer to each other than their
// errors, at a place where that decides (about one in a thousand of 256 experts), has its
// choices and what comes after them within the error sorted again in 64 bits, and so its
// groups; where that many values are in doubt that lanes do not suffice, or a group's
// largest are not clear, it is chosen again altogether (choose_exact).
//
// Bounded by latency and by instructions, not by memory.
#include <float.h>

#include <algorithm>

#include <cuda_bf16.h>

#include "dg_launch.h"
#include "dg_params.h"
#include "dg_route.h"
#include "dg_wait.cuh"
#include "ptx.cuh"

namespace dgk {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr int RT_WARPS = 8;

// Added to the sum that weights are renormalised by (sigmoid
// scores): scores that all underflow give weights of zero.
constexpr float kLeast = 1e-20f;

__device__ __forceinline__ float read_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float read_logit(const __nv_bfloat16* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
}

// The logit as it counts: NaN as -infinity (the expert is not available),
// +infinity as the largest number, -0 as 0.
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : fminf(x, FLT_MAX) + 0.f; }

// Unsigned integers in the order of the floats; 0 stands below them all.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
  return v;
}
// (by exp(-|x|), which does not overflow)
__device__ __forceinline__ float sigmoid(float x) {
  const float e = expf(-fabsf(x));
  return __fdiv_rn(x < 0.f ? e : 1.f, 1.f + e);
}

// Unsigned integers in the order of the doubles, none of them NaN; 0 stands below
// them all.  (Compared as such: FP64 instructions are issued every 16 cycles.)
__device__ __forceinline__ uint64_t order_of(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  return u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double double_of(uint64_t o) {
  return __longlong_as_double(
      static_cast<long long>((o & 0x8000000000000000ull) ? o ^ 0x8000000000000000ull : ~o));
}
__device__ __forceinline__ uint64_t warp_most(uint64_t v) {
  const uint32_t high = __reduce_max_sync(ALL, static_cast<uint32_t>(v >> 32));
  const uint32_t low = __reduce_max_sync(ALL, static_cast<uint32_t>(v >> 32) == high ? static_cast<uint32_t>(v) : 0);
  return static_cast<uint64_t>(high) << 32 | low;
}

template <class X>
__device__ __forceinline__ uint32_t logit_order(const X* p) {
  const float x = clean(read_logit(p));
  return x > -INFINITY ? order_of(x) : 0;
}

// The margin at a value c.  A c of +infinity, by its bias, is held as the largest number
// but for the key's last bits: what is that large is settled in 64 bits, where all of them
// are equal.
__device__ __forceinline__ float margin_at(float c, float margin) {
  return c > 0x1p127f ? fmaxf(margin, 0x1p126f) : margin;
}

// What the choice in fp32 leaves open, in 64 bits.  row: the token's values as
// order_of(c) in fp32 (0: not available), whose differences are off by less than
// `margin`; or by_logit, and the logits themselves decide (even: between the experts of
// the groups that stay).  Only the values that this leaves in doubt are computed, a lane
// one of its own at a time (few lanes have more than one).  Returns the j-th choice in
// lane j.  (All values in 64 bits took 7 us for a token of 128 experts, 13 of 384.)
template <class X, int NPL>
__device__ __noinline__ int choose_exact(const RouteFwd a, const X* logits, const uint32_t* row,
                                         bool even, bool by_logit, float margin) {
  const int lane = threadIdx.x & 31, e0 = lane * NPL;
  uint32_t key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    key[i] = 0;
    if (e0 + i >= a.G) continue;
    key[i] = by_logit ? logit_order(logits + e0 + i) : row[e0 + i];
  }
  uint64_t c[NPL];   // order of the exact values; 0: not needed
#pragma unroll
  for (int i = 0; i < NPL; ++i) c[i] = 0;
  double top = 0, sum = 1;
  if (!a.sigmoid && !by_logit) {
    float m = -INFINITY;
    for (int e = lane; e < a.G; e += 32) m = fmaxf(m, clean(read_logit(logits + e)));
    top = static_cast<double>(float_of(__reduce_max_sync(ALL, order_of(m))));
    sum = 0;
    for (int e = lane; e < a.G; e += 32) {
      const float x = clean(read_logit(logits + e));
      if (x > -INFINITY) sum += exp(static_cast<double>(x) - top);
    }
    sum = warp_sum(sum);
  }
  // computes the values in `want` (a bit per value of the lane)
  auto compute = [&](uint32_t want) {
    while (__any_sync(ALL, want != 0)) {
      const int at = want ? __ffs(want) - 1 : 0;
      uint64_t v = 0;
      if (want) {
        double s = clean(read_logit(logits + e0 + at));
        if (!by_logit) {
          s = a.sigmoid ? 1.0 / (1.0 + exp(-s)) : exp(s - top) / sum;
          if (a.bias) s += static_cast<double>(__ldg(a.bias + e0 + at));
        }
        v = order_of(s);
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (want && i == at) c[i] = v;
      want &= want - 1;
    }
  };
  uint32_t done = 0;
  if (a.groups > a.top_groups) {
    // the values that may be among their group's `best`: not below its best-th in fp32
    // by more than the margin
    const int per = a.G / a.groups;
    uint64_t mine = 0;   // lane g: group g's value
    uint32_t edge = 0;   // lane g: group g's best-th
    for (int g = 0; g < a.groups; ++g) {
      uint32_t one = 0, two = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (e0 + i >= g * per && e0 + i < (g + 1) * per) {
          two = max(two, min(one, key[i]));
          one = max(one, key[i]);
        }
      const uint32_t first = __reduce_max_sync(ALL, one);
      const int owner = __ffs(__ballot_sync(ALL, one == first)) - 1;
      const uint32_t second = __reduce_max_sync(ALL, lane == owner ? two : one);
      if (lane == g) edge = a.best == 2 && second ? second : first;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const uint32_t limit = __shfl_sync(ALL, edge, min((e0 + i) / per, 31));
      if (key[i] && float_of(key[i]) >= float_of(limit) - margin_at(float_of(limit), margin)) done |= 1u << i;
    }
    compute(done);
    for (int g = 0; g < a.groups; ++g) {
      uint64_t one = 0, two = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (c[i] && e0 + i >= g * per && e0 + i < (g + 1) * per) {
          if (c[i] > one) { two = one; one = c[i]; }
          else if (c[i] > two) two = c[i];
        }
      const uint64_t first = warp_most(one);
      // (the first lane that holds the largest gives its second)
      const int owner = __ffs(__ballot_sync(ALL, one == first)) - 1;
      const uint64_t second = warp_most(lane == owner ? two : one);
      if (lane == g) {
        mine = first;
        if (a.best == 2 && second) mine = order_of(double_of(first) + double_of(second));
      }
    }
    uint32_t keep = 0;
    for (int n = 0; n < a.top_groups; ++n) {
      const uint64_t left = (keep >> lane) & 1u ? 0 : mine;
      const uint64_t v = warp_most(left);
      if (v == 0) break;
      keep |= 1u << (__ffs(__ballot_sync(ALL, left == v)) - 1);
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (!((keep >> min((e0 + i) / per, 31)) & 1u)) key[i] = c[i] = 0;
    if (even && !by_logit) {
      by_logit = true;
      margin = 0.f;
      done = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (key[i]) key[i] = logit_order(logits + e0 + i);
    }
  }
  // the values that may be among the k largest: not below the k-th in fp32 by more
  // than the margin
  uint32_t left[NPL], edge = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) left[i] = key[i];
  for (int j = 0; j < a.k; ++j) {
    uint32_t v = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (left[i] > v) { v = left[i]; at = i; }
    const uint32_t best = __reduce_max_sync(ALL, v);
    if (best) edge = best;
    const int owner = __ffs(__ballot_sync(ALL, v == best)) - 1;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (lane == owner && i == at) left[i] = 0;
  }
  uint32_t want = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    if (key[i] && float_of(key[i]) >= float_of(edge) - margin_at(float_of(edge), margin)) {
      if (!((done >> i) & 1u)) want |= 1u << i;
    } else {
      c[i] = 0;
    }
  }
  compute(want);
  int chosen = -1;
  for (int j = 0; j < a.k; ++j) {
    uint64_t v = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (c[i] > v) { v = c[i]; at = i; }
    const uint64_t best = warp_most(v);
    if (best == 0) break;
    const int owner = __ffs(__ballot_sync(ALL, v == best)) - 1;
    const int e = __shfl_sync(ALL, e0 + at, owner);
    if (lane == j) chosen = e;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (lane == owner && i == at) c[i] = 0;
  }
  return chosen;
}

// ex2 and rcp approximated (2^-22 and 2^-23 of the result): for the choice, where what
// they are off by is counted; the weights are computed with expf and division.
__device__ __forceinline__ float exp_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// More than what the difference of two c near `c` may be off by in fp32, `bias`
// the largest bias' magnitude; u = 2^-24.
// A sigmoid: e by (4 + 1.5 |x|) u of itself (ex2.approx, its argument), s = 1 / (1 + e)
// by a quarter of that at most and |x| s (1 - s) < 0.23, sum, reciprocal and product by
// 4 u: below 2^-21 each.
// A softmax's s, `share` (1 / the sum) the largest of them: e by (4 + 2.5 d) u of itself,
// d = |x - max| = ln(share / s), below 88 where e is held; the sum, common to
// both, by (4 + 2.5 ln(1024)) u for its terms and 40 u for its additions and its
// reciprocal: with s d < 0.37 share below 2^-17 share in all, with d < 88 below 2^-14 of
// s.  (2769 tokens of 160 experts in 8 groups by sums of two: 10.9 us, with 2^-17 for all
// 18.6.)  From there on, below 2^-126, e is 0, which is off by all that it was: 2^-125 for
// both, whatever s is.
// Each c: u of itself, and by NPL 2^-23 of itself, as a key whose last bits say which of
// the lane's values it is.
template <int NPL>
__device__ __forceinline__ float doubt(bool sigmoid, float c, float bias, float share) {
  const float s =
      sigmoid ? 0x1p-19f : fminf(0x1p-17f * share, 0x1p-14f * (fabsf(c) + bias)) + 0x1p-125f;
  return s + (NPL + 1) * 0x1p-22f * fabsf(c);
}

// A lane's NPL consecutive logits (or biases) from e0 on, -infinity behind the last.
// `whole`: the row lies on 16 bytes, or on as many as a lane's elements take.
template <int NPL>
__device__ __forceinline__ void read_row(const float* p, int e0, int G, bool whole, float (&x)[NPL]) {
  if (whole && NPL >= 4) {
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e0 + i < G) v = __ldg(reinterpret_cast<const float4*>(p + e0 + i));
      x[i] = v.x;
      x[i + 1 < NPL ? i + 1 : i] = v.y;
      x[i + 2 < NPL ? i + 2 : i] = v.z;
      x[i + 3 < NPL ? i + 3 : i] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) x[i] = e0 + i < G ? __ldg(p + e0 + i) : -INFINITY;
  }
}
template <int NPL>
__device__ __forceinline__ void read_row(const __nv_bfloat16* p, int e0, int G, bool whole,
                                         float (&x)[NPL]) {
  constexpr uint32_t kNone = 0xff80ff80u;   // -infinity twice
  if (whole && NPL >= 4) {
    constexpr int STEP = NPL >= 8 ? 8 : 4;
#pragma unroll
    for (int i = 0; i < NPL; i += STEP) {
      uint32_t v[4] = {kNone, kNone, kNone, kNone};
      if (e0 + i < G) {
        if constexpr (STEP == 8) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(p + e0 + i));
          v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
        } else {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(p + e0 + i));
          v[0] = w.x; v[1] = w.y;
        }
      }
#pragma unroll
      for (int j = 0; j < STEP && i + j < NPL; ++j)
        x[i + j] = __uint_as_float(j & 1 ? v[j >> 1] & 0xFFFF0000u : v[j >> 1] << 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) x[i] = e0 + i < G ? read_logit(p + e0 + i) : -INFINITY;
  }
}

// Whether every row of G elements at p lies as read_row's whole rows do.
template <class X, int NPL>
bool whole_rows(const void* p, int G) {
  constexpr int step = NPL * static_cast<int>(sizeof(X)) >= 16 ? 16 / sizeof(X) : NPL;
  return NPL >= 4 && G % step == 0 && (reinterpret_cast<uintptr_t>(p) & (step * sizeof(X) - 1)) == 0;
}

template <int NPL>
__device__ __forceinline__ uint32_t largest(const uint32_t (&key)[NPL]) {
  uint32_t v[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) v[i] = key[i];
#pragma unroll
  for (int n = NPL / 2; n >= 1; n >>= 1)
#pragma unroll
    for (int i = 0; i < NPL / 2; ++i)
      if (i < n) v[i] = max(v[i], v[i + n]);
  return v[0];
}

// Over the LANES lanes of a token.
template <int LANES>
__device__ __forceinline__ uint32_t team_max(uint32_t v) {
  if constexpr (LANES == 32) {
    return __reduce_max_sync(ALL, v);
  } else {
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) v = max(v, __shfl_xor_sync(ALL, v, o));
    return v;
  }
}
template <int LANES>
__device__ __forceinline__ float team_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
  return v;
}
// The first lane of the token (counted in it) that has `p`; -1: none.
template <int LANES>
__device__ __forceinline__ int team_first(bool p, int team) {
  uint32_t b = __ballot_sync(ALL, p);
  if (LANES < 32) b = b >> (team * LANES) & ((1u << (LANES & 31)) - 1);
  return __ffs(b) - 1;
}

// What the host works out once.
struct RoutePlan {
  int per;             // experts of a group
  uint32_t per_inv;    // x / per = __umulhi(x, per_inv) for x < 2^16 (per = 1: 0)
  bool grouped;        // groups are left out
  bool lane_group;     // a lane's experts are of one group
  bool whole, whole_bias;
};

// NPL: experts per lane, LANES: lanes per token (the others of the warp take further
// tokens: 9268 tokens of 16 experts took 9 us with a warp each).  LOGITS: there are no
// biases and no sums of two, so that the logits decide (16384 tokens of 128 experts in
// bf16: 8.9 us without instances of its own).  The blocks per SM leave 48 or 64
// registers a thread of up to 8 experts, and spills (of 8 experts with biases 178 bytes, in
// bf16 246): with a block less 8192 tokens of 256 in 8 groups by sums of two with biases take
// 18.6 us, so 17.0, by softmax 23.2 and 22.3, but 2769 of 160 without biases 9.6 and 10.9.
template <class X, int NPL, int LANES, bool LOGITS>
__global__ void __launch_bounds__(32 * RT_WARPS, NPL <= 4 ? 5 : NPL == 8 ? 4 : NPL == 16 ? 2 : 1)
route_kernel(const RouteFwd a, const RoutePlan plan) {
  constexpr int TEAMS = 32 / LANES;
  constexpr uint32_t TEAM = LANES == 32 ? ALL : (1u << (LANES & 31)) - 1;   // a team's lanes in a ballot
  extern __shared__ uint32_t route_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = lane / LANES, member = lane % LANES, e0 = member * NPL;
  uint32_t* rows = route_smem + warp * TEAMS * a.G;   // the tokens' values in order (if kept)
  uint32_t* row = rows + team * a.G;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int first_t = (blockIdx.x * RT_WARPS + warp) * TEAMS;
  // (a token behind the last is read as the last, and not written)
  auto logits_of = [&](int t) {
    return static_cast<const X*>(a.logits) + static_cast<size_t>(min(t, a.T - 1)) * a.G;
  };
  float x[NPL];
  // (the first row and the biases asked for together)
  if (first_t < a.T) read_row<NPL>(logits_of(first_t + team), e0, a.G, plan.whole, x);
  // all biases equal: the choice is by the logits
  bool even = true;   // (a constant with LOGITS)
  float bias_most = 0.f;
  if (!LOGITS && a.bias) {
    float b[NPL];
    read_row<NPL>(a.bias, e0, a.G, plan.whole_bias, b);
    const float first = __shfl_sync(ALL, b[0], 0);
    even = first > -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (e0 + i < a.G) {
        even = even && b[i] == first;
        bias_most = fmaxf(bias_most, fabsf(b[i]));
      }
    even = __all_sync(ALL, even);
    bias_most = __uint_as_float(__reduce_max_sync(ALL, __float_as_uint(bias_most)));
    if (bias_most == INFINITY) {   // (in all lanes) the largest finite one
      bias_most = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (e0 + i < a.G && fabsf(b[i]) < INFINITY) bias_most = fmaxf(bias_most, fabsf(b[i]));
      bias_most = __uint_as_float(__reduce_max_sync(ALL, __float_as_uint(bias_most)));
    }
  }
  const bool grouped = plan.grouped;
  const bool by_logit = LOGITS || (even && (!grouped || a.best == 1));
  const bool full = even && sizeof(X) == 2;   // (in the end) keys that say the expert
  for (int t0 = first_t; t0 < a.T; t0 += gridDim.x * RT_WARPS * TEAMS) {
    const int t = t0 + team;
    const X* logits = logits_of(t);
    if (t0 != first_t) read_row<NPL>(logits, e0, a.G, plan.whole, x);
    // Order of c, or of the logit; 0: not available.  The last bits of a key say which
    // value it is: of bf16 logits, whose order leaves 16 bits free, the expert (the lower,
    // the larger), else which of the lane's (so that values that differ no further are in
    // doubt).
    uint32_t key[NPL];
    bool there_is[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      there_is[i] = x[i] > -INFINITY;   // (false for NaN)
      x[i] = fminf(x[i], FLT_MAX);
    }
    auto low_bits = [&](uint32_t o, int i) { return (o & ~(NPL - 1u)) | (NPL - 1 - i); };
    auto logit_key = [&](float x, int i) {
      const uint32_t o = order_of(x + 0.f);   // (-0 as 0)
      return full ? (o & 0xFFFF0000u) | (0xFFFFu - (e0 + i)) : low_bits(o, i);
    };
    float top = 0.f, sum = 1.f;
    float share = 1.f;   // 1 / the sum of a softmax, where c is computed
    // the scores are needed in full for c, or for a softmax's sum
    if (!a.sigmoid && !(by_logit && a.renormalize)) {
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i) most = max(most, there_is[i] ? order_of(x[i]) : 0);
      most = team_max<LANES>(most);
      top = most ? float_of(most) : 0.f;
    }
    if (by_logit) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) key[i] = there_is[i] ? logit_key(x[i], i) : 0;
      if (!a.sigmoid && !a.renormalize) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) sum += there_is[i] ? expf(x[i] - top) : 0.f;
        sum = team_sum<LANES>(sum);
      }
    } else {
      if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float e = exp_fast(-fabsf(x[i]));
          x[i] = (x[i] < 0.f ? e : 1.f) * rcp_fast(1.f + e);
        }
      } else {
        sum = 0.f;
        // (also the weights' sum, where they are not renormalised)
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float d = x[i] - top;
          x[i] = !there_is[i] ? 0.f : a.renormalize ? exp_fast(d) : expf(d);
          sum += x[i];
        }
        sum = team_sum<LANES>(sum);
      }
      if (!a.sigmoid) share = rcp_fast(sum);
      float b[NPL] = {};
      if (a.bias) read_row<NPL>(a.bias, e0, a.G, plan.whole_bias, b);   // (in L1)
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const float c = fmaf(x[i], share, b[i]);
        key[i] = there_is[i] && c > -INFINITY ? low_bits(order_of(fminf(c, FLT_MAX)), i) : 0;
      }
    }
    // (|c| at most that of the scores and the biases)
    const float margin = 2.f * doubt<NPL>(a.sigmoid, share + bias_most, bias_most, share);
    // a softmax's sum in 64 bits (of the whole team), and c of an expert
    auto exact_total = [&]() {
      double total = 1.0;
      if (!a.sigmoid) {
        float y[NPL];
        read_row<NPL>(logits, e0, a.G, plan.whole, y);
        total = 0.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          if (there_is[i]) total += exp(static_cast<double>(fminf(y[i], FLT_MAX)) - static_cast<double>(top));
#pragma unroll
        for (int o = LANES / 2; o >= 1; o >>= 1) total += __shfl_xor_sync(ALL, total, o);
      }
      return total;
    };
    auto exact_score = [&](int e, double total) {
      double v = clean(read_logit(logits + e));
      v = a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - static_cast<double>(top)) / total;
      return a.bias ? v + static_cast<double>(__ldg(a.bias + e)) : v;
    };
    bool sure = true;
    if (grouped || !by_logit) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (e0 + i < a.G)   // (the logits' order itself: a group's largest is not in doubt)
          row[e0 + i] = !by_logit ? key[i] : there_is[i] ? order_of(x[i] + 0.f) : 0;
      __syncwarp();
    }
    if (grouped) {
      // LANES / groups lanes (a power of two) to a group's two largest values
      const int shift = 31 - __clz(LANES / a.groups), width = 1 << shift;
      const int g = member >> shift;
      uint32_t one = 0, two = 0;
      if (g < a.groups)
#pragma unroll 4
        for (int e = member & (width - 1); e < plan.per; e += width) {
          const uint32_t v = row[g * plan.per + e];
          two = max(two, min(one, v));
          one = max(one, v);
        }
      for (int o = width >> 1; o >= 1; o >>= 1) {
        const uint32_t p = __shfl_xor_sync(ALL, one, o), q = __shfl_xor_sync(ALL, two, o);
        two = max(max(two, q), min(one, p));
        one = max(one, p);
      }
      uint32_t value = one;
      if (a.best == 2 && two) value = order_of(float_of(one) + float_of(two));
      // a group's rank: the groups of a larger value, and of the same before it
      const bool mine = g < a.groups;
      value = mine ? value : 0;
      int rank = 0;
      for (int h = 0; h < a.groups; ++h) {
        const uint32_t v = __shfl_sync(ALL, value, team * LANES + (h << shift));
        rank += v > value || (v == value && h < g);
      }
      bool stays = mine && value && rank < a.top_groups;
      uint32_t lanes = __ballot_sync(ALL, stays) >> (team * LANES);
      const uint32_t last = ~team_max<LANES>(stays ? ~value : 0);
      const uint32_t next = team_max<LANES>(stays ? 0 : value);
      // What is rounded are a sum's two values: of opposite signs they are larger than it, by
      // no more than the bias of the negative one.
      const float more = !LOGITS && a.best == 2 ? bias_most : 0.f;
      if (!by_logit && next) {
        const float l = float_of(last), n = float_of(next);
        sure = l - n > 2.f * doubt<NPL>(a.sigmoid, fmaxf(fabsf(l), fabsf(n)) + more, bias_most, share);
      }
      if (__any_sync(ALL, !sure)) {
        // The groups' values in 64 bits, by the first lane of each, of its largest values in
        // fp32.  Where the next one is within the margin of them: of its largest logits, if
        // the biases are equal, else by choose_exact.
        const double total = exact_total();
        uint64_t exact = 0;
        bool clear = true;
        const bool first = mine && (member & (width - 1)) == 0;
        if (first) {
          uint32_t v1, v2, v3;
          int e1, e2;
          auto largest_of = [&](bool logit) {
            v1 = v2 = v3 = 0;
            e1 = e2 = 0;
#pragma unroll 4
            for (int e = g * plan.per; e < (g + 1) * plan.per; ++e) {
              const uint32_t v = logit ? logit_order(logits + e) : row[e];
              if (v > v1) {
                v3 = v2;
                v2 = v1;
                e2 = e1;
                v1 = v;
                e1 = e;
              } else if (v > v2) {
                v3 = v2;
                v2 = v;
                e2 = e;
              } else {
                v3 = max(v3, v);
              }
            }
          };
          largest_of(false);
          const uint32_t in = a.best == 2 ? v2 : v1, out = a.best == 2 ? v3 : v2;
          clear = !(in && out && float_of(in) - float_of(out) <= margin);
          if (!clear && even) {
            largest_of(true);
            clear = true;
          }
          if (v1) {
            double v = exact_score(e1, total);
            if (a.best == 2 && v2) v += exact_score(e2, total);
            exact = order_of(v);
          }
        }
        int place = 0;
        for (int h = 0; h < a.groups; ++h) {
          const uint64_t v = __shfl_sync(ALL, exact, team * LANES + (h << shift));
          place += v > exact || (v == exact && h < g);
        }
        // (a group's other lanes follow the first)
        const int from = team * LANES + (min(g, a.groups - 1) << shift);
        // (asked for by all lanes, also those without a group)
        const int theirs = __shfl_sync(ALL, exact && place < a.top_groups ? 1 : 0, from);
        const bool stay = mine && theirs != 0;
        const uint32_t unclear = __ballot_sync(ALL, !clear) >> (team * LANES);
        const uint32_t settled = __ballot_sync(ALL, stay) >> (team * LANES);
        if (!sure && (unclear & TEAM) == 0) {
          sure = true;
          lanes = settled;
        }
      }
      auto stays_at = [&](int i) {
        const uint32_t of = plan.per_inv ? __umulhi(e0 + i, plan.per_inv) : e0 + i;
        return ((lanes >> (of << shift & 31)) & 1u) != 0;
      };
      if (plan.lane_group) {
        const bool all = stays_at(0);
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = all ? key[i] : 0;
      } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = stays_at(i) ? key[i] : 0;
      }
    }
    if (even && !by_logit) {
      // the groups chosen by sums of c: their experts by the logits again
      read_row<NPL>(logits, e0, a.G, plan.whole, x);   // (in L1)
#pragma unroll
      for (int i = 0; i < NPL; ++i) key[i] = key[i] ? logit_key(fminf(x[i], FLT_MAX), i) : 0;
    }
    // k rounds, and one more for what the last choice was close to
    int chosen = -1;
    if (full) {
      for (int j = 0; j < a.k; ++j) {
        const uint32_t best = team_max<LANES>(largest<NPL>(key));
        if (member == j && best) chosen = 0xFFFF - (best & 0xFFFFu);
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = key[i] == best ? 0 : key[i];
      }
    } else {
      // lane j: the j-th key and whose it is (also of the last round, where there is a lane)
      uint32_t mine = 0, best = 0;
      int whose = -1;
      auto pick = [&](int j) {
        const uint32_t v = largest<NPL>(key);
        best = team_max<LANES>(v);
        const int owner = team_first<LANES>(v == best, team);
        if (member == j && best) {
          whose = owner * NPL + NPL - 1 - static_cast<int>(best & (NPL - 1u));
          mine = best;
        }
        const uint32_t gone = member == owner ? best : 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = key[i] == gone ? 0 : key[i];
      };
      for (int j = 0; j <= a.k; ++j) pick(j);
      chosen = member < a.k ? whose : -1;
      // each choice against the next one
      uint32_t next = __shfl_down_sync(ALL, mine, 1);
      if (member == a.k - 1) next = best;
      bool apart = true;
      if (member < a.k && mine && next) {
        const float l = float_of(mine), n = float_of(next);
        apart = even ? (mine ^ next) >= static_cast<uint32_t>(NPL)
                     : l - n > doubt<NPL>(a.sigmoid, fmaxf(fabsf(l), fabsf(n)), bias_most, share);
      }
      const uint32_t close = __ballot_sync(ALL, !apart);
      const bool open = ((close >> (team * LANES)) & TEAM) != 0;
      if (a.k >= LANES) {
        sure = sure && !open;
      } else if (__any_sync(ALL, open && sure)) {
        // The choices and all that come after them within the margin (of logits: of the same
        // key but for the last bits), one to a lane, in 64 bits, and their order by that.
        const uint32_t last_in = __shfl_sync(ALL, mine, team * LANES + a.k - 1);
        int n = a.k + 1;
        const float reach = margin_at(float_of(last_in), margin);
        bool more = open && sure && last_in != 0;
        auto near_last = [&]() {
          return best && (even ? (last_in ^ best) < static_cast<uint32_t>(NPL)
                               : float_of(last_in) - float_of(best) <= reach);
        };
        more = more && near_last();
        while (__any_sync(ALL, more && n < LANES)) {
          // (a team that is done, or full, takes none: its `more` stays as it is)
          const bool go = more && n < LANES;
          pick(go ? n : LANES);
          if (go) {
            ++n;
            more = near_last();
          }
        }
        const double total = even ? 1.0 : exact_total();
        uint64_t exact = 0;
        if (mine && member < n) {
          exact = even ? static_cast<uint64_t>(logit_order(logits + whose)) << 32
                       : order_of(exact_score(whose, total));
        }
        int rank = 0;
        const int most = static_cast<int>(__reduce_max_sync(ALL, static_cast<unsigned>(n)));
        for (int i = 0; i < most; ++i) {
          const uint64_t v = __shfl_sync(ALL, exact, team * LANES + i);
          const int e = __shfl_sync(ALL, whose, team * LANES + i);
          rank += v > exact || (v == exact && v && e < whose);
        }
        int sorted = -1;
        for (int j = 0; j < a.k; ++j) {
          const int from = team_first<LANES>(exact && rank == j, team);
          const int e = __shfl_sync(ALL, whose, team * LANES + max(from, 0));
          if (member == j && from >= 0) sorted = e;
        }
        // (more within the margin than lanes: by choose_exact)
        if (open && sure) {
          if (more) sure = false;
          else if (member < a.k) chosen = sorted;
        }
      }
    }
    const uint32_t unsettled = __ballot_sync(ALL, !sure);
    if (unsettled) {
      // all lanes take one token at a time
      for (int i = 0; i < TEAMS; ++i) {
        if (!((unsettled >> (i * LANES)) & 1u)) continue;
        const float within = by_logit ? 0.f : __shfl_sync(ALL, margin, i * LANES);
        const int e = choose_exact<X, (NPL * LANES + 31) / 32>(a, logits_of(t0 + i), rows + i * a.G, even,
                                                               by_logit, within);
        const int theirs = __shfl_sync(ALL, e, member);
        if (team == i) chosen = theirs;
      }
    }
    // weights: lane j that of the j-th choice
    const bool there = member < a.k && chosen >= 0;
    const float y = there ? clean(read_logit(logits + chosen)) : -INFINITY;
    float s;
    if (a.sigmoid) {
      s = there ? sigmoid(y) : 0.f;
      if (a.renormalize) s = __fdiv_rn(s, team_sum<LANES>(s) + kLeast);
    } else if (a.renormalize) {
      // (relative to the largest chosen: no underflow of them all)
      const uint32_t m = team_max<LANES>(there ? order_of(y) : 0);
      s = there ? expf(y - float_of(m)) : 0.f;
      const float total = team_sum<LANES>(s);
      s = there ? __fdiv_rn(s, total) : 0.f;
    } else {
      s = there ? __fdiv_rn(expf(y - top), sum) : 0.f;
    }
    if (member < a.k && t < a.T) {
      const size_t at = static_cast<size_t>(t) * a.k + member;
      if (!in_bounds(a, at, 1, static_cast<size_t>(a.T) * a.k)) continue;
      a.experts[at] = chosen;
      a.weights[at] = s * a.scale;
    }
  }
}

__device__ __forceinline__ void write_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void write_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Element i of the gradient of token t.
template <class X>
__device__ __forceinline__ void write_logit(const RouteBwd& a, int t, int i, float v) {
  const size_t at = static_cast<size_t>(t) * a.G + i;
  if (in_bounds(a, at, 1, static_cast<size_t>(a.T) * a.G)) write_logit(static_cast<X*>(a.d_logits) + at, v);
}

// Gradient of the logits, the choice taken as it is.  With d_j the gradient of
// w_j times the scale:
//   renormalised: ds_j = (d_j - sum_i d_i s_i / S) / S, S the sum of the chosen s
//   sigmoid: dx = ds s (1 - s);  softmax: dx_e = s_e (ds_e - sum_i ds_i s_i)
// In the renormalised softmax the last sum vanishes, so that, as with sigmoid
// scores, only the chosen logits have a gradient and only they are read: a token takes
// LANES lanes, one for each choice, which write zeros and then the chosen ones'.
template <class X, int LANES>
__global__ void __launch_bounds__(32 * RT_WARPS)
route_backward_few_kernel(const RouteBwd a, bool whole) {
  constexpr int TEAMS = 32 / LANES, STEP = 16 / sizeof(X);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = lane / LANES, member = lane % LANES;
  grid_dep_wait();
  grid_dep_launch_dependents();
  for (int t0 = (blockIdx.x * RT_WARPS + warp) * TEAMS; t0 < a.T; t0 += gridDim.x * RT_WARPS * TEAMS) {
    const int t = t0 + team;
    const X* logits = static_cast<const X*>(a.logits) + static_cast<size_t>(t) * a.G;
    X* out = static_cast<X*>(a.d_logits) + static_cast<size_t>(t) * a.G;
    const size_t pair = static_cast<size_t>(t) * a.k + member;
    int e = -1;
    float d = 0.f;
    if (member < a.k && t < a.T) {
      e = __ldg(a.experts + pair);
      d = __ldg(a.d_weights + pair) * a.scale;
      if (e >= a.G || e < -1) {
        atomicCAS(a.status, 0u, ST_EXPERT_RANGE);
        e = -1;
      }
    }
    const float x = e >= 0 ? clean(read_logit(logits + e)) : -INFINITY;
    const bool there = x > -INFINITY;
    if (t < a.T) {
      if (whole) {
        for (int i = member * STEP; i < a.G; i += LANES * STEP)
          if (in_bounds(a, static_cast<size_t>(t) * a.G + i, STEP, static_cast<size_t>(a.T) * a.G))
            *reinterpret_cast<uint4*>(out + i) = make_uint4(0, 0, 0, 0);
      } else {
        for (int i = member; i < a.G; i += LANES) write_logit<X>(a, t, i, 0.f);
      }
    }
    if (!there) d = 0.f;
    float s, g;
    if (a.sigmoid) {
      s = there ? sigmoid(x) : 0.f;
      if (a.renormalize) {
        const float total = team_sum<LANES>(s) + kLeast;
        d = __fdiv_rn(d - team_sum<LANES>(d * __fdiv_rn(s, total)), total);
      }
      g = there ? d * s * sigmoid(-x) : 0.f;   // (1 - s without cancellation)
    } else {
      const uint32_t m = team_max<LANES>(there ? order_of(x) : 0);
      s = there ? expf(x - float_of(m)) : 0.f;
      const float total = team_sum<LANES>(s);
      s = there ? __fdiv_rn(s, total) : 0.f;
      g = s * (d - team_sum<LANES>(d * s));
    }
    // an expert that is named twice gets both, in order (the choices before a lane's own)
    bool first = true;
    float sum = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int ej = __shfl_sync(ALL, e, team * LANES + j);
      const float gj = __shfl_sync(ALL, g, team * LANES + j);
      if (ej == e) {
        sum += gj;
        first = first && j >= member;
      }
    }
    __syncwarp();   // (the zeros come before the values)
    if (e >= 0 && first) write_logit<X>(a, t, e, sum);
  }
}

// A softmax that is not renormalised: a warp a token, the row put together in shared
// memory.
template <class X>
__global__ void __launch_bounds__(32 * RT_WARPS)
route_backward_kernel(const RouteBwd a) {
  extern __shared__ float route_rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = route_rows + warp * a.G;
  grid_dep_wait();
  grid_dep_launch_dependents();
  for (int t = blockIdx.x * RT_WARPS + warp; t < a.T; t += gridDim.x * RT_WARPS) {
    const X* logits = static_cast<const X*>(a.logits) + static_cast<size_t>(t) * a.G;
    const size_t pair = static_cast<size_t>(t) * a.k + lane;
    int e = -1;
    float d = 0.f;
    if (lane < a.k) {
      e = __ldg(a.experts + pair);
      d = __ldg(a.d_weights + pair) * a.scale;
      if (e >= a.G || e < -1) {
        atomicCAS(a.status, 0u, ST_EXPERT_RANGE);
        e = -1;
      }
    }
    const float x = e >= 0 ? clean(read_logit(logits + e)) : -INFINITY;
    const bool there = x > -INFINITY;
    if (!there) d = 0.f;
    uint32_t m = 0;
    for (int i = lane; i < a.G; i += 32) {
      const float v = clean(read_logit(logits + i));
      if (v > -INFINITY) m = max(m, order_of(v));
      row[i] = 0.f;
    }
    m = __reduce_max_sync(ALL, m);
    const float top = m ? float_of(m) : 0.f;
    float sum = 0.f;
    for (int i = lane; i < a.G; i += 32) sum += expf(clean(read_logit(logits + i)) - top);
    sum = warp_sum(sum);
    const float share = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
    const float dot = warp_sum(there ? d * (expf(x - top) * share) : 0.f);
    __syncwarp();
    for (int j = 0; j < a.k; ++j) {
      const int ej = __shfl_sync(ALL, e, j);
      const float dj = __shfl_sync(ALL, d, j);
      // (the same lane for the same expert: its additions are in order)
      if (ej >= 0 && (ej & 31) == lane) row[ej] += dj;
    }
    __syncwarp();
    for (int i = lane; i < a.G; i += 32)
      write_logit<X>(a, t, i, expf(clean(read_logit(logits + i)) - top) * share * (row[i] - dot));
    __syncwarp();
  }
}

// Blocks for T tokens, `teams` of them to a warp.
int route_grid(int T, int teams, int num_sms, bool limited) {
  const int each = RT_WARPS * teams, blocks = (T - 1) / each + 1;
  return limited ? std::min(blocks, num_sms) : blocks;
}

template <class X, int NPL, int LANES>
cudaError_t launch_fwd(const RouteFwd& a, int num_sms, bool limited, cudaStream_t stream) {
  constexpr int TEAMS = 32 / LANES;
  RoutePlan p{};
  p.per = a.G / a.groups;
  p.per_inv = p.per > 1 ? 0xffffffffu / p.per + 1 : 0;
  p.grouped = a.groups > a.top_groups;
  p.lane_group = p.per % NPL == 0;
  p.whole = whole_rows<X, NPL>(a.logits, a.G);
  p.whole_bias = whole_rows<float, NPL>(a.bias, a.G);
  const int smem = p.grouped || a.bias ? RT_WARPS * TEAMS * a.G * 4 : 0;
  const bool logits = !a.bias && (!p.grouped || a.best == 1);
  return launch_dependent(logits ? route_kernel<X, NPL, LANES, true> : route_kernel<X, NPL, LANES, false>,
                          dim3(route_grid(a.T, TEAMS, num_sms, limited)), 32 * RT_WARPS, stream, smem, a, p);
}

template <class X>
cudaError_t launch_fwd(const RouteFwd& a, int num_sms, bool limited, cudaStream_t stream) {
  // a lane for each choice and each group at least; as few lanes, and registers for the
  // row of logits, as its length needs
  // (and one for what the last choice is compared with)
  const int least = std::max(a.k + 1, a.groups);
  if (a.G <= 8 && least <= 8) return launch_fwd<X, 1, 8>(a, num_sms, limited, stream);
  if (a.G <= 16 && least <= 8) return launch_fwd<X, 2, 8>(a, num_sms, limited, stream);
  if (a.G <= 32 && least <= 8) return launch_fwd<X, 4, 8>(a, num_sms, limited, stream);
  if (a.G <= 64 && least <= 16) return launch_fwd<X, 4, 16>(a, num_sms, limited, stream);
  if (a.G <= 64) return launch_fwd<X, 2, 32>(a, num_sms, limited, stream);
  if (a.G <= 128) return launch_fwd<X, 4, 32>(a, num_sms, limited, stream);
  if (a.G <= 256) return launch_fwd<X, 8, 32>(a, num_sms, limited, stream);
  if (a.G <= 512) return launch_fwd<X, 16, 32>(a, num_sms, limited, stream);
  return launch_fwd<X, 32, 32>(a, num_sms, limited, stream);
}

template <class X>
cudaError_t launch_bwd(const RouteBwd& a, int num_sms, bool limited, cudaStream_t stream) {
  if (!a.sigmoid && !a.renormalize)
    return launch_dependent(route_backward_kernel<X>, dim3(route_grid(a.T, 1, num_sms, limited)),
                            32 * RT_WARPS, stream, RT_WARPS * a.G * 4, a);
  const bool whole = a.G % (16 / sizeof(X)) == 0 && (reinterpret_cast<uintptr_t>(a.d_logits) & 15) == 0;
  const int lanes = a.k <= 8 ? 8 : a.k <= 16 ? 16 : 32;
  const dim3 grid(route_grid(a.T, 32 / lanes, num_sms, limited));
  auto go = [&](auto kernel) { return launch_dependent(kernel, grid, 32 * RT_WARPS, stream, 0, a, whole); };
  return lanes == 8    ? go(route_backward_few_kernel<X, 8>)
         : lanes == 16 ? go(route_backward_few_kernel<X, 16>)
                       : go(route_backward_few_kernel<X, 32>);
}

}  // namespace

cudaError_t launch_route(const RouteFwd& a, bool bf16, int num_sms, bool limited, cudaStream_t stream) {
  return bf16 ? launch_fwd<__nv_bfloat16>(a, num_sms, limited, stream)
              : launch_fwd<float>(a, num_sms, limited, stream);
}

cudaError_t launch_route_backward(const RouteBwd& a, bool bf16, int num_sms, bool limited,
                                  cudaStream_t stream) {
  return bf16 ? launch_bwd<__nv_bfloat16>(a, num_sms, limited, stream)
              : launch_bwd<float>(a, num_sms, limited, stream);
}

}  // namespace dgk
