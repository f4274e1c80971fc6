// Routing of tokens to experts, and its gradient.  Per token, of its G logits x
// and the experts' bias b:
//
//   s_e = 1 / (1 + exp(-x_e)), or softmax(x)_e;   c_e = s_e + b_e
//   of n groups of consecutive experts the m with the largest value stay, a
//   group's value the sum of its (one or two) largest c
//   the k largest c among them are chosen, equal ones by their index
//   w_j = scale s_j, or scale s_j / (sum of the chosen s)
//
// A warp takes a token, a lane every 32nd expert: the k largest are k rounds of
// a maximum over the warp (redux on the values' order as unsigned integers, then
// on the index among the lanes that hold it).
//
// The choice is that of the formulas in 64 bits, whatever the rounding here: where all
// biases are equal it is made by the logits themselves (both scores rise with
// them), else by c in fp32, and a token with two values nearer to each other
// than their errors, at a place where that decides, is chosen again in 64 bits
// (choose_exact; about one token in a thousand of 256 experts).
//
// Bounded by latency and by instructions, not by memory.
#include <float.h>

#include <algorithm>

#include <cuda_bf16.h>

#include "dg_launch.h"
#include "dg_params.h"
#include "dg_route.h"
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
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmax(v, __shfl_xor_sync(ALL, v, o));
  return v;
}

// (by exp(-|x|), which does not overflow)
__device__ __forceinline__ float sigmoid(float x) {
  const float e = expf(-fabsf(x));
  return __fdiv_rn(x < 0.f ? e : 1.f, 1.f + e);
}

// Largest (value, lowest index) over the warp; -1 where all are -infinity.
__device__ __forceinline__ int warp_argmax(double v, int index) {
  const double top = warp_max(v);
  return top == -INFINITY ? -1
                          : static_cast<int>(__reduce_min_sync(
                                ALL, v == top ? static_cast<unsigned>(index) : 0x7fffffffu));
}

// The token's choice in 64 bits: lane j returns the j-th expert.
template <class X, int NPL>
__device__ __noinline__ int choose_exact(const RouteFwd& a, const X* logits) {
  const int lane = threadIdx.x & 31;
  double c[NPL];
  double top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 32 * i;
    c[i] = e < a.G ? static_cast<double>(clean(read_logit(logits + e))) : -INFINITY;
    top = fmax(top, c[i]);
  }
  if (!a.sigmoid) {
    top = warp_max(top);
    double sum = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (c[i] != -INFINITY) sum += exp(c[i] - top);
    sum = warp_sum(sum);
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (c[i] != -INFINITY) c[i] = exp(c[i] - top) / sum;
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (c[i] != -INFINITY) c[i] = 1.0 / (1.0 + exp(-c[i]));
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 32 * i;
    if (a.bias && e < a.G) c[i] += static_cast<double>(__ldg(a.bias + e));
    if (!(c[i] > -INFINITY)) c[i] = -INFINITY;
  }
  if (a.groups > a.top_groups) {
    const int per = a.G / a.groups;
    double mine = -INFINITY;   // lane g: group g's value
    for (int g = 0; g < a.groups; ++g) {
      double one = -INFINITY, two = -INFINITY;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        if (e >= g * per && e < (g + 1) * per) {
          two = fmax(two, fmin(one, c[i]));
          one = fmax(one, c[i]);
        }
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        const double p = __shfl_xor_sync(ALL, one, o), q = __shfl_xor_sync(ALL, two, o);
        two = fmax(fmax(two, q), fmin(one, p));
        one = fmax(one, p);
      }
      if (lane == g) mine = a.best == 2 && two != -INFINITY ? one + two : one;
    }
    uint32_t keep = 0;
    for (int n = 0; n < a.top_groups; ++n) {
      const int g = warp_argmax((keep >> lane) & 1u || lane >= a.groups ? -INFINITY : mine, lane);
      if (g < 0) break;
      keep |= 1u << g;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      if (e < a.G && !((keep >> (e / per)) & 1u)) c[i] = -INFINITY;
    }
  }
  int chosen = -1;
  for (int j = 0; j < a.k; ++j) {
    double v = -INFINITY;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (c[i] > v) { v = c[i]; at = lane + 32 * i; }
    const int e = warp_argmax(v, at);
    if (lane == j) chosen = e;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (e == lane + 32 * i) c[i] = -INFINITY;
  }
  return chosen;
}

// More than what the difference of two c near `c` may be off by in fp32, `bias`
// the largest bias' magnitude.  A sigmoid: 2^-22 of 1 (expf, the sum, the quotient)
// each.  A softmax's s: expf by 2^-22 of itself and by |x - max| 2^-24 (its
// argument's rounding, |x - max| at most 88, and at most -ln s), the sum, common to
// both, by 44 2^-24 (its roundings and its terms').  Each c: 2^-24 of itself.
__device__ __forceinline__ float doubt(bool sigmoid, float c, float bias) {
  const float s = sigmoid ? 0x1p-20f : fminf(0x1p-18f, 0x1p-16f * (fabsf(c) + bias));
  return s + 0x1p-22f * fabsf(c);
}

// NPL: experts per lane.
template <class X, int NPL>
__global__ void __launch_bounds__(32 * RT_WARPS)
route_kernel(const RouteFwd a) {
  extern __shared__ uint32_t route_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* row = route_smem + warp * a.G;   // (with groups) the values' order
  grid_dep_wait();
  grid_dep_launch_dependents();
  // all biases equal: the choice is by the logits
  bool even = true;
  float bias_most = 0.f;
  if (a.bias) {
    const float first = __ldg(a.bias);
    bool same = first > -INFINITY;
    for (int e = lane; e < a.G; e += 32) {
      const float b = __ldg(a.bias + e);
      same = same && b == first;
      bias_most = fmaxf(bias_most, fabsf(b));
    }
    even = __all_sync(ALL, same);
    bias_most = __uint_as_float(__reduce_max_sync(ALL, __float_as_uint(bias_most)));
  }
  const bool grouped = a.groups > a.top_groups;
  const bool by_logit = even && (!grouped || a.best == 1);
  const int per = a.G / a.groups;
  for (int t = blockIdx.x * RT_WARPS + warp; t < a.T; t += gridDim.x * RT_WARPS) {
    const X* logits = static_cast<const X*>(a.logits) + static_cast<size_t>(t) * a.G;
    float x[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      x[i] = e < a.G ? clean(read_logit(logits + e)) : -INFINITY;
    }
    uint32_t key[NPL];   // order of c, or of the logit; 0: not available
    uint32_t key_top = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      key[i] = x[i] > -INFINITY ? order_of(x[i]) : 0;
      key_top = max(key_top, key[i]);
    }
    // the scores are needed in full for c, or for a softmax's sum
    float top = 0.f, sum = 1.f;
    if (!a.sigmoid && !(by_logit && a.renormalize)) {
      key_top = __reduce_max_sync(ALL, key_top);
      top = key_top ? float_of(key_top) : 0.f;
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const float s = expf(x[i] - top);   // (0 for -infinity)
        sum += s;
        if (!by_logit) x[i] = key[i] ? s : -INFINITY;
      }
      sum = warp_sum(sum);
    } else if (!by_logit) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) x[i] = key[i] ? sigmoid(x[i]) : -INFINITY;
    }
    if (!by_logit) {
      const float share = a.sigmoid ? 1.f : __frcp_rn(sum);
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        const float c = e < a.G ? fmaf(x[i], share, a.bias ? __ldg(a.bias + e) : 0.f) : -INFINITY;
        key[i] = c > -INFINITY ? order_of(c) : 0;
      }
    }
    bool sure = true;
    if (grouped) {
      // 32 / groups lanes (a power of two) to a group's two largest values
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (lane + 32 * i < a.G) row[lane + 32 * i] = key[i];
      __syncwarp();
      const int width = 1 << (31 - __clz(32 / a.groups));
      const int g = lane / width;
      uint32_t one = 0, two = 0;
      if (g < a.groups)
        for (int e = lane & (width - 1); e < per; e += width) {
          const uint32_t v = row[g * per + e];
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
      uint32_t keep = 0;
      const bool mine = g < a.groups && (lane & (width - 1)) == 0;
      uint32_t last = 0, left = mine ? value : 0;
      for (int n = 0; n < a.top_groups; ++n) {
        const uint32_t v = __reduce_max_sync(ALL, left);
        if (v == 0) break;
        const unsigned who = __reduce_min_sync(ALL, left == v ? static_cast<unsigned>(lane) : 32u);
        keep |= 1u << (who / width);
        if (lane == static_cast<int>(who)) left = 0;
        last = v;
      }
      const uint32_t next = __reduce_max_sync(ALL, left);
      if (!by_logit && next) {
        const float l = float_of(last), n = float_of(next);
        sure = l - n > 2.f * doubt(a.sigmoid, fmaxf(fabsf(l), fabsf(n)), bias_most);
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        if (e < a.G && !((keep >> (e / per)) & 1u)) key[i] = 0;
      }
    }
    // k rounds, and one more for what the last choice was close to
    int chosen = -1;
    const int rounds = by_logit ? a.k : a.k + 1;
    uint32_t before = 0;
    for (int j = 0; j < rounds; ++j) {
      uint32_t v = 0;
      int at = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (key[i] > v) { v = key[i]; at = i; }
      const uint32_t best = __reduce_max_sync(ALL, v);
      if (best == 0) break;
      if (!by_logit && j > 0) {
        const float l = float_of(before), n = float_of(best);
        sure = sure && l - n > doubt(a.sigmoid, fmaxf(fabsf(l), fabsf(n)), bias_most);
      }
      before = best;
      const unsigned e =
          __reduce_min_sync(ALL, v == best ? static_cast<unsigned>(lane + 32 * at) : 0x7fffffffu);
      if (lane == j && j < a.k) chosen = static_cast<int>(e);
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (e == static_cast<unsigned>(lane + 32 * i)) key[i] = 0;
    }
    if (!sure) chosen = choose_exact<X, NPL>(a, logits);
    // weights: lane j that of the j-th choice
    const bool there = lane < a.k && chosen >= 0;
    const float y = there ? clean(read_logit(logits + chosen)) : -INFINITY;
    float s;
    if (a.sigmoid) {
      s = there ? sigmoid(y) : 0.f;
      if (a.renormalize) s = __fdiv_rn(s, warp_sum(s) + kLeast);
    } else if (a.renormalize) {
      // (relative to the largest chosen: no underflow of them all)
      const uint32_t m = __reduce_max_sync(ALL, there ? order_of(y) : 0);
      s = there ? expf(y - float_of(m)) : 0.f;
      const float total = warp_sum(s);
      s = there ? __fdiv_rn(s, total) : 0.f;
    } else {
      s = there ? __fdiv_rn(expf(y - top), sum) : 0.f;
    }
    if (lane < a.k) {
      const size_t at = static_cast<size_t>(t) * a.k + lane;
      a.experts[at] = chosen;
      a.weights[at] = s * a.scale;
    }
  }
}

__device__ __forceinline__ void write_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void write_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Gradient of the logits, the choice taken as it is.  With d_j the gradient of
// w_j times the scale:
//   renormalised: ds_j = (d_j - sum_i d_i s_i / S) / S, S the sum of the chosen s
//   sigmoid: dx = ds s (1 - s);  softmax: dx_e = s_e (ds_e - sum_i ds_i s_i)
// In the renormalised softmax the last sum vanishes, so that, as with sigmoid
// scores, only the chosen logits have a gradient and only they are read.  The row
// is put together in shared memory (an expert that is named twice gets both
// contributions, in order).
template <class X>
__global__ void __launch_bounds__(32 * RT_WARPS)
route_backward_kernel(const RouteBwd a) {
  extern __shared__ float route_rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = route_rows + warp * a.G;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const bool few = a.sigmoid || a.renormalize;
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
    for (int i = lane; i < a.G; i += 32) row[i] = 0.f;
    float x = e >= 0 ? clean(read_logit(logits + e)) : -INFINITY;
    const bool there = x > -INFINITY;
    if (!there) d = 0.f;
    float s = 0.f, g, top = 0.f, share = 0.f;
    if (a.sigmoid) {
      s = there ? sigmoid(x) : 0.f;
      if (a.renormalize) {
        const float total = warp_sum(s) + kLeast;
        d = __fdiv_rn(d - warp_sum(d * __fdiv_rn(s, total)), total);
      }
      g = there ? d * s * sigmoid(-x) : 0.f;   // (1 - s without cancellation)
    } else if (a.renormalize) {
      const uint32_t m = __reduce_max_sync(ALL, there ? order_of(x) : 0);
      s = there ? expf(x - float_of(m)) : 0.f;
      const float total = warp_sum(s);
      s = there ? __fdiv_rn(s, total) : 0.f;
      g = s * (d - warp_sum(d * s));
    } else {
      uint32_t m = 0;
      for (int i = lane; i < a.G; i += 32) {
        const float v = clean(read_logit(logits + i));
        if (v > -INFINITY) m = max(m, order_of(v));
      }
      m = __reduce_max_sync(ALL, m);
      top = m ? float_of(m) : 0.f;
      float sum = 0.f;
      for (int i = lane; i < a.G; i += 32) sum += expf(clean(read_logit(logits + i)) - top);
      sum = warp_sum(sum);
      share = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
      s = there ? expf(x - top) * share : 0.f;
      g = d;   // ds: the row's other term follows below
    }
    const float dot = few ? 0.f : warp_sum(d * s);
    __syncwarp();
    for (int j = 0; j < a.k; ++j) {
      const int ej = __shfl_sync(ALL, e, j);
      const float gj = __shfl_sync(ALL, g, j);
      // (the same lane for the same expert: its additions are in order)
      if (ej >= 0 && (ej & 31) == lane) row[ej] += gj;
    }
    __syncwarp();
    X* out = static_cast<X*>(a.d_logits) + static_cast<size_t>(t) * a.G;
    for (int i = lane; i < a.G; i += 32) {
      float v = row[i];
      if (!few) v = expf(clean(read_logit(logits + i)) - top) * share * (v - dot);
      write_logit(out + i, v);
    }
    __syncwarp();
  }
}

int route_grid(int T, int num_sms, bool limited) {
  const int blocks = (T - 1) / RT_WARPS + 1;
  return limited ? std::min(blocks, num_sms) : std::min(blocks, 8 * num_sms);
}

template <class X>
cudaError_t launch_fwd(const RouteFwd& a, int num_sms, bool limited, cudaStream_t stream) {
  const dim3 grid(route_grid(a.T, num_sms, limited));
  const int smem = a.groups > a.top_groups ? RT_WARPS * a.G * 4 : 0;
  auto go = [&](auto kernel) { return launch_dependent(kernel, grid, 32 * RT_WARPS, stream, smem, a); };
  // registers for the row of logits: as many as its length needs
  if (a.G <= 32) return go(route_kernel<X, 1>);
  if (a.G <= 64) return go(route_kernel<X, 2>);
  if (a.G <= 128) return go(route_kernel<X, 4>);
  if (a.G <= 256) return go(route_kernel<X, 8>);
  if (a.G <= 512) return go(route_kernel<X, 16>);
  return go(route_kernel<X, 32>);
}

}  // namespace

cudaError_t launch_route(const RouteFwd& a, bool bf16, int num_sms, bool limited, cudaStream_t stream) {
  return bf16 ? launch_fwd<__nv_bfloat16>(a, num_sms, limited, stream)
              : launch_fwd<float>(a, num_sms, limited, stream);
}

cudaError_t launch_route_backward(const RouteBwd& a, bool bf16, int num_sms, bool limited,
                                  cudaStream_t stream) {
  const dim3 grid(route_grid(a.T, num_sms, limited));
  const int smem = RT_WARPS * a.G * 4;
  return bf16 ? launch_dependent(route_backward_kernel<__nv_bfloat16>, grid, 32 * RT_WARPS, stream, smem, a)
              : launch_dependent(route_backward_kernel<float>, grid, 32 * RT_WARPS, stream, smem, a);
}

}  // namespace dgk
