// Conversions and the 1x128 scale arithmetic shared by the kernels that write
// or read e4m3 activations (the quantiser, the norm, the gated activation).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dgk {

constexpr float kScaleFloor = 1e-4f;  // smallest group maximum a scale is made from
// largest one: values computed from bf16 ones (a norm's, an activation's) may pass
// fp32; with it a scale stays finite and they get the largest code of their sign
constexpr float kScaleTop = 3.402823466e38f;

// two fp32 -> two e4m3 codes (round to nearest even, saturating to +-448),
// `lo` in the low byte
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d) {
  return cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
}

// two e4m3 codes (low byte first) -> two fp32, exactly (every e4m3 value is a
// binary16 value)
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  __half2_raw r;
  r.x = static_cast<uint16_t>(h);
  r.y = static_cast<uint16_t>(h >> 16);
  return __half22float2(__half2(r));
}

__device__ __forceinline__ uint4 ld_stream_v4(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// eight bf16 values (16 bytes) -> fp32
__device__ __forceinline__ void bf16x8_to_float(const uint4& v, float* x) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x);
  x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z);
  x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}

// eight fp32 -> bf16 (round to nearest even), 16 bytes
__device__ __forceinline__ uint4 float_to_bf16x8(const float* x) {
  uint4 v;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.x) : "f"(x[1]), "f"(x[0]));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.y) : "f"(x[3]), "f"(x[2]));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.z) : "f"(x[5]), "f"(x[4]));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.w) : "f"(x[7]), "f"(x[6]));
  return v;
}

// Two fp32 products or sums in one instruction (round to nearest, the same
// results as one by one).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// a b + c
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// Eight values as four pairs.
struct Pairs {
  float2 v[4];
};
__device__ __forceinline__ Pairs bf16x8_to_pairs(const uint4& w) {
  return Pairs{{make_float2(bf16_lo(w.x), bf16_hi(w.x)), make_float2(bf16_lo(w.y), bf16_hi(w.y)),
                make_float2(bf16_lo(w.z), bf16_hi(w.z)), make_float2(bf16_lo(w.w), bf16_hi(w.w))}};
}
__device__ __forceinline__ uint4 pairs_to_bf16x8(const Pairs& p) {
  uint4 w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(p.v[0].y), "f"(p.v[0].x));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(p.v[1].y), "f"(p.v[1].x));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.z) : "f"(p.v[2].y), "f"(p.v[2].x));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.w) : "f"(p.v[3].y), "f"(p.v[3].x));
  return w;
}
// e4m3 codes of the values times f
__device__ __forceinline__ uint2 pairs_to_e4m3x8(const Pairs& p, float f) {
  const float2 f2 = make_float2(f, f);
  const float2 a = mul2(p.v[0], f2), b = mul2(p.v[1], f2), c = mul2(p.v[2], f2), d = mul2(p.v[3], f2);
  return make_uint2(cvt_e4m3x4(a.x, a.y, b.x, b.y), cvt_e4m3x4(c.x, c.y, d.x, d.y));
}
// the values of eight codes times s
__device__ __forceinline__ Pairs e4m3x8_to_pairs(const uint2& w, float s) {
  const float2 s2 = make_float2(s, s);
  return Pairs{{mul2(e4m3x2_to_float2(w.x & 0xFFFFu), s2), mul2(e4m3x2_to_float2(w.x >> 16), s2),
                mul2(e4m3x2_to_float2(w.y & 0xFFFFu), s2), mul2(e4m3x2_to_float2(w.y >> 16), s2)}};
}
__device__ __forceinline__ float pairs_amax(const Pairs& p) {
  return fmaxf(fmaxf(fmaxf(fabsf(p.v[0].x), fabsf(p.v[0].y)), fmaxf(fabsf(p.v[1].x), fabsf(p.v[1].y))),
               fmaxf(fmaxf(fabsf(p.v[2].x), fabsf(p.v[2].y)), fmaxf(fabsf(p.v[3].x), fabsf(p.v[3].y))));
}
// largest magnitude of eight bf16 values, exactly
__device__ __forceinline__ float bf16x8_amax(const uint4& w) {
  auto mag = [](uint32_t x) {
    __nv_bfloat162_raw r;
    r.x = static_cast<uint16_t>(x);
    r.y = static_cast<uint16_t>(x >> 16);
    return __habs2(__nv_bfloat162(r));
  };
  const float2 m = __bfloat1622float2(
      __hmax2(__hmax2(mag(w.x), mag(w.y)), __hmax2(mag(w.z), mag(w.w))));
  return fmaxf(m.x, m.y);
}

// The factor a group's values are multiplied by before the conversion to
// e4m3, from its maximum a (floored, finite): 448 / a, or with UE8M0 scales 1 / s with
// s the smallest power of two >= a / 448, whose exponent code is e8.
template <bool UE8M0>
__device__ __forceinline__ void group_factor(float a, float& factor, uint32_t& e8) {
  e8 = 0;
  if constexpr (UE8M0) {
    // t = a / 448 is a normal fp32 number here (1e-4 <= a <= the largest finite
    // fp32 number, so e8 <= 247); its power-of-two ceiling is 2^(E - 127) when the mantissa is zero, else
    // 2^(E - 126), E the biased exponent; the factor 1 / s is exact
    const uint32_t tb = __float_as_uint(__fdiv_rn(a, 448.0f));
    e8 = ((tb >> 23) & 0xFFu) + ((tb & 0x7FFFFFu) != 0u ? 1u : 0u);
    factor = __uint_as_float((254u - e8) << 23);
  } else {
    factor = __fdiv_rn(448.0f, a);
  }
}

// Stores the scale of row m and group g of batch z: fp32 a / 448 in
// sa[z][g][ld_sa], or byte g % 4 of the packed word [z][g / 4][m].
template <bool UE8M0>
__device__ __forceinline__ void store_scale(float* sa, int z, int kb, int ld_sa, int g, int m,
                                            float a, uint32_t e8) {
  if constexpr (UE8M0) {
    const int kbp = (kb + 3) >> 2;
    reinterpret_cast<uint8_t*>(sa)[((static_cast<size_t>(z) * kbp + (g >> 2)) * ld_sa + m) * 4 +
                                   (g & 3)] = static_cast<uint8_t>(e8);
  } else {
    sa[(static_cast<size_t>(z) * kb + g) * ld_sa + m] = __fdiv_rn(a, 448.0f);
  }
}

}  // namespace dgk
