// e4m3.cuh -- 8-bit codes of the quantised prefix cache: conversions, and the
// page scale.
#pragma once

#include <stdint.h>

namespace losa {

// Two fp32 values -> two e4m3 codes (round to nearest even; beyond 448 and
// infinities -> 448; NaN -> NaN), `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four codes, byte i from value i.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// Four fp32 values -> four e5m2 codes (5 exponent bits, bias 15, and 2 mantissa
// bits; round to nearest even), byte i from value i.
__device__ __forceinline__ uint32_t e5m2x4(float a, float b, float c, float d) {
  unsigned short lo, hi;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return lo | (static_cast<uint32_t>(hi) << 16);
}
// Four codes -> fp16 pairs (codes 0, 1) and (codes 2, 3).
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
      " cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}
// Four codes -> bf16 pairs (codes 0, 1) and (codes 2, 3), exact (an e4m3 number has
// 4 significant bits, so the upper halves of the fp32 numbers hold all of it).
__device__ __forceinline__ void e4m3x4_to_bf16x2(uint32_t c, uint32_t& lo, uint32_t& hi) {
  uint32_t a, b;
  e4m3x4_to_f16x2(c, a, b);
  const float2 x = f16x2_to_f32(a), y = f16x2_to_f32(b);
  lo = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
  hi = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
}
__device__ __forceinline__ uint32_t f16x2_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four codes as fp32 (exact).
__device__ __forceinline__ float4 e4m3x4_to_f32(uint32_t c) {
  uint32_t lo, hi;
  e4m3x4_to_f16x2(c, lo, hi);
  const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
  return make_float4(a.x, a.y, b.x, b.y);
}

// The scale of a page whose largest finite magnitude is `amax` (>= 0): the
// smallest power of two >= 2^-100 with amax <= 448 * scale, at most 2^119; 1
// for a page of zeros.  448 = 1.75 * 2^8, so with amax = m 2^e, 1 <= m < 2,
// the exponent is e - 8, one more when m > 1.75.
__device__ __forceinline__ int page_scale_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return amax == 0.f ? 0 : min(max(e, -100), 119);
}
__device__ __forceinline__ float exp2_int(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

}  // namespace losa
