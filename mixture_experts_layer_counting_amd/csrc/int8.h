// INT8 with one fp32 scale per row (activations) or per output column (weights).
//   scale  s = max(fl32(amax / 127), 2^-120); 1 for an all-zero row, NaN where the row holds a NaN or
//          an infinity (its codes are then 0)
//   code   q = nearest integer to x / s, ties to even, as if in infinite precision; |q| <= 127
// The floor 2^-120 keeps s and the border (n + 1/2) s normal numbers, so that the comparison of a
// value with a border below is exact. It is reached by rows whose largest value is below 127 * 2^-120.
#pragma once
#include "moe_common.h"

namespace moe {

// Largest magnitude as the bits of |x| (NaN and infinity compare above every finite value).
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ float int8_scale(uint32_t amax_bits) {
  if (amax_bits == 0) return 1.0f;
  if (amax_bits >= 0x7f800000u) return __builtin_nanf("");
  const float s = __fdiv_rn(__uint_as_float(amax_bits), 127.0f);
  return s < 0x1p-120f ? 0x1p-120f : s;
}

// x / s by one product with inv = fl32(1 / s) is off by less than 2^-14 (|x / s| <= 127.01, three
// roundings of 2^-24): only a quotient that lands within 2^-13 of a half step can round the wrong
// way. There the border b = n + 1/2 is compared with x itself: b s has at most 32 significant
// bits and fma rounds once, so the sign of x - b s is exact.
__device__ __forceinline__ float int8_code(float x, float s, float inv) {
  const float v = x * inv;
  float r = __builtin_rintf(v);
  const float d = v - r;
  if (__builtin_fabsf(d) > 0.5f - 0x1p-13f) {
    const float b = r + __builtin_copysignf(0.5f, d);
    const float e = __builtin_fmaf(-b, s, x);
    r = e > 0.f ? b + 0.5f : e < 0.f ? b - 0.5f : 2.0f * __builtin_rintf(0.5f * b);
  }
  return r;
}

__device__ __forceinline__ uint32_t pack_i8x4(float a, float b, float c, float d) {
  return ((uint32_t)(int)a & 0xffu) | ((uint32_t)(int)b & 0xffu) << 8 | ((uint32_t)(int)c & 0xffu) << 16 |
         (uint32_t)(int)d << 24;
}

__device__ __forceinline__ float i8_at(uint32_t w, int i) { return (float)((int)(w << (24 - 8 * i)) >> 24); }

}  // namespace moe
