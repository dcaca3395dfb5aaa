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

// Codes of n values with their scales s and inv = fl32(1 / s), as the low bytes of code[].
// x inv, rounded once to an integer by the addition of 1.5 * 2^23 (whose low byte is then the code), is off
// from x / s by less than 2^-16 (|x / s| <= 127.01, inv by 2^-24 of it): only a quotient within 2^-13 of a
// half step can round the wrong way. There the border b = n + 1/2 is compared with x itself: b s has at most 32 significant
// bits and fma rounds once, so the sign of x - b s is exact. `bad`: some inv is 0, a column with a NaN or an
// infinity, whose codes are 0.
template <int N, int NS>
__device__ __forceinline__ void int8_codes(const float (&x)[N], const float (&s)[NS], const float (&inv)[NS], bool bad,
                                           uint32_t (&code)[N]) {
  constexpr float M = 12582912.0f;
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = __builtin_fmaf(x[i], inv[i % NS], M);
    code[i] = __float_as_uint(t);
    off = __builtin_fmaxf(off, __builtin_fabsf(__builtin_fmaf(x[i], inv[i % NS], -(t - M))));
  }
  if (bad || off > 0.5f - 0x1p-13f) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float si = s[i % NS], ii = inv[i % NS];
      float r = __uint_as_float(code[i]) - M;
      const float d = __builtin_fmaf(x[i], ii, -r);
      if (__builtin_fabsf(d) > 0.5f - 0x1p-13f) {
        const float b = r + __builtin_copysignf(0.5f, d);
        const float e = __builtin_fmaf(-b, si, x[i]);
        r = e > 0.f ? b + 0.5f : e < 0.f ? b - 0.5f : 2.0f * __builtin_rintf(0.5f * b);
      }
      code[i] = ii == 0.f ? 0u : __float_as_uint(r + M);
    }
  }
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u), __builtin_amdgcn_perm(b, a, 0x0c0c0400u),
                               0x05040100u);
}

__device__ __forceinline__ float i8_at(uint32_t w, int i) { return (float)((int)(w << (24 - 8 * i)) >> 24); }

}  // namespace moe
