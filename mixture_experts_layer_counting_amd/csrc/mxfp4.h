// MXFP4 (OCP Microscaling: e2m1 codes, one e8m0 scale per 32 elements) on the device.
//
// A block's scale is X = 2^(floor(log2 amax) - 2), the largest power of two under which amax / X
// stays below 8, so that the largest element lands on 4 or 6; codes are e2m1
// round-to-nearest-even of v / X, saturating at 6. The scale byte is X's biased exponent:
// amax's own exponent field less 2, at least 0 (an all-zero or subnormal block: 2^-127). X is a
// power of two, so v / X is exact and the codes do not depend on evaluation order. A block that
// holds an infinity or a NaN has no such scale: it gets byte 255, the format's NaN, and zero
// codes, so all its values read back as NaN.
#pragma once

#include "moe_common.h"

namespace moe {

constexpr uint32_t MX_NAN_SCALE = 255;

// Scale byte of a block from the bits of max |v| (NaN and infinity compare above every number).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t f = amax_bits >> 23;
  return f == 255u ? MX_NAN_SCALE : f > 2u ? f - 2u : 0u;
}

// The scale as fp32: 2^(b - 127); byte 0 is the subnormal 2^-127, byte 255 NaN.
__device__ __forceinline__ float mx_scale_f32(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == MX_NAN_SCALE ? 0x7fc00000u : b << 23);
}

// Eight values -> eight codes in k order, low nibble first, for the block's scale byte
// (v_cvt_scalef32_pk_fp4_f32 divides by the scale's exponent and rounds to nearest even,
// saturating; adding +0 turns -0 into +0, so an exact zero has code 0).
__device__ __forceinline__ uint32_t mx_pack8(const float* v, uint32_t byte) {
  const float s = mx_scale_f32(byte);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] + 0.0f, v[1] + 0.0f, s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] + 0.0f, v[3] + 0.0f, s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] + 0.0f, v[5] + 0.0f, s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] + 0.0f, v[7] + 0.0f, s, 3);
  return byte == MX_NAN_SCALE ? 0u : r;
}

// The two values of byte SEL of w times x (exact in fp32 and, its mantissa being two bits, in
// bf16).
template <int SEL>
__device__ __forceinline__ void mx_unpack2(uint32_t w, float x, float& lo, float& hi) {
  const auto v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, SEL);
  lo = v[0] * x;
  hi = v[1] * x;
}

}  // namespace moe
