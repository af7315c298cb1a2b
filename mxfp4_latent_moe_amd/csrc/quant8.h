// e4m3 activations with one power-of-two scale per row and block of 128
// inputs: the block's arithmetic, shared by the kernels that write them.
//
// The scale 2^e is the smallest power of two with max|v| <= 448 * 2^e (448 is
// the largest e4m3 value), so v / 2^e is exact and the one rounding is the
// conversion to e4m3 (to nearest, ties to even).  The maximum is taken over
// the block's finite values; values that are not finite become the NaN code.
// e is held to [-126, 127] and stored as the byte e + 127; a block of zeros
// stores 1 (e = -126).
#pragma once
#include "common.h"

namespace moe {

constexpr int Q8_BLOCK = 128;

MOE_DEV float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= 3.4028234663852886e38f ? a : 0.f;  // false for NaN and infinity
}

// the scale byte e + 127 of a block whose largest finite magnitude is amax
MOE_DEV uint32_t q8_scale_byte(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  // amax = 1.m * 2^(E - 127); 1.m * 2^8 <= 448 iff 1.m <= 1.75
  const int b = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(b < 1 ? 1 : b);
}
// 2^-e for the byte e + 127 in 1..247
MOE_DEV float q8_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// four values as e4m3 codes, low byte first
MOE_DEV uint32_t q8_pack4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
  const float v[4] = {a, b, c, d};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!(fabsf(v[i]) <= 3.4028234663852886e38f)) w = (w & ~(0xFF << (8 * i))) | (0x7F << (8 * i));
  return (uint32_t)w;
}

}  // namespace moe
