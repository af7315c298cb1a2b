// MXFP4: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), one power-of-two
// scale per block of 32 values, stored as its exponent byte e + 127: the
// block's arithmetic, shared by the kernels that write such rows.
//
// Two rules for the scale of a block whose largest magnitude is amax:
//   fit   the smallest 2^e with amax <= 6 2^e: no value saturates
//   ocp   2^(floor(log2 amax) - 2), the MX format's own: magnitudes above
//         6 2^e become 6 2^e
// Either way v / 2^e is exact and the one rounding is to e2m1 (to nearest, ties
// to even).  e is held to [-125, 126], so that every code but zero stands for a
// normal number; a block of zeros has e = -125.  e2m1 has no code for values
// that are not finite: a block that holds one gets the scale byte 255, NaN.
#pragma once
#include "common.h"

namespace moe {

constexpr int MX4_BLOCK = 32;

// the scale byte of a block from the bits of its largest magnitude
MOE_DEV uint32_t mx4_scale_byte(uint32_t amax, bool ocp) {
  // amax = 1.m * 2^(E - 127); 1.m * 4 <= 6 iff 1.m <= 1.5
  const int b = (int)(amax >> 23) - 2 + (!ocp && (amax & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return amax >= 0x7F800000u ? 255u : (uint32_t)(b < 2 ? 2 : b);
}
// 2^-e for the byte e + 127 in 2..253; 0 for 255
MOE_DEV float mx4_inverse(uint32_t byte) { return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23); }
// 2^e for any byte: 0 is the subnormal 2^-127, 255 is NaN
MOE_DEV float mx4_scale(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// eight values, already over their scale, as codes, the first in the low bits
template <typename V>
MOE_DEV uint32_t mx4_codes(const V &v) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], 1.0f, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], 1.0f, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], 1.0f, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], 1.0f, 3);
  return q;
}

}  // namespace moe
