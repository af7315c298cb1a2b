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

// the scale byte e + 127 of a block whose largest finite magnitude is amax
MOE_DEV uint32_t q8_scale_byte(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  // amax = 1.m * 2^(E - 127); 1.m * 2^8 <= 448 iff 1.m <= 1.75
  const int b = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(b < 1 ? 1 : b);
}
// 2^-e for the byte e + 127 in 1..247
MOE_DEV float q8_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// the maximum over 16 neighbouring lanes (a row of the cross-lane unit)
MOE_DEV uint32_t max16(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));   // lanes 1 0 3 2
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));   // 2 3 0 1
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));  // 7 .. 0 of each half
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));  // 15 .. 0
}

// Eight values of a lane, 16 lanes a block, as e4m3 codes (lo: the first four,
// low byte first); returns the block's scale byte.  All lanes of the wave take
// part.  Magnitudes compare as their bit patterns, which also shows values that
// are not finite: waves without any (all, as a rule) skip their treatment.
template <typename V>
MOE_DEV uint32_t q8_block(const V &v, uint32_t &lo, uint32_t &hi) {
  constexpr uint32_t INF = 0x7F800000u;
  uint32_t a[8], m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = max(m, a[i]);
  }
  const bool finite = __ballot(m >= INF) == 0;
  if (!finite) {
    m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, a[i] < INF ? a[i] : 0u);
  }
  const uint32_t sb = q8_scale_byte(__uint_as_float(max16(m)));
  const float inv = q8_inverse(sb);
  int w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, 0, false);
    w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, w[h], true);
  }
  if (!finite) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (a[i] >= INF) w[i >> 2] = (w[i >> 2] & ~(0xFF << (8 * (i & 3)))) | (0x7F << (8 * (i & 3)));
  }
  lo = (uint32_t)w[0];
  hi = (uint32_t)w[1];
  return sb;
}

}  // namespace moe
