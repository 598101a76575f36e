// e2m1 payloads of microscaled 4-bit floats: 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a
// sign, two to a byte, the lower channel in the lower half.
#pragma once

#include "mxq_device.hpp"

namespace mxq {

// Exponent of a group's scale from the fp32 magnitude bits of its largest
// value: the smallest e with amax <= 6 * 2^e (6 = 1.5 * 2^2), or
// floor(log2 amax) - 2, clamped below at -127; the largest finite fp32 gives
// 126.  e2m1 has no NaN: a group that holds one (whose bits lie above
// infinity's) gets 128, scale byte 255, which makes all of it NaN whatever its
// codes are.
template <int RULE>
__device__ __forceinline__ int e2m1_exponent(uint32_t m) {
  int e = (int)(m >> 23) - 129;
  if constexpr (RULE == kNoClip) e += (m & 0x7FFFFFu) > 0x400000u ? 1 : 0;
  e = e < -127 ? -127 : e;
  return m > 0x7F800000u ? 128 : e;
}

// Eight values over their scale -> eight codes, nearest even, with gfx950's
// v_cvt_scalef32_pk_fp4_f32, which takes what lies above 6 as 6.
__device__ __forceinline__ uint32_t pack8_e2m1(const float (&v)[8], float f) {
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, v[0] * f, v[1] * f,
                                                        1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * f, v[3] * f, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * f, v[5] * f, 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * f, v[7] * f, 1.0f,
                                                  3);
}

// The largest magnitude of eight values, as bits.
__device__ __forceinline__ uint32_t absmax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// Eight channels of a lane, whose group is the four lanes of a quad: their
// codes, and the group's exponent.  All four lanes must be active.
template <int RULE>
__device__ __forceinline__ uint32_t quant8_e2m1(const float (&v)[8], int& e) {
  e = e2m1_exponent<RULE>(group_max<4>(absmax8(v)));
  return pack8_e2m1(v, pow2_neg(e));
}

// Eight codes -> eight e4m3 bytes: magnitudes looked up in a table of eight
// bytes by v_perm, four at a time, even and odd channels apart.
__device__ __forceinline__ uint2 e2m1_to_e4m3(uint32_t w) {
  constexpr uint32_t kLo = 0x3C383000u, kHi = 0x4C484440u;
  const uint32_t h = w >> 4;
  const uint32_t even =
      __builtin_amdgcn_perm(kHi, kLo, w & 0x07070707u) |
      ((w & 0x08080808u) << 4);
  const uint32_t odd = __builtin_amdgcn_perm(kHi, kLo, h & 0x07070707u) |
                       ((h & 0x08080808u) << 4);
  return uint2{__builtin_amdgcn_perm(odd, even, 0x05010400u),
               __builtin_amdgcn_perm(odd, even, 0x07030602u)};
}

}  // namespace mxq
