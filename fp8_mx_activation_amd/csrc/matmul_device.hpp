// Pieces shared by the experts' product kernels: the arguments, the rows an
// expert holds, the block-scaled MFMA and the fused end of a row (bias,
// activation, residual, rounding or quantization).
#pragma once

#include "mxq_device.hpp"

namespace mxq {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

enum MatmulOut { kOutBf16 = 0, kOutG128 = 1, kOutG32 = 2 };
enum MatmulAct { kActNone = 0, kActSilu = 1, kActSiluMul = 2 };

struct MatmulArgs {
  const uint8_t* q;  // [num_rows, ld_q] e4m3
  int64_t ld_q;
  const uint8_t* s;  // [num_rows, ld_s] scale bytes
  int64_t ld_s;
  int64_t num_rows;
  const uint8_t* w;   // [E, N, H] e4m3
  const uint8_t* ws;  // [E, ceil(N/128), nbk] scale bytes
  int32_t E, N, H, nbk;
  const int32_t* offsets;  // [E + 1]
  const int32_t* counts;   // [E]
  const float* bias;       // [E, N] or null
  int32_t act;
  int32_t NO;           // output columns: N, or N / 2 when gated
  const uint16_t* res;  // [num_rows, ld_r] bf16 or null
  int64_t ld_r;
  uint8_t* out;  // bf16 or e4m3 [num_rows, ld_out]
  int64_t ld_out;
  uint8_t* so;  // scale bytes [num_rows, ld_so] when quantized
  int64_t ld_so;
  int32_t vec;  // bf16 out and residual rows start on 16 bytes, not just 8
};

// First row and number of live rows of expert e, inside the buffers whatever
// the device data say.
struct ExpertRows {
  int64_t first;
  int32_t count;
};

__device__ __forceinline__ ExpertRows expert_rows(const MatmulArgs& a, int e) {
  const int64_t first = a.offsets[e];
  int64_t n = (int64_t)a.offsets[e + 1] - first;
  n = min(n, (int64_t)a.counts[e]);
  n = min(n, a.num_rows - first);
  if (first < 0 || n < 0) n = 0;
  return ExpertRows{first, (int32_t)n};
}

// x / (1 + exp(-x)) with the hardware's power of two and reciprocal.  The
// product -x log2(e) is rounded once and the constant is 0.22 * 2^-24 of itself
// off, so exp(-x) is off by a factor of at most 1 + (1.22 |x| + 2) 2^-24.  A
// reciprocal below 2^-126 is 0, and so is the quotient from -87.4 down (where
// it is above -2^-119).
__device__ __forceinline__ float silu(float x) {
  constexpr float kLog2e = 1.44269504088896341f;
  return x * __builtin_amdgcn_rcpf(1.0f +
                                   __builtin_amdgcn_exp2f(-x * kLog2e));
}

// Power-of-two exponent of a group from the fp32 magnitude bits of its
// largest value: the smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8),
// clamped below at -127; the largest finite fp32 gives 120.
__device__ __forceinline__ int pow2_exponent_f32(uint32_t m) {
  const int e = (int)(m >> 23) - 135 + (((m & 0x7FFFFFu) > 0x600000u) ? 1 : 0);
  return e < -127 ? -127 : e;
}

// The residual's eight channels from column c of row r (four where the row
// ends after them: NO % 4 == 0), or zeros.  Reads inside the row only.
__device__ __forceinline__ u32x4 load_residual(const MatmulArgs& a, int64_t r,
                                               int c) {
  u32x4 d{0, 0, 0, 0};
  if (a.res == nullptr || c >= a.NO) return d;
  const uint16_t* p = a.res + r * a.ld_r + c;
  const bool whole = c + 8 <= a.NO;
  if (a.vec && whole) return load16(p);
  const uint2 lo = *reinterpret_cast<const uint2*>(p);
  d.x = lo.x;
  d.y = lo.y;
  if (whole) {
    const uint2 hi = *reinterpret_cast<const uint2*>(p + 4);
    d.z = hi.x;
    d.w = hi.y;
  }
  return d;
}

// Eight finished channels from column c of row r, with their residual.  The
// lanes of a group (4 for 32 channels, 16 for 128) hold neighbouring columns
// and are all here.  Quantization takes the fp32 values: the only rounding is
// the payload's.
template <int OUT>
__device__ __forceinline__ void store_channels(const MatmulArgs& a, int64_t r,
                                               int c, bool live, float (&v)[8],
                                               const u32x4& res) {
  if constexpr (OUT == kOutBf16) {
    if (!live) return;
    const bool whole = c + 8 <= a.NO;  // else four columns
    v[0] += bf16_lo(res.x);
    v[1] += bf16_hi(res.x);
    v[2] += bf16_lo(res.y);
    v[3] += bf16_hi(res.y);
    v[4] += bf16_lo(res.z);
    v[5] += bf16_hi(res.z);
    v[6] += bf16_lo(res.w);
    v[7] += bf16_hi(res.w);
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i]) |
             ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i + 1])
              << 16);
    uint8_t* o = a.out + (r * a.ld_out + c) * 2;
    if (a.vec && whole) {
      store16(o, u32x4{p[0], p[1], p[2], p[3]});
    } else {
      *reinterpret_cast<uint2*>(o) = uint2{p[0], p[1]};
      if (whole) *reinterpret_cast<uint2*>(o + 8) = uint2{p[2], p[3]};
    }
  } else {
    constexpr int G = OUT == kOutG128 ? 128 : 32;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = group_max<G / 8>(m);
    const int e = pow2_exponent_f32(m);
    const float f = pow2_neg(e);
    if (!live) return;
    uint2 w;
    w.x = pack4_e4m3(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
    w.y = pack4_e4m3(v[4] * f, v[5] * f, v[6] * f, v[7] * f);
    *reinterpret_cast<uint2*>(a.out + r * a.ld_out + c) = w;
    if (c % G == 0) a.so[r * a.ld_so + c / G] = (uint8_t)(e + 127);
  }
}

}  // namespace mxq
