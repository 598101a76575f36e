// Access to the router's rows, shared by the router and its balance loss: a
// lane's consecutive experts of a row of logits or of their gradients.
#pragma once

#include <algorithm>

#include "mxq_device.hpp"
#include "mxq_host.hpp"

namespace mxq {

constexpr float kFltMax = 3.402823466e38f;

// The lane's PER values from e0 on, -inf past E.
template <int PER, bool BF16>
__device__ __forceinline__ void load_row(const void* row, int E, int e0,
                                         bool vec, float (&raw)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) raw[i] = -__builtin_inff();
  if constexpr (BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(row);
    if (PER % 4 == 0 && vec && e0 + PER <= E) {
#pragma unroll
      for (int i = 0; i + 3 < PER; i += 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(p + e0 + i);
        raw[i] = bf16_lo(w.x);
        raw[i + 1] = bf16_hi(w.x);
        raw[i + 2] = bf16_lo(w.y);
        raw[i + 3] = bf16_hi(w.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e0 + i < E) raw[i] = __uint_as_float((uint32_t)p[e0 + i] << 16);
    }
  } else {
    const float* p = static_cast<const float*>(row);
    if (PER % 4 == 0 && vec && e0 + PER <= E) {
#pragma unroll
      for (int i = 0; i + 3 < PER; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(p + e0 + i);
        raw[i] = w.x;
        raw[i + 1] = w.y;
        raw[i + 2] = w.z;
        raw[i + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e0 + i < E) raw[i] = p[e0 + i];
    }
  }
}

// Logits: -inf (never chosen, score 0) for NaN too; +inf counts as the largest
// finite value.
template <int PER, bool BF16>
__device__ __forceinline__ void load_logits(const void* row, int E, int e0,
                                            bool vec, float (&l)[PER]) {
  load_row<PER, BF16>(row, E, e0, vec, l);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float v = l[i];
    l[i] = v != v ? -__builtin_inff() : (v > kFltMax ? kFltMax : v);
  }
}

template <int PER, bool BF16>
__device__ __forceinline__ void store_row(void* row, int E, int e0, bool vec,
                                          const float (&g)[PER]) {
  if constexpr (BF16) {
    uint16_t* p = static_cast<uint16_t*>(row);
    uint16_t h[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
      h[i] = __builtin_bit_cast(uint16_t, (__bf16)g[i]);
    if (PER % 4 == 0 && vec && e0 + PER <= E) {
#pragma unroll
      for (int i = 0; i + 3 < PER; i += 4)
        *reinterpret_cast<uint2*>(p + e0 + i) =
            uint2{(uint32_t)h[i] | ((uint32_t)h[i + 1] << 16),
                  (uint32_t)h[i + 2] | ((uint32_t)h[i + 3] << 16)};
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e0 + i < E) p[e0 + i] = h[i];
    }
  } else {
    float* p = static_cast<float*>(row);
    if (PER % 4 == 0 && vec && e0 + PER <= E) {
#pragma unroll
      for (int i = 0; i + 3 < PER; i += 4)
        *reinterpret_cast<float4*>(p + e0 + i) =
            float4{g[i], g[i + 1], g[i + 2], g[i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e0 + i < E) p[e0 + i] = g[i];
    }
  }
}

// Calls f(first token, tokens, blocks) for every launch that T tokens take.
template <typename F>
void by_launches(int64_t T, int waves, F&& f) {
  const int64_t most = max_blocks(waves * 64) * waves;
  for (int64_t t = 0; t < T; t += most) {
    const int64_t n = std::min(most, T - t);
    f(t, n, (unsigned)ceil_div(n, waves));
  }
}

inline bool row_vec(const void* p, int64_t ld, int64_t esz) {
  return aligned16(p) && (ld * esz) % 16 == 0;
}

}  // namespace mxq
