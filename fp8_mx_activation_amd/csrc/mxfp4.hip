// mxfp4_quant_rows, moe_scatter_quant_mxfp4, mxfp4_to_e4m3,
// upscale_mxfp4_to_bf16: rows to microscaled 4-bit floats and back.
//
//   e    the smallest exponent with amax <= 6 * 2^e over 32 channels, or
//        floor(log2 amax) - 2
//   q    = e2m1(x * 2^-e), nearest even; scale byte e + 127
//
// Every kernel is bound by what it reads and writes.  A lane owns eight
// neighbouring channels: 16 bytes of bf16 or of e4m3's two lanes' worth, 4
// bytes of codes; a group's four lanes are a DPP quad.
#include <algorithm>

#include "mxfp4_device.hpp"
#include "mxq_host.hpp"

namespace {

using namespace mxq;

constexpr int kThreads = 256;
constexpr int kDepth = 4;  // units of eight channels a lane has in flight
constexpr int kUnits = kThreads * kDepth;

// Eight channels as fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int c, float (&v)[8]) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(
        static_cast<const float*>(row) + c);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const u32x4 a = load16(static_cast<const uint16_t*>(row) + c);
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x);
    v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z);
    v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
  }
}

// Calls f(slot, row, unit of the row) for the units of the block's rows that
// this lane owns, kDepth at a time.  A group's units lie in one quad: all four
// are there or none.
template <typename Load, typename Use>
__device__ __forceinline__ void over_units(int64_t rows, int32_t upr,
                                           int32_t rpb, Load load, Use use) {
  const int64_t row0 = (int64_t)blockIdx.x * rpb;
  const int n = (int)min((int64_t)rpb, rows - row0) * upr;
  for (int base = threadIdx.x; base < n; base += kUnits) {
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      const int u = base + i * kThreads;
      if (u < n) load(i, row0 + u / upr, u % upr);
    }
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      const int u = base + i * kThreads;
      if (u < n) use(i, row0 + u / upr, u % upr);
    }
  }
}

template <bool F32, int RULE>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(
    const void* __restrict__ x, int64_t ld_x, int64_t rows, int32_t upr,
    int32_t rpb, uint8_t* __restrict__ q, int64_t ld_q,
    uint8_t* __restrict__ s, int64_t ld_s) {
  float v[kDepth][8];
  over_units(
      rows, upr, rpb,
      [&](int i, int64_t r, int u) {
        load8<F32>(static_cast<const char*>(x) + r * ld_x * (F32 ? 4 : 2),
                   u * 8, v[i]);
      },
      [&](int i, int64_t r, int u) {
        int e;
        const uint32_t w = quant8_e2m1<RULE>(v[i], e);
        *reinterpret_cast<uint32_t*>(q + r * ld_q + u * 4) = w;
        if (u % 4 == 0) s[r * ld_s + u / 4] = (uint8_t)(e + 127);
      });
}

__global__ __launch_bounds__(kThreads) void to_e4m3_kernel(
    const uint8_t* __restrict__ q, int64_t ld_q, int64_t rows, int32_t upr,
    int32_t rpb, uint8_t* __restrict__ out, int64_t ld_out) {
  uint32_t w[kDepth];
  over_units(
      rows, upr, rpb,
      [&](int i, int64_t r, int u) {
        w[i] = *reinterpret_cast<const uint32_t*>(q + r * ld_q + u * 4);
      },
      [&](int i, int64_t r, int u) {
        *reinterpret_cast<uint2*>(out + r * ld_out + u * 8) =
            e2m1_to_e4m3(w[i]);
      });
}

__global__ __launch_bounds__(kThreads) void upscale_kernel(
    const uint8_t* __restrict__ q, int64_t ld_q, const uint8_t* __restrict__ s,
    int64_t ld_s, int64_t rows, int32_t upr, int32_t rpb,
    uint16_t* __restrict__ out, int64_t ld_out) {
  uint32_t w[kDepth], b[kDepth];
  over_units(
      rows, upr, rpb,
      [&](int i, int64_t r, int u) {
        w[i] = *reinterpret_cast<const uint32_t*>(q + r * ld_q + u * 4);
        b[i] = s[r * ld_s + u / 4];
      },
      [&](int i, int64_t r, int u) {
        // 2^(b - 127): subnormal for 0, NaN for 255; a payload's two bits
        // times it are bf16 numbers but where they overflow
        const float f = __uint_as_float(b[i] == 0     ? 0x400000u
                                        : b[i] == 255 ? 0x7FC00000u
                                                      : b[i] << 23);
        auto two = [&](auto pair) {
          const uint32_t h = __builtin_bit_cast(uint32_t, pair);
          const float lo = bf16_lo(h) * f, hi = bf16_hi(h) * f;
          return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) |
                 ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16);
        };
        store16(out + r * ld_out + u * 8,
                u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(
                          w[i], 1.0f, 0)),
                      two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(
                          w[i], 1.0f, 1)),
                      two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(
                          w[i], 1.0f, 2)),
                      two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(
                          w[i], 1.0f, 3))});
      });
}

// One block per token: the row is quantized once into LDS and written from
// there to its destinations, all of the block's threads sharing the 16-byte
// chunks of all of them.
template <int RULE>
__global__ __launch_bounds__(1024) void scatter_kernel(
    const uint16_t* __restrict__ x, int64_t ld_x, int32_t H,
    const int32_t* __restrict__ src2dst, int32_t K, uint8_t* __restrict__ q,
    int64_t ld_q, uint8_t* __restrict__ s, int64_t ld_s, int64_t num_rows) {
  extern __shared__ __align__(16) uint8_t row[];  // [H/2] codes, [H/32] scales
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63;
  const int32_t d_lane = src2dst[t * K + min(lane, K - 1)];
  const bool valid = lane < K && d_lane >= 0 && (int64_t)d_lane < num_rows;
  if (__ballot(valid) == 0) return;  // the same in every wavefront
  const uint16_t* xr = x + t * ld_x;
  for (int c = threadIdx.x * 8; c < H; c += blockDim.x * 8) {
    float v[8];
    load8<false>(xr, c, v);
    int e;
    *reinterpret_cast<uint32_t*>(row + c / 2) = quant8_e2m1<RULE>(v, e);
    if ((c & 31) == 0) row[H / 2 + c / 32] = (uint8_t)(e + 127);
  }
  __syncthreads();
  const int nw = blockDim.x >> 6;
  for (int j = threadIdx.x >> 6; j < K; j += nw) {
    const int64_t d = __builtin_amdgcn_readlane(d_lane, j);
    if (d < 0 || d >= num_rows) continue;
    for (int c = lane * 16; c < H / 2; c += 64 * 16)
      store16_nt(q + d * ld_q + c, *reinterpret_cast<const u32x4*>(row + c));
    for (int g = lane; g < H / 32; g += 64)
      s[d * ld_s + g] = row[H / 2 + g];
  }
}

// Rows per block: about kUnits units of eight channels.
struct RowsGrid {
  int32_t upr, rpb;
  int64_t blocks;
};

RowsGrid rows_grid(int64_t rows, int32_t H) {
  RowsGrid g;
  g.upr = H / 8;
  g.rpb = std::max(1, kUnits / g.upr);
  g.blocks = ceil_div(rows, g.rpb);
  return g;
}

bool row_bytes_ok(const void* p, int64_t ld_bytes) {
  return aligned16(p) && ld_bytes % 16 == 0;
}

bool rule_ok(mxq_scale_rule r) {
  return r == MXQ_RULE_NO_CLIP || r == MXQ_RULE_OCP_FLOOR;
}

}  // namespace

extern "C" mxq_status mxfp4_quant_rows(const void* x, mxq_out_dtype dtype,
                                       int64_t ld_x, int64_t rows, int32_t H,
                                       mxq_scale_rule rule, void* q_fp4,
                                       int64_t ld_q, uint8_t* scales,
                                       int64_t ld_s, void* stream) {
  if ((dtype != MXQ_OUT_BF16 && dtype != MXQ_OUT_F32) || !rule_ok(rule))
    return MXQ_ERR_UNSUPPORTED;
  if (rows < 0 || H < 32 || H % 32 != 0) return MXQ_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MXQ_OK;
  const int64_t esz = dtype == MXQ_OUT_BF16 ? 2 : 4;
  if (x == nullptr || q_fp4 == nullptr || scales == nullptr || ld_x < H ||
      ld_q < H / 2 || ld_s < H / 32 || !row_bytes_ok(x, ld_x * esz) ||
      !row_bytes_ok(q_fp4, ld_q))
    return MXQ_ERR_INVALID_ARGUMENT;
  const RowsGrid g = rows_grid(rows, H);
  if (g.blocks > max_blocks(kThreads)) return MXQ_ERR_UNSUPPORTED;
  auto* k = dtype == MXQ_OUT_BF16
                ? (rule == MXQ_RULE_NO_CLIP
                       ? &quant_rows_kernel<false, kNoClip>
                       : &quant_rows_kernel<false, kOcpFloor>)
                : (rule == MXQ_RULE_NO_CLIP
                       ? &quant_rows_kernel<true, kNoClip>
                       : &quant_rows_kernel<true, kOcpFloor>);
  k<<<(unsigned)g.blocks, kThreads, 0, as_stream(stream)>>>(
      x, ld_x, rows, g.upr, g.rpb, static_cast<uint8_t*>(q_fp4), ld_q, scales,
      ld_s);
  return launch_status();
}

extern "C" mxq_status moe_scatter_quant_mxfp4(
    const void* x_bf16, int64_t ld_x, int64_t T, int32_t H,
    const int32_t* src2dst, int32_t K, mxq_scale_rule rule, void* q_fp4,
    int64_t ld_q, uint8_t* scales, int64_t ld_s, int64_t num_rows,
    void* stream) {
  if (!rule_ok(rule)) return MXQ_ERR_UNSUPPORTED;
  if (T < 0 || H < 32 || H % 32 != 0 || K < 0 || K > MXQ_MAX_TOPK ||
      num_rows < 0 || num_rows > INT32_MAX)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (H > MXQ_MAX_HIDDEN) return MXQ_ERR_UNSUPPORTED;
  if (T == 0 || K == 0 || num_rows == 0) return MXQ_OK;
  if (x_bf16 == nullptr || src2dst == nullptr || q_fp4 == nullptr ||
      scales == nullptr || ld_x < H || ld_q < H / 2 || ld_s < H / 32 ||
      !row_bytes_ok(x_bf16, ld_x * 2) || !row_bytes_ok(q_fp4, ld_q))
    return MXQ_ERR_INVALID_ARGUMENT;
  const int threads = std::max(row_block_threads(H, 8), std::min(K, 8) * 64);
  if (T > max_blocks(threads)) return MXQ_ERR_UNSUPPORTED;
  auto* k = rule == MXQ_RULE_NO_CLIP ? &scatter_kernel<kNoClip>
                                     : &scatter_kernel<kOcpFloor>;
  k<<<(unsigned)T, threads, H / 2 + H / 32, as_stream(stream)>>>(
      static_cast<const uint16_t*>(x_bf16), ld_x, H, src2dst, K,
      static_cast<uint8_t*>(q_fp4), ld_q, scales, ld_s, num_rows);
  return launch_status();
}

extern "C" mxq_status mxfp4_to_e4m3(const void* q_fp4, int64_t ld_q,
                                    int64_t rows, int32_t H, void* out_fp8,
                                    int64_t ld_out, void* stream) {
  if (rows < 0 || H < 32 || H % 32 != 0) return MXQ_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MXQ_OK;
  if (q_fp4 == nullptr || out_fp8 == nullptr || ld_q < H / 2 || ld_out < H ||
      !row_bytes_ok(q_fp4, ld_q) || !row_bytes_ok(out_fp8, ld_out))
    return MXQ_ERR_INVALID_ARGUMENT;
  const RowsGrid g = rows_grid(rows, H);
  if (g.blocks > max_blocks(kThreads)) return MXQ_ERR_UNSUPPORTED;
  to_e4m3_kernel<<<(unsigned)g.blocks, kThreads, 0, as_stream(stream)>>>(
      static_cast<const uint8_t*>(q_fp4), ld_q, rows, g.upr, g.rpb,
      static_cast<uint8_t*>(out_fp8), ld_out);
  return launch_status();
}

extern "C" mxq_status upscale_mxfp4_to_bf16(
    const void* q_fp4, int64_t ld_q, const uint8_t* scales, int64_t ld_s,
    int64_t num_rows, int32_t H, void* out_bf16, int64_t ld_out,
    void* stream) {
  if (num_rows < 0 || H < 32 || H % 32 != 0) return MXQ_ERR_INVALID_ARGUMENT;
  if (num_rows == 0) return MXQ_OK;
  if (q_fp4 == nullptr || scales == nullptr || out_bf16 == nullptr ||
      ld_q < H / 2 || ld_s < H / 32 || ld_out < H ||
      !row_bytes_ok(q_fp4, ld_q) || !row_bytes_ok(out_bf16, ld_out * 2))
    return MXQ_ERR_INVALID_ARGUMENT;
  const RowsGrid g = rows_grid(num_rows, H);
  if (g.blocks > max_blocks(kThreads)) return MXQ_ERR_UNSUPPORTED;
  upscale_kernel<<<(unsigned)g.blocks, kThreads, 0, as_stream(stream)>>>(
      static_cast<const uint8_t*>(q_fp4), ld_q, scales, ld_s, num_rows, g.upr,
      g.rpb, static_cast<uint16_t*>(out_bf16), ld_out);
  return launch_status();
}
