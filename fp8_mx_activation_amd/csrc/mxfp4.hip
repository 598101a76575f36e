// mxfp4_quant_rows, moe_scatter_quant_mxfp4, mxfp4_to_e4m3,
// upscale_mxfp4_to_bf16: rows to microscaled 4-bit floats and back.
//
//   e    the smallest exponent with amax <= 6 * 2^e over 32 channels, or
//        floor(log2 amax) - 2
//   q    = e2m1(x * 2^-e), nearest even; scale byte e + 127
//
// Every kernel is bound by what it reads and writes.  To quantize or to widen to
// e4m3, a lane owns 16 neighbouring channels (32 bytes of bf16, 8 of codes); a
// group's two lanes are neighbours.  16384 rows of 7168 bf16 channels (297 MB)
// are quantized in 52.8 us (5.6 TB/s; 8 channels a lane with ordinary loads and
// stores 77); 40832 rows of 4 bits become e4m3 in 70 us (6.3 TB/s).  Back to bf16
// a lane owns 8: 49.1 us for the 16384 rows (6.0; 60 with ordinary stores).
#include <algorithm>

#include "mxfp4_device.hpp"
#include "mxq_host.hpp"

namespace {

using namespace mxq;

constexpr int kThreads = 256;
constexpr int kUnits = kThreads * 2;  // of 16 channels, of a block

// Sixteen channels as they lie in memory: 32 bytes of bf16, 64 of fp32.
template <bool F32>
struct Raw16 {
  u32x4 v[F32 ? 4 : 2];
};

template <bool F32>
__device__ __forceinline__ Raw16<F32> load_raw(const void* row, int c) {
  Raw16<F32> r;
  const char* p = static_cast<const char*>(row) + (int64_t)c * (F32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 2); ++i) r.v[i] = load16_nt(p + 16 * i);
  return r;
}

// The codes of a lane's 16 channels, whose group it shares with its neighbour,
// and the group's exponent.  Both lanes must be active.
template <bool F32, int RULE>
__device__ __forceinline__ uint2 quant16_e2m1(const Raw16<F32>& r, int& e) {
  float a[8], b[8];
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 x = r.v[i], y = r.v[2 + i];
      a[4 * i] = __uint_as_float(x.x);
      a[4 * i + 1] = __uint_as_float(x.y);
      a[4 * i + 2] = __uint_as_float(x.z);
      a[4 * i + 3] = __uint_as_float(x.w);
      b[4 * i] = __uint_as_float(y.x);
      b[4 * i + 1] = __uint_as_float(y.y);
      b[4 * i + 2] = __uint_as_float(y.z);
      b[4 * i + 3] = __uint_as_float(y.w);
    }
  } else {
    auto eight = [](const u32x4& w, float (&v)[8]) {
      v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x);
      v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
      v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z);
      v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
    };
    eight(r.v[0], a);
    eight(r.v[1], b);
  }
  e = e2m1_exponent<RULE>(group_max<2>(max(absmax8(a), absmax8(b))));
  const float f = pow2_neg(e);
  return uint2{pack8_e2m1(a, f), pack8_e2m1(b, f)};
}

// Calls load and then use (slot, row, unit of the row) for the units (upr of
// them in a row) of the block's rows that this lane owns, DEPTH at a time.  A
// group's units lie in neighbouring lanes: all are there or none.
template <int DEPTH, typename Load, typename Use>
__device__ __forceinline__ void over_units(int64_t rows, int32_t upr,
                                           int32_t rpb, Load load, Use use) {
  const int64_t row0 = (int64_t)blockIdx.x * rpb;
  const int n = (int)min((int64_t)rpb, rows - row0) * upr;
  for (int base = threadIdx.x; base < n; base += DEPTH * kThreads) {
    int64_t r[DEPTH];
    int u[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
      const int at = base + i * kThreads;
      r[i] = row0 + at / upr;
      u[i] = at % upr;
      if (at < n) load(i, r[i], u[i]);
    }
#pragma unroll
    for (int i = 0; i < DEPTH; ++i)
      if (base + i * kThreads < n) use(i, r[i], u[i]);
  }
}

__device__ __forceinline__ void store8_nt(void* p, const uint2& v) {
  uint32_t* d = reinterpret_cast<uint32_t*>(p);
  __builtin_nontemporal_store(v.x, d);
  __builtin_nontemporal_store(v.y, d + 1);
}

template <bool F32, int RULE>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(
    const void* __restrict__ x, int64_t ld_x, int64_t rows, int32_t upr,
    int32_t rpb, uint8_t* __restrict__ q, int64_t ld_q,
    uint8_t* __restrict__ s, int64_t ld_s) {
  Raw16<F32> v[2];
  over_units<2>(
      rows, upr, rpb,
      [&](int i, int64_t r, int u) {
        v[i] = load_raw<F32>(
            static_cast<const char*>(x) + r * ld_x * (F32 ? 4 : 2), u * 16);
      },
      [&](int i, int64_t r, int u) {
        int e;
        store8_nt(q + r * ld_q + u * 8, quant16_e2m1<F32, RULE>(v[i], e));
        if (u % 2 == 0) s[r * ld_s + u / 2] = (uint8_t)(e + 127);
      });
}

__global__ __launch_bounds__(kThreads) void to_e4m3_kernel(
    const uint8_t* __restrict__ q, int64_t ld_q, int64_t rows, int32_t upr,
    int32_t rpb, uint8_t* __restrict__ out, int64_t ld_out) {
  uint2 w[2];
  over_units<2>(
      rows, upr, rpb,
      [&](int i, int64_t r, int u) {
        w[i] = *reinterpret_cast<const uint2*>(q + r * ld_q + u * 8);
      },
      [&](int i, int64_t r, int u) {
        const uint2 a = e2m1_to_e4m3(w[i].x), b = e2m1_to_e4m3(w[i].y);
        store16_nt(out + r * ld_out + u * 16, u32x4{a.x, a.y, b.x, b.y});
      });
}

// Eight codes times f = 2^(b - 127) as bf16: exact but where they overflow.
__device__ __forceinline__ u32x4 e2m1_to_bf16(uint32_t w, float f) {
  auto two = [&](auto pair) {
    const uint32_t h = __builtin_bit_cast(uint32_t, pair);
    const float lo = bf16_lo(h) * f, hi = bf16_hi(h) * f;
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) |
           ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16);
  };
  return u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3))};
}

__global__ __launch_bounds__(kThreads) void upscale_kernel(
    const uint8_t* __restrict__ q, int64_t ld_q, const uint8_t* __restrict__ s,
    int64_t ld_s, int64_t rows, int32_t upr, int32_t rpb,
    uint16_t* __restrict__ out, int64_t ld_out) {
  // units of eight channels: a wavefront's stores are whole lines (streaming
  // stores of 16 channels a lane in two halves took twice the time)
  uint32_t w[4], b[4];
  over_units<4>(
      rows, 2 * upr, rpb,
      [&](int i, int64_t r, int u) {
        w[i] = *reinterpret_cast<const uint32_t*>(q + r * ld_q + u * 4);
        b[i] = s[r * ld_s + u / 4];
      },
      [&](int i, int64_t r, int u) {
        // subnormal for 0, NaN for 255
        const float f = __uint_as_float(b[i] == 0     ? 0x400000u
                                        : b[i] == 255 ? 0x7FC00000u
                                                      : b[i] << 23);
        store16_nt(out + r * ld_out + u * 8, e2m1_to_bf16(w[i], f));
      });
}

// One block per token: the row is quantized once into LDS and written from
// there to its destinations, all of the block's threads sharing the 16-byte
// chunks of all of them.  4096 rows of 7168 channels to 32768 destinations
// (184 MB) take 36 us (5.1 TB/s), 128 rows to 1024 4.3 us.
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
  for (int c = threadIdx.x * 16; c < H; c += blockDim.x * 16) {
    int e;
    *reinterpret_cast<uint2*>(row + c / 2) =
        quant16_e2m1<false, RULE>(load_raw<false>(xr, c), e);
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

// Rows per block: about kUnits units of 16 channels.
struct RowsGrid {
  int32_t upr, rpb;
  int64_t blocks;
};

RowsGrid rows_grid(int64_t rows, int32_t H) {
  RowsGrid g;
  g.upr = H / 16;
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
  const int threads = std::max(row_block_threads(H, 16), std::min(K, 8) * 64);
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
