// moe_expert_matmul_mxfp4, moe_expert_matmul_mxfp4_quant: the experts' products
// with weights in microscaled 4-bit floats.
//
//   a[r, n] = sum_k q[r, k] 2^(s[r, k/32] - 127) w[e, n, k]
//             2^(ws[e, n, k/32] - 127) + bias[e, n]     for the live rows r of e
//   out     = act(a) (+ residual), as bf16 or quantized again with group scales
//
// Rows are e2m1 or e4m3, both with a scale per 32 channels.  The scales go
// into gfx950's block-scaled MFMA, whose operands may have one type each: with
// both in 4 bits it takes half the cycles of 8 bits, with one in 8 bits the
// whole.  A lane holds 32 channels of a row either way: 16 bytes of e2m1 at
// channel 32 g, or two times 16 bytes of e4m3 at 16 g and as far behind the
// first half of the step's channels.
#include <type_traits>

#include "matmul_device.hpp"
#include "mxq_host.hpp"

namespace {

using namespace mxq;

constexpr int kFmtFp8 = 0, kFmtFp4 = 4;  // the MFMA's operand types

// An e2m1 operand: 16 bytes, the upper half of the registers is not read.
__device__ __forceinline__ v8i half(const v4i& a) {
  return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
}

// ------------------------------------------------------------ few rows
//
// With few rows an expert's weights are read once for all of them (16 at a
// time), and the kernel is bound by that stream.  A block of four wavefronts
// owns 64 NG weight rows of one expert and all rows of that expert; its
// wavefronts take 64 weight rows each and, where NG < 4, split the K axis in
// 4 / NG interleaved parts (neighbouring 128-byte lines are in flight at
// once), joined in LDS at the end.
//
// Each wavefront keeps a ring of three steps of 256 channels of its own in
// LDS, filled by copies that bring whole lines of weights and need no
// registers.  The weight rows are the MFMA's A operand, the token rows its B
// operand: a lane ends up with four neighbouring output channels of one token.
// Three steps; two of 8-bit rows whose scales, all of which are in LDS from the
// start, leave no room for a third (above 20320 channels).
template <bool X8, int RING>
struct SmallStep {
  static constexpr int kRow = X8 ? 256 : 128;  // bytes of a token row
  static constexpr int kX = 64 * 128;          // where the token rows begin,
  static constexpr int kS = kX + 16 * kRow;    // and the weights' scales
  static constexpr int kBytes = kS + 64 * 8;
  static constexpr int kCopies = 8 + (X8 ? 4 : 2) + 2;
  static constexpr int kRings = 4 * RING * kBytes;
};

// Scale bytes of a token in LDS: whole words, an odd number of them.
inline int small_scale_ld(int groups) { return (groups + 7) / 8 * 8 + 4; }

// 4 bytes per lane into LDS at lds + 4 * lane, as copy_to_lds.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy4_to_lds(const v4i& buf, uint32_t lds,
                                             uint32_t voff, uint32_t soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(buf), "s"(soff)
      : "m0", "memory");
}
#pragma clang diagnostic pop

template <bool X8, int RING, int NG, int OUT>
__global__ __launch_bounds__(256, 1) void matmul4_small_kernel(
    MatmulArgs a, int32_t blocks_n, int32_t ld_xs) {
  using St = SmallStep<X8, RING>;
  constexpr int KS = 4 / NG;
  constexpr int NB = 64 * NG;
  constexpr int LDT = NB + 4;  // floats per staged token
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int e = blockIdx.x / blocks_n;
  const ExpertRows er = expert_rows(a, e);
  if (er.count == 0) return;
  const bool gated = a.act == kActSiluMul;
  const int nbo = gated ? NB / 2 : NB;
  const int n0 = (int)(blockIdx.x % blocks_n) * nbo;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ng = wave / KS, ks = wave % KS;
  const int r16 = lane & 15, g = lane >> 4;
  const int H = a.H;
  const int ld_w = H / 2;              // bytes of a weight row
  const int ld_x = X8 ? H : H / 2;     // and of a token row
  const int groups = H / 32;
  const int nsteps = (H + 255) / 256;
  const int mine = (nsteps - ks + KS - 1) / KS;  // steps of this wavefront
  uint8_t* ring = lds + wave * RING * St::kBytes;
  uint8_t* xscale = lds + St::kRings;
  const uint32_t ring0 = (uint32_t)(uintptr_t)(
      __attribute__((address_space(3))) uint8_t*)ring;

  // weight row (within the expert's matrix) of local row lr of the block
  auto weight_row = [&](int lr) {
    if (!gated) return min(n0 + lr, a.N - 1);
    return lr < nbo ? min(n0 + lr, a.NO - 1)
                    : a.NO + min(n0 + lr - nbo, a.NO - 1);
  };
  // copy i brings rows 8 i + (l >> 3); odd copies' chunks differ by 4
  const int chunk0 = place(lane & 7, lane >> 3);
  uint32_t woff[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    woff[i] = (uint32_t)((weight_row(ng * 64 + 8 * i + (lane >> 3)) - n0) *
                         ld_w);
  const v4i wbuf = buffer_of(a.w + ((int64_t)e * a.N + n0) * ld_w,
                             (uint32_t)((a.N - n0) * ld_w));
  // scales: lane l brings those of row l, four blocks at a time
  const uint32_t soff =
      (uint32_t)((weight_row(ng * 64 + lane) - n0) * a.nbk);
  const v4i sbuf = buffer_of(a.ws + ((int64_t)e * a.N + n0) * a.nbk,
                             (uint32_t)((a.N - n0) * a.nbk));

  for (int base = 0; base < er.count; base += 16) {
    const int rows = min(er.count - base, 16);
    const int64_t row0 = er.first + base;
    const v4i xbuf = buffer_of(a.q + row0 * a.ld_q,
                               (uint32_t)((rows - 1) * a.ld_q + ld_x));
    uint32_t xoff[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      xoff[i] = (uint32_t)(min(8 * i + (lane >> 3), rows - 1) * (int)a.ld_q);
    // In a last step that ends inside the 256 channels, chunks past H repeat
    // the step's first: in bounds, and cleared when they are read.
    auto copy_step = [&](int i) {
      const int step = ks + i * KS;
      const int k0 = step * 128;  // bytes of a weight row
      const uint32_t at = ring0 + (uint32_t)(i % RING) * St::kBytes;
      const int c1 = chunk0 ^ 4;
      const uint32_t o0 = k0 + 16 * chunk0 < ld_w ? 16 * chunk0 : 0;
      const uint32_t o1 = k0 + 16 * c1 < ld_w ? 16 * c1 : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        copy_to_lds(wbuf, at + j * 1024, woff[j] + (j & 1 ? o1 : o0), k0);
      if constexpr (X8) {
        // two halves of 128 channels, each as the rows of 4 bits
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = (j & 1 ? c1 : chunk0) + 8 * (j >> 1);
          copy_to_lds(xbuf, at + St::kX + j * 1024,
                      xoff[j & 1] + (2 * k0 + 16 * c < ld_x ? 16 * c : 0),
                      2 * k0);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          copy_to_lds(xbuf, at + St::kX + j * 1024,
                      xoff[j] + (j & 1 ? o1 : o0), k0);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        copy4_to_lds(sbuf, at + St::kS + j * 256,
                     soff + (step * 8 + 4 * j < groups ? 4 * j : 0), step * 8);
    };
    for (int i = threadIdx.x; i < 16 * groups; i += 256) {
      const int r = i / groups;
      xscale[r * ld_xs + i % groups] =
          a.s[(row0 + min(r, rows - 1)) * a.ld_s + i % groups];
    }
#pragma unroll
    for (int i = 0; i < RING; ++i)
      if (i < mine) copy_step(i);
    landed_barrier<63, 0>();  // the scale bytes are down

    v4f acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = v4f{0, 0, 0, 0};

    for (int i = 0; i < mine; ++i) {
      // this step's copies have landed; later ones may be on their way
      if (i + RING <= mine)
        wait_for<(RING - 1) * St::kCopies, 15>();
      else
        wait_for<0, 15>();
      const int step = ks + i * KS;
      const uint8_t* at = ring + i % RING * St::kBytes;
      v4i w[4][2], x[2], x8[2];
      uint32_t sw[4][2], sx[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 4 * h + g;
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          w[f][h] = *reinterpret_cast<const v4i*>(
              at + (f * 16 + r16) * 128 + place(c, r16) * 16);
          sw[f][h] = *reinterpret_cast<const uint32_t*>(
              at + St::kS + h * 256 + (f * 16 + r16) * 4);
        }
        if constexpr (X8) {
          const uint8_t* xr = at + St::kX + h * 2048 + r16 * 128;
          x[h] = *reinterpret_cast<const v4i*>(xr + place(g, r16) * 16);
          x8[h] = *reinterpret_cast<const v4i*>(xr + place(4 + g, r16) * 16);
        } else {
          x[h] = *reinterpret_cast<const v4i*>(at + St::kX + r16 * 128 +
                                               place(c, r16) * 16);
        }
        sx[h] = *reinterpret_cast<const uint32_t*>(xscale + r16 * ld_xs +
                                                   step * 8 + 4 * h);
      }
      wait_for<63, 0>();  // read: the ring's place may be filled again
      if (i + RING < mine) copy_step(i + RING);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sx[h] >>= 8 * g;
#pragma unroll
        for (int f = 0; f < 4; ++f) sw[f][h] >>= 8 * g;
      }
      if (step * 256 + 256 > H) {
        // blocks past H: zeros, whose scales have to be finite ones
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (X8 && step * 256 + 128 * h + 16 * g >= H) x[h] = v4i{0, 0, 0, 0};
          if (X8 && step * 256 + 128 * h + 64 + 16 * g >= H)
            x8[h] = v4i{0, 0, 0, 0};
          if (step * 256 + 128 * h + 32 * g < H) continue;
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            w[f][h] = v4i{0, 0, 0, 0};
            sw[f][h] = 127;
          }
          if (!X8) x[h] = v4i{0, 0, 0, 0};
          sx[h] = 127;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < 4; ++f)
          acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              half(w[f][h]), X8 ? join(x[h], x8[h]) : half(x[h]), acc[f],
              kFmtFp4, X8 ? kFmtFp8 : kFmtFp4, 0, (int)sw[f][h], 0,
              (int)sx[h]);
    }

    // join the K parts: part[ks][token][channel], over the rings
    __syncthreads();
    float* part = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int f = 0; f < 4; ++f)
      *reinterpret_cast<v4f*>(part + (ks * 16 + r16) * LDT + ng * 64 +
                              f * 16 + 4 * g) = acc[f];
    __syncthreads();
    const int lanes = nbo / 8;  // lanes per token
    for (int i = threadIdx.x; i < 16 * lanes; i += 256) {
      const int tok = i / lanes;
      const int c = i % lanes * 8;
      float v[8];
      auto sum = [&](int col, float (&o)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = 0.0f;
#pragma unroll
        for (int p = 0; p < KS; ++p) {
          const float* src = part + (p * 16 + tok) * LDT + col;
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] += src[j];
        }
      };
      const int col = n0 + c;
      const bool in = col < a.NO;
      sum(c, v);
      if (a.bias != nullptr)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] += a.bias[(int64_t)e * a.N + min(col + j, a.NO - 1)];
      if (gated) {
        float u[8];
        sum(nbo + c, u);
        if (a.bias != nullptr)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            u[j] += a.bias[(int64_t)e * a.N + a.NO + min(col + j, a.NO - 1)];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = silu(v[j]) * u[j];
      } else if (a.act == kActSilu) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = silu(v[j]);
      }
      const bool live = in && tok < rows;
      const int64_t row = row0 + min(tok, rows - 1);
      u32x4 res{0, 0, 0, 0};
      if constexpr (OUT == kOutBf16) res = load_residual(a, row, col);
      store_channels<OUT>(a, row, col, live, v, res);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ entry points

constexpr int kLds = 160 * 1024;  // of a CU

template <bool X8, int RING, int NG, int OUT>
mxq_status launch_small(const MatmulArgs& a, hipStream_t s) {
  using St = SmallStep<X8, RING>;
  const int nbo = a.act == kActSiluMul ? 32 * NG : 64 * NG;
  const int64_t bn = ceil_div(a.NO, nbo);
  if (bn * a.E > max_blocks(256)) return MXQ_ERR_UNSUPPORTED;
  const int ld_xs = small_scale_ld(a.H / 32);
  const int lds = St::kRings + 16 * ld_xs;
  if constexpr (RING == 3) {
    if (lds > kLds) return launch_small<X8, 2, NG, OUT>(a, s);
  }
  static_assert(St::kRings >= 4 * 16 * (64 + 4) * 4 &&
                    St::kRings >= 16 * (256 + 4) * 4,
                "the joined K parts fit the rings");
  auto* k = &matmul4_small_kernel<X8, RING, NG, OUT>;
  if (hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                          hipFuncAttributeMaxDynamicSharedMemorySize,
                          lds) != hipSuccess) {
    (void)hipGetLastError();
    return MXQ_ERR_HIP;
  }
  k<<<(unsigned)(bn * a.E), 256, lds, s>>>(a, (int32_t)bn, ld_xs);
  return launch_status();
}

template <bool X8, int OUT>
mxq_status launch(const MatmulArgs& a, int64_t expected, hipStream_t s) {
  (void)expected;
  if (ceil_div(a.N, 256) * a.E >= 256) return launch_small<X8, 3, 4, OUT>(a, s);
  return launch_small<X8, 3, 1, OUT>(a, s);
}

template <int OUT>
mxq_status checked(const void* q, int64_t ld_q, const uint8_t* scales,
                   int64_t ld_s, int64_t num_rows, mxq_scale_fmt fmt,
                   const void* w, const uint8_t* w_scales, int64_t ld_ws,
                   int32_t E, int32_t N, int32_t H, const int32_t* offsets,
                   const int32_t* counts, const float* bias, mxq_act act,
                   const void* residual, int64_t ld_r, int64_t expected_m,
                   void* out, int64_t ld_out, uint8_t* so, int64_t ld_so,
                   void* stream) {
  if (fmt != MXQ_SCALE_MXFP4 && fmt != MXQ_SCALE_E8M0_G32)
    return MXQ_ERR_UNSUPPORTED;
  const bool x8 = fmt == MXQ_SCALE_E8M0_G32;
  if (expected_m > INT32_MAX) expected_m = INT32_MAX;
  if (act != MXQ_ACT_NONE && act != MXQ_ACT_SILU && act != MXQ_ACT_SILU_MUL)
    return MXQ_ERR_UNSUPPORTED;
  if (E < 1 || E > MXQ_MAX_LOCAL_EXPERTS || N < 1 || H < 1 || H % 32 != 0 ||
      num_rows < 0 || num_rows > INT32_MAX || expected_m < 0)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (act == MXQ_ACT_SILU_MUL && N % 2 != 0) return MXQ_ERR_INVALID_ARGUMENT;
  const int32_t NO = act == MXQ_ACT_SILU_MUL ? N / 2 : N;
  if (NO % (OUT == kOutBf16 ? 4 : 32) != 0) return MXQ_ERR_INVALID_ARGUMENT;
  // row counts are rounded up to whole tiles in 32 bits
  if (H > MXQ_MAX_HIDDEN || (int64_t)N * H > INT32_MAX ||
      num_rows > MXQ_MAX_MATMUL_ROWS)
    return MXQ_ERR_UNSUPPORTED;
  if (num_rows == 0) return MXQ_OK;
  if (q == nullptr || scales == nullptr || w == nullptr ||
      w_scales == nullptr || offsets == nullptr || counts == nullptr ||
      out == nullptr)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || ld_q % 16 != 0 || ld_q < (x8 ? H : H / 2) ||
      ld_s < H / 32 || !aligned16(w))
    return MXQ_ERR_INVALID_ARGUMENT;
  // the weights' scales are read four at a time
  if ((reinterpret_cast<uintptr_t>(w_scales) & 3u) != 0 || ld_ws % 4 != 0 ||
      ld_ws < H / 32)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (ld_q > MXQ_MAX_MATMUL_LD || ld_s > MXQ_MAX_MATMUL_LD ||
      ld_ws * N > INT32_MAX)
    return MXQ_ERR_UNSUPPORTED;
  if constexpr (OUT == kOutBf16) {
    if (ld_out < NO || !aligned8(out) || ld_out % 4 != 0)
      return MXQ_ERR_INVALID_ARGUMENT;
    if (residual != nullptr &&
        (!aligned8(residual) || ld_r < NO || ld_r % 4 != 0))
      return MXQ_ERR_INVALID_ARGUMENT;
  } else {
    if (!aligned16(out) || ld_out % 16 != 0 ||
        ld_out < (OUT == kOutFp4 ? NO / 2 : NO) || so == nullptr ||
        ld_so < NO / 32)
      return MXQ_ERR_INVALID_ARGUMENT;
  }
  MatmulArgs a{};
  a.q = static_cast<const uint8_t*>(q);
  a.ld_q = ld_q;
  a.s = scales;
  a.ld_s = ld_s;
  a.num_rows = num_rows;
  a.w = static_cast<const uint8_t*>(w);
  a.ws = w_scales;
  a.E = E;
  a.N = N;
  a.H = H;
  a.nbk = (int32_t)ld_ws;
  a.offsets = offsets;
  a.counts = counts;
  a.bias = bias;
  a.act = act == MXQ_ACT_SILU_MUL ? kActSiluMul
          : act == MXQ_ACT_SILU   ? kActSilu
                                  : kActNone;
  a.NO = NO;
  a.res = static_cast<const uint16_t*>(residual);
  a.ld_r = ld_r;
  a.out = static_cast<uint8_t*>(out);
  a.ld_out = ld_out;
  a.so = so;
  a.ld_so = ld_so;
  a.vec = aligned16(out) && ld_out % 8 == 0 &&
          (residual == nullptr || (aligned16(residual) && ld_r % 8 == 0));
  hipStream_t s = as_stream(stream);
  return x8 ? launch<true, OUT>(a, expected_m, s)
            : launch<false, OUT>(a, expected_m, s);
}

}  // namespace

extern "C" mxq_status moe_expert_matmul_mxfp4(
    const void* q, int64_t ld_q, const uint8_t* scales, int64_t ld_s,
    int64_t num_rows, mxq_scale_fmt fmt, const void* w_fp4,
    const uint8_t* w_scales, int64_t ld_ws, int32_t E, int32_t N, int32_t H,
    const int32_t* expert_offsets, const int32_t* counts, const float* bias,
    mxq_act act, const void* residual_bf16, int64_t ld_r, int64_t expected_m,
    void* out_bf16, int64_t ld_out, void* stream) {
  return checked<kOutBf16>(q, ld_q, scales, ld_s, num_rows, fmt, w_fp4,
                           w_scales, ld_ws, E, N, H, expert_offsets, counts,
                           bias, act, residual_bf16, ld_r, expected_m,
                           out_bf16, ld_out, nullptr, 0, stream);
}

extern "C" mxq_status moe_expert_matmul_mxfp4_quant(
    const void* q, int64_t ld_q, const uint8_t* scales, int64_t ld_s,
    int64_t num_rows, mxq_scale_fmt fmt, const void* w_fp4,
    const uint8_t* w_scales, int64_t ld_ws, int32_t E, int32_t N, int32_t H,
    const int32_t* expert_offsets, const int32_t* counts, const float* bias,
    mxq_act act, int64_t expected_m, mxq_scale_fmt out_fmt, void* q_out,
    int64_t ld_out, uint8_t* scales_out, int64_t ld_so, void* stream) {
  switch (out_fmt) {
    case MXQ_SCALE_MXFP4:
      return checked<kOutFp4>(q, ld_q, scales, ld_s, num_rows, fmt, w_fp4,
                              w_scales, ld_ws, E, N, H, expert_offsets, counts,
                              bias, act, nullptr, 0, expected_m, q_out, ld_out,
                              scales_out, ld_so, stream);
    case MXQ_SCALE_E8M0_G32:
      return checked<kOutG32>(q, ld_q, scales, ld_s, num_rows, fmt, w_fp4,
                              w_scales, ld_ws, E, N, H, expert_offsets, counts,
                              bias, act, nullptr, 0, expected_m, q_out, ld_out,
                              scales_out, ld_so, stream);
    default:
      return MXQ_ERR_UNSUPPORTED;
  }
}
