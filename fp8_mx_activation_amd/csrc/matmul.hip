// moe_expert_matmul, moe_expert_matmul_quant: the experts' products on the
// quantized rows of a layout.
//
//   a[r, n] = sum_k q[r, k] 2^(s[r, k/G] - 127) w[e, n, k] 2^(ws[e, n/128,
//             k/128] - 127) + bias[e, n]        for the live rows r of e
//   out     = act(a) (+ residual), as bf16 or as e4m3 with group scales
//
// The scales go into gfx950's block-scaled MFMA, which multiplies 32 channels
// of both operands by 2^(sx + sw) and adds into fp32.  The matrix unit aligns
// the 32 products that one lane's registers hold to the largest one's exponent
// and drops what lies more than 13 bits below it (measured with two large
// products that cancel and a small one: kept at 2^-13, gone at 2^-14, and
// kept down to fp32's own step when the small one sits in other lanes'
// registers); that is far below the rounding of the inputs, and everything
// else, the joined parts of K, bias, activation and residual among it, is
// fp32 up to the one rounding at the end of the row.
#include <type_traits>

#include "matmul_device.hpp"
#include "mxq_host.hpp"

namespace {

using namespace mxq;

// ------------------------------------------------------------ few rows
//
// Weights are what few rows read: each is needed once per 16 MT rows, so it
// goes from memory straight into the registers of the one wavefront that
// multiplies it, with no LDS and no barrier.  A block owns 64 NG weight rows
// of one expert and all rows of that expert; its wavefronts split the weight
// rows in groups of 64 and the K axis in KS interleaved parts (neighbouring
// 128-byte lines are in flight at once), joined in LDS at the end.  The weight
// rows are the MFMA's A operand, the token rows its B operand, so a lane ends
// up with four neighbouring output channels of one token.
//
// A 16x16x128 step: lane l = 16 g + r holds channels 16 g + [0, 16) and
// 64 + 16 g + [0, 16) of row r; the scale of 32-channel block g of row r
// comes from lane l.
template <int MT>
struct SmallStep {
  v4i w[4][2];
  v4i x[MT][2];
  int sw[4];
  int sx[MT];
};

__device__ __forceinline__ v8i join(const v4i& a, const v4i& b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int G, int MT, int NG, int KS, int OUT>
__global__ __launch_bounds__(64 * NG * KS) void matmul_small_kernel(
    MatmulArgs a, int32_t blocks_n) {
  constexpr int NB = 64 * NG;
  constexpr int LDT = NB + 4;  // floats per staged token
  extern __shared__ __attribute__((aligned(16))) float part[];
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
  const int nsteps = (H + 127) / 128;

  // weight row of the lane in each fragment, clamped to the matrix
  const uint8_t* wrow[4];
  const uint8_t* wsrow[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int lr = ng * 64 + f * 16 + r16;
    int n;
    if (gated)
      n = lr < nbo ? min(n0 + lr, a.NO - 1)
                   : a.NO + min(n0 + lr - nbo, a.NO - 1);
    else
      n = min(n0 + lr, a.N - 1);
    wrow[f] = a.w + ((int64_t)e * a.N + n) * H + 16 * g;
    wsrow[f] = a.ws + ((int64_t)e * ((a.N + 127) / 128) + n / 128) * a.nbk;
  }

  for (int base = 0; base < er.count; base += 16 * MT) {
    const uint8_t* xrow[MT];
    const uint8_t* sxrow[MT];
    v4f acc[4][MT];
#pragma unroll
    for (int x = 0; x < MT; ++x) {
      const int64_t row =
          er.first + min(base + x * 16 + r16, er.count - 1);
      xrow[x] = a.q + row * a.ld_q + 16 * g;
      sxrow[x] = a.s + row * a.ld_s;
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[f][x] = v4f{0, 0, 0, 0};
    }
    auto load = [&](SmallStep<MT>& t, int step) {
      const int k0 = step * 128;
      // the last step may end inside the 128 channels (H % 32 == 0): what
      // lies past H is zero, with a scale of one
      const bool lo = k0 + 16 * g < H, hi = k0 + 64 + 16 * g < H;
      const v4i zero{0, 0, 0, 0};
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        t.w[f][0] =
            lo ? *reinterpret_cast<const v4i*>(wrow[f] + k0) : zero;
        t.w[f][1] =
            hi ? *reinterpret_cast<const v4i*>(wrow[f] + k0 + 64) : zero;
        t.sw[f] = wsrow[f][step];
      }
#pragma unroll
      for (int x = 0; x < MT; ++x) {
        t.x[x][0] =
            lo ? *reinterpret_cast<const v4i*>(xrow[x] + k0) : zero;
        t.x[x][1] =
            hi ? *reinterpret_cast<const v4i*>(xrow[x] + k0 + 64) : zero;
        if constexpr (G == 128)
          t.sx[x] = sxrow[x][step];
        else
          t.sx[x] = k0 + 32 * g < H ? sxrow[x][step * 4 + g] : 127;
      }
    };
    auto multiply = [&](const SmallStep<MT>& t) {
#pragma unroll
      for (int x = 0; x < MT; ++x)
#pragma unroll
        for (int f = 0; f < 4; ++f)
          acc[f][x] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              join(t.w[f][0], t.w[f][1]), join(t.x[x][0], t.x[x][1]),
              acc[f][x], 0, 0, 0, t.sw[f], 0, t.sx[x]);
    };
    if (ks < nsteps) {
      SmallStep<MT> s0, s1;
      load(s0, ks);
      for (int step = ks; step < nsteps; step += 2 * KS) {
        if (step + KS < nsteps) load(s1, step + KS);
        multiply(s0);
        if (step + KS >= nsteps) break;
        if (step + 2 * KS < nsteps) load(s0, step + 2 * KS);
        multiply(s1);
      }
    }

    // join the K parts: part[ks][token][channel]
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
      for (int f = 0; f < 4; ++f)
        *reinterpret_cast<v4f*>(
            part + ((int64_t)(ks * 16 * MT + x * 16 + r16)) * LDT + ng * 64 +
            f * 16 + 4 * g) = acc[f][x];
    __syncthreads();
    const int lanes = nbo / 8;  // lanes per token
    for (int i = threadIdx.x; i < 16 * MT * lanes; i += 64 * NG * KS) {
      const int tok = i / lanes;
      const int c = i % lanes * 8;
      float v[8];
      auto sum = [&](int col, float (&o)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = 0.0f;
#pragma unroll
        for (int p = 0; p < KS; ++p) {
          const float* src = part + (int64_t)(p * 16 * MT + tok) * LDT + col;
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
      const bool live = in && base + tok < er.count;
      const int64_t row = er.first + min(base + tok, er.count - 1);
      store_channels<OUT>(a, row, col, live, v);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ entry points

template <int G, int MT, int NG, int KS, int OUT>
mxq_status launch_small(const MatmulArgs& a, hipStream_t s) {
  const int nbo = a.act == kActSiluMul ? 32 * NG : 64 * NG;
  const int64_t bn = ceil_div(a.NO, nbo);
  if (bn * a.E > INT32_MAX) return MXQ_ERR_UNSUPPORTED;
  const size_t lds = (size_t)KS * 16 * MT * (64 * NG + 4) * sizeof(float);
  auto* k = &matmul_small_kernel<G, MT, NG, KS, OUT>;
  if (lds > 65536 &&
      hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                          hipFuncAttributeMaxDynamicSharedMemorySize,
                          (int)lds) != hipSuccess) {
    (void)hipGetLastError();
    return MXQ_ERR_HIP;
  }
  k<<<(unsigned)(bn * a.E), 64 * NG * KS, lds, s>>>(a, (int32_t)bn);
  return launch_status();
}

template <int G, int OUT>
mxq_status launch(const MatmulArgs& a, int64_t expected, hipStream_t s) {
  if constexpr (OUT == kOutG128) {
    // a group of 128 outputs stays in one block: 128 weight rows, or 256
    if (a.act == kActSiluMul) return launch_small<G, 1, 4, 2, OUT>(a, s);
    return launch_small<G, 1, 2, 4, OUT>(a, s);
  } else {
    if (expected <= 16) return launch_small<G, 1, 1, 4, OUT>(a, s);
    return launch_small<G, 4, 1, 4, OUT>(a, s);
  }
}

inline bool aligned8(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 7u) == 0;
}

template <int OUT>
mxq_status checked(const void* q, int64_t ld_q, const uint8_t* scales,
                   int64_t ld_s, int64_t num_rows, mxq_scale_fmt fmt,
                   const void* w, const uint8_t* w_scales, int32_t E,
                   int32_t N, int32_t H, const int32_t* offsets,
                   const int32_t* counts, const float* bias, mxq_act act,
                   const void* residual, int64_t ld_r, int64_t expected_m,
                   void* out, int64_t ld_out, uint8_t* so, int64_t ld_so,
                   void* stream) {
  const int G = group_of(fmt);
  if (G == 0) return MXQ_ERR_UNSUPPORTED;
  if (act != MXQ_ACT_NONE && act != MXQ_ACT_SILU && act != MXQ_ACT_SILU_MUL)
    return MXQ_ERR_UNSUPPORTED;
  if (E < 1 || E > MXQ_MAX_LOCAL_EXPERTS || N < 1 || H < 1 || H % G != 0 ||
      num_rows < 0 || num_rows > INT32_MAX || expected_m < 0)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (act == MXQ_ACT_SILU_MUL && N % 2 != 0) return MXQ_ERR_INVALID_ARGUMENT;
  const int32_t NO = act == MXQ_ACT_SILU_MUL ? N / 2 : N;
  const int unit = OUT == kOutBf16 ? 4 : OUT == kOutG128 ? 128 : 32;
  if (NO % unit != 0) return MXQ_ERR_INVALID_ARGUMENT;
  if (H > MXQ_MAX_HIDDEN) return MXQ_ERR_UNSUPPORTED;
  if (num_rows == 0) return MXQ_OK;
  if (q == nullptr || scales == nullptr || w == nullptr ||
      w_scales == nullptr || offsets == nullptr || counts == nullptr ||
      out == nullptr)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || ld_q % 16 != 0 || ld_q < H || ld_s < H / G ||
      !aligned16(w) || ld_out < NO)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (ld_q > MXQ_MAX_MATMUL_LD) return MXQ_ERR_UNSUPPORTED;
  if constexpr (OUT == kOutBf16) {
    if (!aligned8(out) || ld_out % 4 != 0) return MXQ_ERR_INVALID_ARGUMENT;
    if (residual != nullptr &&
        (!aligned8(residual) || ld_r < NO || ld_r % 4 != 0))
      return MXQ_ERR_INVALID_ARGUMENT;
  } else {
    if (!aligned16(out) || ld_out % 16 != 0 || so == nullptr || ld_so < NO / unit)
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
  a.nbk = (int32_t)ceil_div(H, 128);
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
  return G == 128 ? launch<128, OUT>(a, expected_m, s)
                  : launch<32, OUT>(a, expected_m, s);
}

}  // namespace

extern "C" mxq_status moe_expert_matmul(
    const void* q_fp8, int64_t ld_q, const uint8_t* scales, int64_t ld_s,
    int64_t num_rows, mxq_scale_fmt fmt, const void* w_fp8,
    const uint8_t* w_scales, int32_t E, int32_t N, int32_t H,
    const int32_t* expert_offsets, const int32_t* counts, const float* bias,
    mxq_act act, const void* residual_bf16, int64_t ld_r, int64_t expected_m,
    void* out_bf16, int64_t ld_out, void* stream) {
  return checked<kOutBf16>(q_fp8, ld_q, scales, ld_s, num_rows, fmt, w_fp8,
                           w_scales, E, N, H, expert_offsets, counts, bias,
                           act, residual_bf16, ld_r, expected_m, out_bf16,
                           ld_out, nullptr, 0, stream);
}

extern "C" mxq_status moe_expert_matmul_quant(
    const void* q_fp8, int64_t ld_q, const uint8_t* scales, int64_t ld_s,
    int64_t num_rows, mxq_scale_fmt fmt, const void* w_fp8,
    const uint8_t* w_scales, int32_t E, int32_t N, int32_t H,
    const int32_t* expert_offsets, const int32_t* counts, const float* bias,
    mxq_act act, int64_t expected_m, mxq_scale_fmt out_fmt, void* q_out,
    int64_t ld_out, uint8_t* scales_out, int64_t ld_so, void* stream) {
  switch (out_fmt) {
    case MXQ_SCALE_UE8M0_G128:
      return checked<kOutG128>(q_fp8, ld_q, scales, ld_s, num_rows, fmt,
                               w_fp8, w_scales, E, N, H, expert_offsets,
                               counts, bias, act, nullptr, 0, expected_m,
                               q_out, ld_out, scales_out, ld_so, stream);
    case MXQ_SCALE_E8M0_G32:
      return checked<kOutG32>(q_fp8, ld_q, scales, ld_s, num_rows, fmt,
                              w_fp8, w_scales, E, N, H, expert_offsets,
                              counts, bias, act, nullptr, 0, expected_m,
                              q_out, ld_out, scales_out, ld_so, stream);
  }
  return MXQ_ERR_UNSUPPORTED;
}
