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

// Up to 16 scale bytes of a row from byte `at` on, 127 behind the last of
// `groups`.
__device__ __forceinline__ u32x4 last_scales(const uint8_t* row, int at,
                                             int groups) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = 0x7F7F7F7Fu;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int c = at + 4 * i + b;
      if (c < groups)
        v[i] = (v[i] & ~(0xFFu << (8 * b))) | ((uint32_t)row[c] << (8 * b));
    }
  }
  return u32x4{v[0], v[1], v[2], v[3]};
}

// The end of few rows: token rows `rows` of them live, from row0 on, whose sums
// over KS parts of K stand in part[ks][16 NT tokens][NB + 4]; gate rows are the
// first half of the NB, their factors the second.
template <int KS, int NB, int NT, int OUT>
__device__ __forceinline__ void finish_few(const MatmulArgs& a, int e,
                                           int64_t row0, int rows, int n0,
                                           const float* part) {
  constexpr int LDT = NB + 4;
  const bool gated = a.act == kActSiluMul;
  const int nbo = gated ? NB / 2 : NB;
  const int lanes = nbo / 8;  // lanes per token
  for (int i = threadIdx.x; i < 16 * NT * lanes; i += 256) {
    if (NT > 1 && i / lanes >= (rows + 15) / 16 * 16) break;
    const int tok = i / lanes;
    const int c = i % lanes * 8;
    float v[8];
    auto sum = [&](int col, float (&o)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = 0.0f;
#pragma unroll
      for (int p = 0; p < KS; ++p) {
        const float* src = part + (p * 16 * NT + tok) * LDT + col;
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
}

// ------------------------------------------------------------ few blocks
//
// With few rows an expert's weights are read once for all of them, and the
// kernels are bound by that stream.  Where few experts and few weight rows make
// few blocks (up to 128 of 128 weight rows), a block of four wavefronts owns 64
// weight rows of one expert and up to 16 of its rows at a time; its wavefronts
// split the K axis in four interleaved parts (neighbouring 128-byte lines are
// in flight at once), joined in LDS at the end.  One to four experts of 4096 x
// 4096 with one row each: 11.1 us against 13.3 without the split.
//
// Each wavefront keeps a ring of steps of 256 channels of its own in LDS,
// filled by copies that bring whole lines of weights and need no registers, and
// no barrier orders them.  The weight rows are the MFMA's A operand, the token
// rows its B operand: a lane ends up with four neighbouring output channels of
// one token.  Three steps; two of 8-bit rows whose scales, all of which are in
// LDS from the start, leave no room for a third (above 20224 channels).
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

template <bool X8, int RING, int OUT>
__global__ __launch_bounds__(256, 1) void matmul4_small_kernel(
    MatmulArgs a, int32_t blocks_n, int32_t ld_xs) {
  using St = SmallStep<X8, RING>;
  constexpr int KS = 4, NB = 64;
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
  const int ks = wave;
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
    woff[i] = (uint32_t)((weight_row(8 * i + (lane >> 3)) - n0) *
                         ld_w);
  const v4i wbuf = buffer_of(a.w + ((int64_t)e * a.N + n0) * ld_w,
                             (uint32_t)((a.N - n0) * ld_w));
  // scales: lane l brings those of row l, four blocks at a time
  const uint32_t soff =
      (uint32_t)((weight_row(lane) - n0) * a.nbk);
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
      *reinterpret_cast<v4f*>(part + (ks * 16 + r16) * LDT + f * 16 +
                              4 * g) = acc[f];
    __syncthreads();
    finish_few<KS, NB, 1, OUT>(a, e, row0, rows, n0, part);
    __syncthreads();
  }
}

// ------------------------------------------------------------ few rows
//
// Where there are blocks enough, a block's four wavefronts take 16 FW weight
// rows each and share up to 16 NT token rows.  A step is 256 channels of all of
// them.  The weights are a wavefront's own affair, as above; the token rows are
// brought by all four, and one barrier a step says that they are there, and
// that those of the step before may be overwritten.  Three steps are held: while
// one is multiplied, two are on their way.
//
// FW = 2: blocks of 128 weight rows that fit a CU twice, so that the start and
// the end of one (a chain of loads, the outputs) lie behind the other's stream.
// FW = 4, NT = 4 (8-bit rows: 3): an expert's rows go through in one pass where
// 16 or 32 at a time would read its weights twice.
//
// One row of each of eight experts, 4096 x 7168 gated (125 MB): 24.9 us, 5.0
// TB/s, a block's start and end the rest; 8-bit rows of 128 tokens, top-2 over 32
// experts: 90 us (5.6 TB/s), and 7168 x 2048 55 us (4.5).
//
// Scales come in chunks of 16 bytes per weight row, two steps' worth, copied
// straight into LDS two steps ahead; what is left of a row behind whole chunks
// is put there at the start, with 127 (a factor of one) for the blocks behind
// the last.  The tokens' scales are all in LDS from the start of a pass.
template <bool X8, int NT, int FW>
struct Stream {
  static constexpr int kRows = 64 * FW;    // weight rows of a block
  static constexpr int kX = kRows * 128;   // bytes of a step's weights
  static constexpr int kStage = kX + NT * 16 * (X8 ? 256 : 128);
  static constexpr int kRing = 3;
  static constexpr int kChunk = kRows * 16;  // scales: two in turn, the last
  static constexpr int kScales = kRing * kStage;
  static constexpr int kXScales = kScales + 3 * kChunk;
  static constexpr int kCopiesX = NT * (X8 ? 4 : 2) / 4;  // of a wavefront
  static_assert(NT * (X8 ? 4 : 2) % 4 == 0, "every wavefront copies as many");
  static_assert(kScales >= NT * 16 * (kRows + 4) * 4,
                "the sums fit the stages");
};

template <bool X8, int NT, int FW, int OUT>
__global__ __launch_bounds__(256, 1) void matmul4_stream_kernel(
    MatmulArgs a, int32_t blocks_n, int32_t ld_xs) {
  using St = Stream<X8, NT, FW>;
  constexpr int R = St::kRing, CX = St::kCopiesX, CW = 2 * FW;
  constexpr int NB = St::kRows;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  // every expert that holds rows is one tile of them all, so the blocks that
  // have work come first and spread evenly
  TileOf tile;
  if (!find_tile<kAllRows>(a, blocks_n, tile)) return;
  const int e = tile.e;
  const ExpertRows er = tile.rows;
  const bool gated = a.act == kActSiluMul;
  const int nbo = gated ? NB / 2 : NB;
  const int n0 = tile.n * nbo;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int H = a.H;
  const int ld_w = H / 2;           // bytes of a weight row
  const int ld_x = X8 ? H : H / 2;  // and of a token row
  const int groups = H / 32;
  const int nsteps = (H + 255) / 256;
  const int full = groups / 16;  // chunks of scales that end within the row
  const uint32_t lds0 = (uint32_t)(uintptr_t)(
      __attribute__((address_space(3))) uint8_t*)lds;
  uint8_t* scale = lds + St::kScales;
  uint8_t* xscale = lds + St::kXScales;

  // weight row (within the expert's matrix) of local row lr of the block
  auto weight_row = [&](int lr) {
    if (!gated) return min(n0 + lr, a.N - 1);
    return lr < nbo ? min(n0 + lr, a.NO - 1)
                    : a.NO + min(n0 + lr - nbo, a.NO - 1);
  };
  // weight copy i brings rows 8 i + (l >> 3); odd copies' chunks differ by 4
  const int chunk0 = place(lane & 7, lane >> 3);
  uint32_t woff[CW];
#pragma unroll
  for (int i = 0; i < CW; ++i)
    woff[i] = (uint32_t)((weight_row(wave * 16 * FW + 8 * i + (lane >> 3)) - n0) *
                         ld_w);
  const v4i wbuf = buffer_of(a.w + ((int64_t)e * a.N + n0) * ld_w,
                             (uint32_t)((a.N - n0) * ld_w));
  const uint32_t soff =
      (uint32_t)((weight_row(min(wave * 64 + lane, NB - 1)) - n0) * a.nbk);
  const v4i sbuf = buffer_of(a.ws + ((int64_t)e * a.N + n0) * a.nbk,
                             (uint32_t)((a.N - n0) * a.nbk));
  // In a last step that ends inside the 256 channels, chunks past H repeat
  // the step's first: in bounds, and cleared when they are read.
  auto copy_w = [&](int i) {
    const int k0 = i * 128;
    const uint32_t at =
        lds0 + (uint32_t)(i % R) * St::kStage + (uint32_t)wave * 2048 * FW;
    const int c1 = chunk0 ^ 4;
    const uint32_t o0 = k0 + 16 * chunk0 < ld_w ? 16 * chunk0 : 0;
    const uint32_t o1 = k0 + 16 * c1 < ld_w ? 16 * c1 : 0;
#pragma unroll
    for (int j = 0; j < CW; ++j)
      copy_to_lds(wbuf, at + j * 1024, woff[j] + (j & 1 ? o1 : o0), k0);
  };
  // 64 weight rows' by a wavefront: of 128 rows, by two
  auto copy_scales = [&](int j) {
    if (wave >= FW) return;
    copy_to_lds(sbuf,
                lds0 + St::kScales + (j & 1) * St::kChunk + wave * 1024, soff,
                j * 16);
  };
  if (groups % 16 != 0 && (int)threadIdx.x < NB) {
    const uint8_t* p =
        a.ws + ((int64_t)e * a.N + weight_row(threadIdx.x)) * a.nbk;
    *reinterpret_cast<u32x4*>(scale + 2 * St::kChunk + threadIdx.x * 16) =
        last_scales(p, full * 16, groups);
  }

  for (int base = 0; base < er.count; base += 16 * NT) {
    const int rows = min(er.count - base, 16 * NT);
    const int64_t row0 = er.first + base;
    const v4i xbuf = buffer_of(a.q + row0 * a.ld_q,
                               (uint32_t)((rows - 1) * a.ld_q + ld_x));
    // token copy c brings 8 rows' 128 bytes; of 8-bit rows the first 2 NT
    // copies are the first halves, the others the second
    uint32_t xoff[CX];
    int xchunk[CX];
#pragma unroll
    for (int i = 0; i < CX; ++i) {
      const int c = wave * CX + i;
      const int r = c % (2 * NT) * 8 + (lane >> 3);
      xoff[i] = (uint32_t)(min(r, rows - 1) * (int)a.ld_q);
      xchunk[i] = place(lane & 7, r) + (c >= 2 * NT ? 8 : 0);
    }
    auto copy_x = [&](int k) {
      const int k0 = k * (X8 ? 256 : 128);
#pragma unroll
      for (int i = 0; i < CX; ++i)
        copy_to_lds(xbuf,
                    lds0 + (uint32_t)(k % R) * St::kStage + St::kX +
                        (uint32_t)(wave * CX + i) * 1024,
                    xoff[i] + (k0 + 16 * xchunk[i] < ld_x ? 16 * xchunk[i]
                                                          : 0),
                    k0);
    };
    {
      const int words = (groups + 3) / 4;
      for (int i = threadIdx.x; i < rows * words; i += 256) {
        const uint8_t* p = a.s + (row0 + i / words) * a.ld_s;
        const int c = i % words * 4;
        uint32_t v = 0x7F7F7F7Fu;
        if (c + 4 <= groups)
          __builtin_memcpy(&v, p + c, 4);
        else
          for (int b = c; b < groups; ++b)
            v = (v & ~(0xFFu << (8 * (b & 3)))) |
                ((uint32_t)p[b] << (8 * (b & 3)));
        *reinterpret_cast<uint32_t*>(xscale + i / words * ld_xs + c) = v;
      }
    }
    if (full > 0) copy_scales(0);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i < nsteps) copy_w(i);
      if (i < nsteps && i < R - 1) copy_x(i);
    }

    v4f acc[FW][NT];
#pragma unroll
    for (int f = 0; f < FW; ++f)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[f][t] = v4f{0, 0, 0, 0};

    for (int i = 0; i < nsteps; ++i) {
      // this step's weights, tokens and scales have landed: what follows them
      // are the next two steps' weights and the next one's tokens
      if (i + 2 < nsteps)
        landed_barrier<2 * CW + CX, 0>();
      else if (i + 1 < nsteps)
        landed_barrier<CW + CX, 0>();
      else
        landed_barrier<0, 0>();
      if (i + R - 1 < nsteps) copy_x(i + R - 1);
      const uint8_t* at = lds + i % R * St::kStage;
      const uint8_t* sc =
          scale + (i / 2 == full ? 2 : i / 2 & 1) * St::kChunk + (i & 1) * 8;
      v4i w[FW][2], x[NT][2], x8[NT][2];
      uint32_t sw[FW][2], sx[NT][2];
#pragma unroll
      for (int f = 0; f < FW; ++f) {
        const int r = wave * 16 * FW + f * 16 + r16;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[f][h] = *reinterpret_cast<const v4i*>(
              at + r * 128 + place(4 * h + g, r16) * 16);
        const uint2 v = *reinterpret_cast<const uint2*>(sc + r * 16);
        sw[f][0] = v.x;
        sw[f][1] = v.y;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* xr = at + St::kX + (t * 16 + r16) * 128;
          if constexpr (X8) {
            xr += h * NT * 2048;
            x[t][h] = *reinterpret_cast<const v4i*>(xr + place(g, r16) * 16);
            x8[t][h] =
                *reinterpret_cast<const v4i*>(xr + place(4 + g, r16) * 16);
          } else {
            x[t][h] = *reinterpret_cast<const v4i*>(
                xr + place(4 * h + g, r16) * 16);
          }
          sx[t][h] = *reinterpret_cast<const uint32_t*>(
              xscale + (t * 16 + r16) * ld_xs + i * 8 + 4 * h);
        }
      wait_for<63, 0>();  // read: the weights' place may be filled again
      if ((i & 1) == 0 && i / 2 + 1 < full) copy_scales(i / 2 + 1);
      if (i + R < nsteps) copy_w(i + R);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int f = 0; f < FW; ++f) sw[f][h] >>= 8 * g;
#pragma unroll
        for (int t = 0; t < NT; ++t) sx[t][h] >>= 8 * g;
      }
      if (i * 256 + 256 > H) {
        // blocks past H: zeros, whose scales have to be finite ones
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = i * 256 + 128 * h;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (k + (X8 ? 16 : 32) * g >= H) x[t][h] = v4i{0, 0, 0, 0};
            if (X8 && k + 64 + 16 * g >= H) x8[t][h] = v4i{0, 0, 0, 0};
            if (k + 32 * g >= H) sx[t][h] = 127;
          }
          if (k + 32 * g < H) continue;
#pragma unroll
          for (int f = 0; f < FW; ++f) {
            w[f][h] = v4i{0, 0, 0, 0};
            sw[f][h] = 127;
          }
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t > 0 && rows <= 16 * t) continue;  // the same for all wavefronts
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int f = 0; f < FW; ++f)
            acc[f][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                half(w[f][h]), X8 ? join(x[t][h], x8[t][h]) : half(x[t][h]),
                acc[f][t], kFmtFp4, X8 ? kFmtFp8 : kFmtFp4, 0, (int)sw[f][h],
                0, (int)sx[t][h]);
      }
    }

    // over the stages: part[token][channel]
    __syncthreads();
    float* part = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (rows <= 16 * t) continue;
#pragma unroll
      for (int f = 0; f < FW; ++f)
        *reinterpret_cast<v4f*>(part + (t * 16 + r16) * (NB + 4) +
                                wave * 16 * FW +
                                f * 16 + 4 * g) = acc[f][t];
    }
    __syncthreads();
    finish_few<1, NB, NT, OUT>(a, e, row0, rows, n0, part);
    __syncthreads();
  }
}

// ------------------------------------------------------------ many rows
//
// The tiles of the products with 8-bit weights: a block of four wavefronts,
// one per SIMD, owns TM = 64 XF token rows of one expert by 256 weight rows;
// each wavefront multiplies 32 XF tokens by 128 weight rows in 32x32x64 steps.
// K goes by in steps of 128 channels, or 256 where rows of 4 bits meet a tile of
// 256, held in LDS twice: while one step is multiplied, the next is on its way
// from memory straight into LDS.  A step of a 256-row tile is 2048 cycles of
// MFMA per SIMD.
//
// Two tiles of 128 rows fit a CU, of 256 one.  The larger one reads 2/3 of the
// LDS bytes and 2/3 of the memory's per product; of two smaller ones, one's
// start and end (its first copies, its output: 6 us of a pair's time for 4-bit
// rows, 14 for 8-bit ones, against 16 and 21 of one large tile's) pass while the
// other multiplies.  Per 256 channels the pair takes 2.6 us (3.0), the large
// tile 1.7 (2.7): short rows want the smaller one, long rows in 4 bits the
// larger.
//
// A step is multiplied in two halves, A with the first half of the wavefront's
// token fragments, B with the second.  B's token fragments are read from LDS
// during A; the next step's weight fragments and first token fragments during
// B, each weight fragment into the registers that its last MFMA has just left.
// The copies of the step after the next are dealt out evenly over both.
//
// Scales.  A step needs four or eight bytes of every token and weight row.  They
// come in chunks of 16 bytes per row, copied straight into LDS as a step's data
// are, for the weights and for tokens whose scales start on 4 bytes; a chunk
// that ends behind the row is put together at the start, with 127 (a factor of
// one) for the blocks that are not there, in a place of its own.  Tokens' scales
// that start elsewhere go through registers, a chunk at a time; the compiler
// then waits for all copies on their way once per chunk.  So does the tokens'
// last chunk where its place would keep the second tile off the CU.
template <bool X8, int XF>
struct Tile {
  static constexpr int kTM = 64 * XF;
  static constexpr int kChannels = X8 || XF == 2 ? 128 : 256;  // of a step
  static constexpr int kWRow = kChannels / 2;          // bytes of a weight row
  static constexpr int kXRow = X8 ? kChannels : kWRow;  // and of a token row
  static constexpr int kX = kTM * kXRow;                // and of all of them
  static constexpr int kStage = kX + 256 * kWRow;
  // 16-byte pieces of a lane's row, of weights one for an MFMA
  static constexpr int kPieces = kWRow / 32, kXPieces = kXRow / 32;
  static constexpr int kSteps = 512 / kChannels;  // per chunk of scales
  static constexpr int kScaleStep = 16 / kSteps;
  static constexpr int kChunk = (kTM + 256) * 16;
  // two chunks that take turns, and the one that ends behind the row; of
  // 128-row tiles of 8-bit rows two fit a CU with the weights' part of it
  static constexpr bool kLate = X8 && XF == 2;  // the tokens' takes a turn
  static constexpr int kLast = kLate ? 256 * 16 : kChunk;
  static constexpr int kLoop = 2 * kStage + 2 * kChunk + kLast;
  static constexpr int kPX = XF == 2 ? 1 : 2;  // fragments the end stages
  static constexpr int kEnd = 64 * kPX * kStageLd * 4;
  static constexpr int kLds = kLoop > kEnd ? kLoop : kEnd;
  static constexpr int kPerCu = XF == 2 ? 2 : 1;
  // copies of a wavefront: of a fragment (both wavefront columns' or rows'), of
  // half A of a step (weight fragments 0-2, token fragment 0) and of half B
  static constexpr int kCopiesW = kWRow / 64, kCopiesX = kXRow / 64;
  static constexpr int kCopiesA = 3 * kCopiesW + kCopiesX;
  static constexpr int kCopiesB = kCopiesW + kCopiesX * (XF - 1);
};

// A uniform value for an operand that has to be in a scalar register.
__device__ __forceinline__ uint32_t in_scalar(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

// 16-byte chunk c of an LDS row of 64 bytes sits at place c ^ ((row >> 2) & 3).
__device__ __forceinline__ int place64(int c, int row) {
  return c ^ ((row >> 2) & 3);
}

template <bool X8, int XF, int OUT, bool GATED>
__global__
__launch_bounds__(256, (Tile<X8, XF>::kPerCu)) void matmul4_tile_kernel(
    MatmulArgs a, int32_t tiles_n, int32_t xs_words) {
  using T = Tile<X8, XF>;
  constexpr int TM = T::kTM;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  TileOf t;
  if (!find_tile<TM>(a, tiles_n, t)) return;
  const ExpertRows er = t.rows;
  const int rows = min(er.count - t.m0, TM);  // live rows of this tile
  const int64_t row0 = er.first + t.m0;
  const int n0 = t.n * (GATED ? 128 : 256);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r32 = lane & 31, g = lane >> 5;
  const int H = a.H;
  const int ld_w = H / 2;           // bytes of a weight row
  const int ld_x = X8 ? H : H / 2;  // and of a token row
  const int groups = H / 32;
  const int nsteps = (H + T::kChannels - 1) / T::kChannels;

  // weight row (within the expert's matrix) of local row lr of the tile
  auto weight_row = [&](int lr) {
    if (!GATED) return min(n0 + lr, a.N - 1);
    const int c = min(n0 + (lr >> 7) * 64 + (lr & 63), a.NO - 1);
    return (lr & 64) ? a.NO + c : c;
  };

  // Copies of 1 KB: of rows of 128 bytes, 8 rows, where lane l fills place
  // l & 7 of row l >> 3, or 16 rows of 64 bytes.  The 64 rows of a fragment
  // are of both wavefront rows or columns; 32 of one follow 32 of the other,
  // or, where a row is 128 bytes, all rows of one the other's.
  const int row128 = wave * 8 + (lane >> 3), row64 = wave * 16 + (lane >> 2);
  const int chunk128 = place(lane & 7, row128);
  const int chunk64 = place64(lane & 3, row64);
  const int xchunk = T::kXRow == 64 ? chunk64 : chunk128;
  const int wchunk = T::kWRow == 64 ? chunk64 : chunk128;
  uint32_t xoff[XF][T::kCopiesX], woff[4][T::kCopiesW];
  // local row of row r (below 64) of token fragment x, of weight fragment f
  auto both_x = [](int x, int r) {
    return ((r >> 5) * XF + x) * 32 + (r & 31);
  };
  auto both_w = [](int f, int r) {
    return (r >> 5) * 128 + f * 32 + (r & 31);
  };
#pragma unroll
  for (int x = 0; x < XF; ++x)
#pragma unroll
    for (int i = 0; i < T::kCopiesX; ++i)
      xoff[x][i] = (uint32_t)(
          min(both_x(x, T::kXRow == 64 ? row64 : i * 32 + row128), rows - 1) *
              (int)a.ld_q +
          16 * xchunk);
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int i = 0; i < T::kCopiesW; ++i)
      woff[f][i] = (uint32_t)(
          (weight_row(both_w(f, T::kWRow == 64 ? row64 : i * 32 + row128)) -
           n0) * ld_w +
          16 * wchunk);
  const v4i xbuf = buffer_of(a.q + row0 * a.ld_q,
                             (uint32_t)((rows - 1) * a.ld_q + ld_x));
  const v4i wbuf = buffer_of(a.w + ((int64_t)t.e * a.N + n0) * ld_w,
                             (uint32_t)((a.N - n0) * ld_w));
  const uint32_t lds0 = (uint32_t)(uintptr_t)(
      __attribute__((address_space(3))) uint8_t*)lds;
  // In a last step that ends inside its channels, chunks past H repeat chunk 0
  // of the step: in bounds, and cleared when they are read.
  auto x_back = [&](int k) {
    return (uint32_t)(k * T::kXRow + 16 * xchunk >= ld_x ? 16 * xchunk : 0);
  };
  auto w_back = [&](int k) {
    return (uint32_t)(k * T::kWRow + 16 * wchunk >= ld_w ? 16 * wchunk : 0);
  };
  auto copy_w = [&](int k, int f, int i, uint32_t back) {
    copy_to_lds(wbuf,
                lds0 + (k & 1) * T::kStage + T::kX +
                    (T::kWRow == 64 ? f * 64 * 64 : (i * 128 + f * 32) * 128) +
                    wave * 1024,
                woff[f][i] - back, in_scalar(k * T::kWRow));
  };
  auto copy_x = [&](int k, int x, int i, uint32_t back) {
    copy_to_lds(xbuf,
                lds0 + (k & 1) * T::kStage +
                    (T::kXRow == 64 ? x * 64 * 64 : (i * XF + x) * 32 * 128) +
                    wave * 1024,
                xoff[x][i] - back, in_scalar(k * T::kXRow));
  };
  auto copy_a = [&](int k, int c, uint32_t wb, uint32_t xb) {
    if (c < 3 * T::kCopiesW)
      copy_w(k, c / T::kCopiesW, c % T::kCopiesW, wb);
    else
      copy_x(k, 0, c - 3 * T::kCopiesW, xb);
  };
  // token fragments of half A, then the weights', then those of half B
  constexpr int kXA = XF / 2;
  auto copy_b = [&](int k, int c, uint32_t wb, uint32_t xb) {
    constexpr int kC = T::kCopiesX, first = kC * (kXA - 1);
    if (c < first)
      copy_x(k, 1 + c / kC, c % kC, xb);
    else if (c < first + T::kCopiesW)
      copy_w(k, 3, c - first, wb);
    else
      copy_x(k, kXA + (c - first - T::kCopiesW) / kC,
             (c - first - T::kCopiesW) % kC, xb);
  };

  // ---- scales
  uint8_t* scale = lds + 2 * T::kStage;
  const uint32_t scale0 = lds0 + 2 * T::kStage;
  const int full = groups / 16;  // chunks that end within the row
  // wavefront w brings the chunk of token rows [64 w, 64 w + 64) (of a tile of
  // 128, the second two the first two's again) and of as many weight rows
  const int srow = (wave % XF) * 64 + lane;
  const uint32_t xsoff = (uint32_t)(min(srow, rows - 1) * (int)a.ld_s);
  const uint32_t wsoff =
      (uint32_t)((weight_row(wave * 64 + lane) - n0) * a.nbk);
  const uint8_t* xs_first = a.s + row0 * a.ld_s;
  const uint8_t* ws_first = a.ws + ((int64_t)t.e * a.N + n0) * a.nbk;
  const v4i xsbuf = buffer_of(xs_first,
                              (uint32_t)((rows - 1) * a.ld_s + groups));
  const v4i wsbuf = buffer_of(ws_first, (uint32_t)((a.N - n0) * a.nbk));
  auto copy_scales = [&](int j) {
    const uint32_t at = scale0 + (j & 1) * T::kChunk;
    if (xs_words)
      copy_to_lds(xsbuf, at + (wave % XF) * 1024, xsoff, in_scalar(j * 16));
    copy_to_lds(wsbuf, at + TM * 16 + wave * 1024, wsoff, in_scalar(j * 16));
  };
  // Through registers, chunk j of a row.  Where the tokens' last chunk takes a
  // turn, words that reach behind its end (of 32 scales or more) are read where
  // they do not, and shifted.
  auto word_at = [&](int j, int i) {
    const int at = j * 16 + 4 * i;
    return T::kLate ? min(at, groups - 4) : at;
  };
  auto fetch = [&](int j, uint32_t (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __builtin_memcpy(&v[i], xs_first + xsoff + word_at(j, i), 4);
  };
  auto put = [&](int j, const uint32_t (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int bits = 8 * (j * 16 + 4 * i - word_at(j, i));
      w[i] = bits == 0   ? v[i]
             : bits < 32 ? (v[i] >> bits) | (0x7F7F7F7Fu << (32 - bits))
                         : 0x7F7F7F7Fu;
    }
    *reinterpret_cast<u32x4*>(scale + (j & 1) * T::kChunk + threadIdx.x * 16) =
        u32x4{w[0], w[1], w[2], w[3]};
  };
  uint32_t xs_next[4];
  constexpr int kWords = T::kScaleStep / 4;  // of a row's scales in a step
  uint32_t sx[XF][kWords], sw[4][kWords], sx1[XF][kWords], sw1[4][kWords];
  auto read_scales = [&](int k) {
    const int j = k / T::kSteps;
    const int in_row = k % T::kSteps * T::kScaleStep;
    const uint8_t* at =
        scale + (!T::kLate && j == full ? 2 : j & 1) * T::kChunk + in_row;
    const uint8_t* at_w = T::kLate && j == full
                              ? scale + 2 * T::kChunk + in_row
                              : at + TM * 16;
#pragma unroll
    for (int x = 0; x < XF; ++x)
      __builtin_memcpy(sx1[x], __builtin_assume_aligned(
          at + (wm * 32 * XF + x * 32 + r32) * 16, T::kScaleStep),
          T::kScaleStep);
#pragma unroll
    for (int f = 0; f < 4; ++f)
      __builtin_memcpy(sw1[f], __builtin_assume_aligned(
          at_w + (wn * 128 + f * 32 + r32) * 16, T::kScaleStep),
          T::kScaleStep);
  };
  // lane group g takes every second block's
  auto use_scales = [&]() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
#pragma unroll
      for (int x = 0; x < XF; ++x) sx[x][i] = sx1[x][i] >> (8 * g);
#pragma unroll
      for (int f = 0; f < 4; ++f) sw[f][i] = sw1[f][i] >> (8 * g);
    }
  };

  v16f acc[4][XF];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int x = 0; x < XF; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][x][i] = 0.0f;

  // fragments of a step, in 16-byte pieces
  constexpr int kP = T::kPieces;
  constexpr int kPX = T::kXPieces;
  v4i fw[4][kP], fx[XF][kPX];
  auto read_w = [&](int k, int f, int p, auto last) {
    const int c = p * 2 + g;
    const uint8_t* base = lds + (k & 1) * T::kStage + T::kX;
    const uint8_t* at =
        T::kWRow == 64
            ? base + (f * 64 + wn * 32 + r32) * 64 + place64(c, r32) * 16
           : base + (wn * 128 + f * 32 + r32) * 128 + place(c, r32) * 16;
    v4i v = *reinterpret_cast<const v4i*>(at);
    if constexpr (decltype(last)::value)
      if (k * T::kWRow + 16 * c >= ld_w) v = v4i{0, 0, 0, 0};
    fw[f][p] = v;
  };
  auto read_x = [&](int k, int x, int p, auto last) {
    const int c = p * 2 + g;
    const uint8_t* base = lds + (k & 1) * T::kStage;
    const uint8_t* at =
        T::kXRow == 64
            ? base + (x * 64 + wm * 32 + r32) * 64 + place64(c, r32) * 16
            : base + (wm * 32 * XF + x * 32 + r32) * 128 + place(c, r32) * 16;
    v4i v = *reinterpret_cast<const v4i*>(at);
    if constexpr (decltype(last)::value)
      if (k * T::kXRow + 16 * c >= ld_x) v = v4i{0, 0, 0, 0};
    fx[x][p] = v;
  };
  constexpr int kMfma = 4 * kP * kXA;  // of a half
  // MFMA i of a half whose first token fragment is x0: weight fragments one
  // after the other, the pieces of each in turn.  Piece p's scales are byte
  // 2 p of the words that use_scales leaves.
  auto multiply = [&](int i, int x0) {
    const int f = i / (kP * kXA), p = i / kXA % kP, x = x0 + i % kXA;
    const v8i w = half(fw[f][p]);
    const v8i v = X8 ? join(fx[x][2 * p % kPX], fx[x][(2 * p + 1) % kPX])
                     : half(fx[x][p % kPX]);
    constexpr int B = X8 ? kFmtFp8 : kFmtFp4;
    if (p & 1)
      acc[f][x] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          w, v, acc[f][x], kFmtFp4, B, 2, (int)sw[f][p / 2], 2,
          (int)sx[x][p / 2]);
    else
      acc[f][x] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          w, v, acc[f][x], kFmtFp4, B, 0, (int)sw[f][p / 2], 0,
          (int)sx[x][p / 2]);
    __builtin_amdgcn_sched_barrier(0);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  auto copy_all = [&](int k) {
    const uint32_t wb = w_back(k), xb = x_back(k);
#pragma unroll
    for (int c = 0; c < T::kCopiesA; ++c) copy_a(k, c, wb, xb);
#pragma unroll
    for (int c = 0; c < T::kCopiesB; ++c) copy_b(k, c, wb, xb);
  };

  if (full > 0) copy_scales(0);
  copy_all(0);
  if (groups % 16 != 0) {
    uint8_t* last = scale + 2 * T::kChunk;
    if ((!T::kLate || full < 2) && (int)threadIdx.x < TM)
      reinterpret_cast<u32x4*>(
          T::kLate ? scale + full * T::kChunk : last)[threadIdx.x] =
          last_scales(xs_first + xsoff, full * 16, groups);
    reinterpret_cast<u32x4*>(last + (T::kLate ? 0 : TM * 16))[threadIdx.x] =
        last_scales(ws_first + wsoff, full * 16, groups);
  }
  if (!xs_words && full > 0 && (int)threadIdx.x < TM) {
    fetch(0, xs_next);
    put(0, xs_next);
  }
  landed_barrier<0, 0>();
  if (nsteps > 1) copy_all(1);
  read_scales(0);
  use_scales();
#pragma unroll
  for (int x = 0; x < kXA; ++x)
#pragma unroll
    for (int p = 0; p < kPX; ++p) read_x(0, x, p, Yes{});
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int p = 0; p < kP; ++p) read_w(0, f, p, Yes{});
  __builtin_amdgcn_sched_barrier(0);

  // One step.  `more`: another one follows; `copy`: and one after that;
  // `last`: this is, and `next_last`: the next one is, the last.  The waits
  // count the copies that may still be on their way: at barrier A all of the
  // next step's, at barrier B those of its second token fragments and of the
  // step after it.  A chunk of scales is asked for before the copies of its
  // first step, so it has landed where they have.  At barrier A the reads of
  // weight fragment 3, always the last ones, may be under way too: its rows are
  // overwritten after barrier B only.
  auto step = [&](int k, auto more_, auto copy_, auto last, auto next_last) {
    constexpr bool more = decltype(more_)::value;
    constexpr bool copy = decltype(copy_)::value;
    const uint32_t wb = w_back(k + 2), xb = x_back(k + 2);
    const int chunk = (k + 2) / T::kSteps;  // of scales
    const bool first = copy && (k + 2) % T::kSteps == 0;
    const bool ask = first && chunk < full;
    const bool ask_last = T::kLate && first && chunk == full && full > 1;
    landed_barrier<more ? T::kCopiesA + T::kCopiesB : 0, kP>();
    if (ask) copy_scales(chunk);
    if constexpr (more) {
      // fetched two steps before the chunk's first, put down in the one
      // before it, ahead of barrier B
      const int next = (k + 1) / T::kSteps;
      const bool down = (k + 1) % T::kSteps == 0;
      const bool down_last = T::kLate && down && next == full && full > 1;
      if (!xs_words || T::kLate) {
        if ((int)threadIdx.x < TM) {
          if (down_last || (down && !xs_words && next < full))
            put(next, xs_next);
          if (ask_last || (ask && !xs_words)) fetch(chunk, xs_next);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kMfma; ++i) {
      if constexpr (copy) {
#pragma unroll
        for (int c = i * T::kCopiesA / kMfma; c < (i + 1) * T::kCopiesA / kMfma;
             ++c)
          copy_a(k + 2, c, wb, xb);
      }
      constexpr int kEach = kMfma / 8 > 1 ? 2 : 1;  // MFMAs per read
      if (i % kEach == 0 && i / kEach < kPX) {
#pragma unroll
        for (int x = kXA; x < XF; ++x) read_x(k, x, i / kEach, last);
      }
      multiply(i, 0);
    }
    if constexpr (more)
      landed_barrier<(copy ? T::kCopiesA : 0) + T::kCopiesX * kXA, 0>();
    if constexpr (more) read_scales(k + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kMfma; ++i) {
      if constexpr (copy) {
#pragma unroll
        for (int c = i * T::kCopiesB / kMfma; c < (i + 1) * T::kCopiesB / kMfma;
             ++c)
          copy_b(k + 2, c, wb, xb);
      }
      if constexpr (more) {
        // a weight fragment's registers take the next step's as soon as its
        // MFMAs are issued
        constexpr int kF = kP * kXA;  // MFMAs of a weight fragment
        if (i < kF) {
#pragma unroll
          for (int p = i * kPX / kF; p < (i + 1) * kPX / kF; ++p)
#pragma unroll
            for (int x = 0; x < kXA; ++x) read_x(k + 1, x, p, next_last);
        } else {
#pragma unroll
          for (int p = i % kF * kP / kF; p < (i % kF + 1) * kP / kF; ++p)
            read_w(k + 1, i / kF - 1, p, next_last);
        }
      }
      multiply(i, kXA);
    }
    if constexpr (more) {
      use_scales();
#pragma unroll
      for (int p = 0; p < kP; ++p) read_w(k + 1, 3, p, next_last);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  int k = 0;
  for (; k + 2 < nsteps; ++k) step(k, Yes{}, Yes{}, No{}, No{});
  if (k + 1 < nsteps) step(k++, Yes{}, No{}, No{}, Yes{});
  step(k, No{}, No{}, Yes{}, No{});

  finish_tile<XF, OUT, GATED, T::kPX>(a, t.e, row0, rows, n0, acc, lds);
}

// ------------------------------------------------------------ entry points

constexpr int kLds = 160 * 1024;  // of a CU

template <bool X8, int RING, int OUT>
mxq_status launch_small(const MatmulArgs& a, hipStream_t s) {
  using St = SmallStep<X8, RING>;
  const int nbo = a.act == kActSiluMul ? 32 : 64;
  const int64_t bn = ceil_div(a.NO, nbo);
  if (bn * a.E > max_blocks(256)) return MXQ_ERR_UNSUPPORTED;
  const int ld_xs = small_scale_ld(a.H / 32);
  const int lds = St::kRings + 16 * ld_xs;
  // whole words of the longest rows' scales, and one
  constexpr int kMost = 16 * (MXQ_MAX_HIDDEN / 32 + 4);
  if constexpr (X8 && RING == 3) {
    if (lds > kLds) return launch_small<X8, 2, OUT>(a, s);
  } else {
    static_assert(St::kRings + kMost <= kLds, "rows of any length fit");
  }
  static_assert(St::kRings >= 4 * 16 * (64 + 4) * 4,
                "the joined K parts fit the rings");
  auto* k = &matmul4_small_kernel<X8, RING, OUT>;
  if (hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                          hipFuncAttributeMaxDynamicSharedMemorySize,
                          lds) != hipSuccess) {
    (void)hipGetLastError();
    return MXQ_ERR_HIP;
  }
  k<<<(unsigned)(bn * a.E), 256, lds, s>>>(a, (int32_t)bn, ld_xs);
  return launch_status();
}

template <bool X8, int NT, int FW, int OUT>
mxq_status launch_stream(const MatmulArgs& a, hipStream_t s) {
  using St = Stream<X8, NT, FW>;
  static_assert(FW == 4 || St::kXScales + 16 * NT * (MXQ_MAX_HIDDEN / 32 + 4) <=
                               kLds,
                "rows of any length fit");
  const int64_t bn = ceil_div(a.NO, a.act == kActSiluMul ? 32 * FW : 64 * FW);
  if (bn * a.E > max_blocks(256)) return MXQ_ERR_UNSUPPORTED;
  const int ld_xs = small_scale_ld(a.H / 32);
  const int lds = St::kXScales + 16 * NT * ld_xs;
  auto* k = &matmul4_stream_kernel<X8, NT, FW, OUT>;
  if (hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                          hipFuncAttributeMaxDynamicSharedMemorySize,
                          lds) != hipSuccess) {
    (void)hipGetLastError();
    return MXQ_ERR_HIP;
  }
  k<<<(unsigned)(bn * a.E), 256, lds, s>>>(a, (int32_t)bn, ld_xs);
  return launch_status();
}

// Whether a pass of 16 NT rows and all their scales fit a CU.
template <bool X8, int NT, int FW>
bool stream_fits(const MatmulArgs& a) {
  return Stream<X8, NT, FW>::kXScales + 16 * NT * small_scale_ld(a.H / 32) <=
         kLds;
}

template <bool X8, int XF, int OUT>
mxq_status launch_tile(const MatmulArgs& a, hipStream_t s) {
  const int64_t tn = ceil_div(a.NO, a.act == kActSiluMul ? 128 : 256);
  // every expert ends in at most one partial row tile
  const int64_t tm = a.num_rows / (64 * XF) + a.E;
  const int64_t blocks = ceil_div(tm * tn, 8) * 8;
  if (blocks > max_blocks(256)) return MXQ_ERR_UNSUPPORTED;
  constexpr int lds = Tile<X8, XF>::kLds;
  static_assert(lds * Tile<X8, XF>::kPerCu <= kLds, "the tiles fit a CU");
  auto* k = a.act == kActSiluMul ? &matmul4_tile_kernel<X8, XF, OUT, true>
                                 : &matmul4_tile_kernel<X8, XF, OUT, false>;
  if (hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                          hipFuncAttributeMaxDynamicSharedMemorySize,
                          lds) != hipSuccess) {
    (void)hipGetLastError();
    return MXQ_ERR_HIP;
  }
  const bool words =
      (reinterpret_cast<uintptr_t>(a.s) & 3u) == 0 && a.ld_s % 4 == 0;
  k<<<(unsigned)blocks, 256, lds, s>>>(a, (int32_t)tn, words);
  return launch_status();
}

// The kernel for `expected` rows in a busy expert.  Measured with top-2
// (below 25 mean rows) and top-8 routings over 32 experts, gate/up
// (4096 x 7168) and down (7168 x 2048) of 4-bit rows (and 8-bit ones), us:
//   mean rows               4         8        12        16        25
//   few rows, FW = 2     76, 41    88, 49   103, 54
//               (8-bit)  83, 43   107, 54   131, 63
//             FW = 4     80, 46    87, 55    98, 56    99, 62   134, 73
//               (8-bit)  82, 47    90, 57   107, 76   112, 80   158, 82
//   128-row tiles                          114, 63   115, 64   120, 67
//               (8-bit)                    121, 76   123, 77   130, 82
// (the weights alone take 94 and 47 us at 5.3 TB/s; with few rows experts are
// left out, and the last-level cache holds a part).  With more rows:
//   mean rows               40        80       160       320       2048
//   128-row tiles       127, 71  156, 84   207, 111  290, 158  1326, 798
//               (8-bit) 135, 86  172, 104  229, 140  349, 214  1677, 1132
//   256-row tiles       128, 99  134, 109  182, 139  254, 199  1070, 865
//               (8-bit) 204, 148 198, 161  291, 207  392, 304  1630, 1260
// With K = 4096 and 2560 gate/up of 4-bit rows takes 325 and 59 us in 128-row
// tiles and 322 and 58 in 256-row ones (320 rows; I = 4096 and 1024); with
// 2048 rows it is 1513 and 244 against 1335 and 255.
// So 4-bit rows of more than 2560 channels take 256-row tiles from 64 rows on,
// 8-bit ones of more than 4096 from 512 on, but not where these would leave half
// of the CUs without one: 64 rows of one expert and of each of four take 46 and
// 48 in the larger tiles, 35 and 38 in the smaller ones.
//
// Few blocks, gate/up (4096 x 7168):
//   experts, mean rows   1, 16  1, 32  1, 64  4, 16  4, 32
//   K split                 12     19     34     26     44
//   (8-bit)                 13     21     37     27     47
//   128-row tiles           34     35     35     36     37
//   (8-bit)                 46     46     46     46     47
// Two experts of 4096 weight rows and 20 rows each: 512 channels 5.7 (6.0) against
// 8.6 (9.5) in tiles, 1024 6.5 (7.0) against 10.6 (12.4), 4096 12.5 (13.6) against
// 21.7 (28.8); a hundred experts of 64 weight rows, 7168 channels, 24 rows: 18 (20)
// against 34 (46).
//
// Between these, too few blocks of 256 weight rows: gate/up of 6, 10 and 15 experts
// takes, with FW = 2, 19, 33 and 39 us for 16 rows of 4 bits each and 21, 34 and 40
// for 20 (one pass), 36, 40 and 45 in tiles.  8-bit rows: 16 in one pass 19, 33 and
// 40, 20 in two passes 33, 59 and 72, in tiles 46, 47 and 50.  A routing's busy
// experts hold more than the mean (top-2 routings, six each): mean 12 rows of 8
// bits 32, 41 and 58 against 45, 47 and 50, mean 16 39, 52 and 74 against 46, 47 and
// 50, hence tiles above 12; of 4 bits mean 12 21, 33 and 47 against 36, 39 and 44,
// mean 16 23, 40 and 56 against 36, 40 and 45, mean 20 24, 43 and 61 against 36, 39
// and 45.
template <bool X8, int OUT>
mxq_status launch(const MatmulArgs& a, int64_t expected, hipStream_t s) {
  constexpr int64_t kCus = 256;
  constexpr int64_t kFew = X8 ? 4 : 12, kMore = X8 ? 16 : 20, kSmall = 12;
  constexpr int kWide = X8 ? 3 : 4;
  const bool few_blocks = ceil_div(a.N, 128) * a.E <= kCus / 2;
  if (few_blocks && expected <= (a.E == 1 ? 32 : 24))
    return launch_small<X8, 3, OUT>(a, s);
  if (!few_blocks && expected <= kMore) {
    if (expected > kFew && ceil_div(a.N, 256) * a.E >= kCus &&
        stream_fits<X8, kWide, 4>(a))
      return launch_stream<X8, kWide, 4, OUT>(a, s);
    if (expected <= kSmall || !X8)
      return launch_stream<X8, X8 ? 1 : 2, 2, OUT>(a, s);
  }
  const int64_t tiles =
      a.E * ceil_div(a.NO, a.act == kActSiluMul ? 128 : 256) *
      ceil_div(expected, 256);
  const bool wide = tiles > kCus / 2 &&
                    (X8 ? a.H > 4096 && expected >= 512
                        : a.H > 2560 && expected >= 64);
  return wide ? launch_tile<X8, 4, OUT>(a, s) : launch_tile<X8, 2, OUT>(a, s);
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
