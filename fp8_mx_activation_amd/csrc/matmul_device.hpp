// Pieces shared by the experts' product kernels: the arguments, the rows an
// expert holds, copies from memory into LDS, the tile a block works on and the
// fused end of a row (bias, activation, residual, rounding or quantization).
#pragma once

#include "mxfp4_device.hpp"
#include "row_tiles.hpp"

namespace mxq {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

enum MatmulOut { kOutBf16 = 0, kOutG128 = 1, kOutG32 = 2, kOutFp4 = 3 };
enum MatmulAct { kActNone = 0, kActSilu = 1, kActSiluMul = 2 };

struct MatmulArgs {
  const uint8_t* q;  // [num_rows, ld_q] e4m3, or e2m1 pairs
  int64_t ld_q;
  const uint8_t* s;  // [num_rows, ld_s] scale bytes
  int64_t ld_s;
  int64_t num_rows;
  const uint8_t* w;   // [E, N, H] e4m3, or [E, N, H/2] e2m1 pairs
  const uint8_t* ws;  // [E, ceil(N/128), nbk] scale bytes, or [E, N, nbk]
  int32_t E, N, H, nbk;
  const int32_t* offsets;  // [E + 1]
  const int32_t* counts;   // [E]
  const float* bias;       // [E, N] or null
  int32_t act;
  int32_t NO;           // output columns: N, or N / 2 when gated
  const uint16_t* res;  // [num_rows, ld_r] bf16 or null
  int64_t ld_r;
  uint8_t* out;  // bf16, e4m3 or e2m1 pairs [num_rows, ld_out]
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
  } else if constexpr (OUT == kOutFp4) {
    int e;
    const uint32_t w = quant8_e2m1<kNoClip>(v, e);
    if (!live) return;
    *reinterpret_cast<uint32_t*>(a.out + r * a.ld_out + c / 2) = w;
    if (c % 32 == 0) a.so[r * a.ld_so + c / 32] = (uint8_t)(e + 127);
  } else {
    constexpr int G = OUT == kOutG128 ? 128 : 32;
    const uint32_t m = group_max<G / 8>(absmax8(v));
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

// ------------------------------------------------------------ copies to LDS

__device__ __forceinline__ v4i buffer_of(const void* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  v4i r;
  r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)p);
  r.y = __builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32) & 0xFFFF);
  r.z = __builtin_amdgcn_readfirstlane((int)bytes);
  r.w = 0x00020000;  // raw 32-bit data, no swizzle
  return r;
}

// 16 bytes per lane from `buf` at voff + soff into LDS at lds + 16 * lane.
// The lane's address registers are the only operands: nothing is returned to
// registers, so there is no result to wait for but the vmcnt before the next
// barrier.  The clobbers keep LDS accesses, and what the compiler may hold in
// m0, on their side of the copy (it warns that m0 is a register it never
// allocates; it does write it for instructions of its own).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy_to_lds(const v4i& buf, uint32_t lds,
                                            uint32_t voff, uint32_t soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(buf), "s"(soff)
      : "m0", "memory");
}
#pragma clang diagnostic pop

// Waits until all but the last VM loads and copies and the last LGKM LDS reads
// that this wavefront has issued are done.
template <int VM, int LGKM>
__device__ __forceinline__ void wait_for() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | 0x70 |
                             (LGKM << 8));
  asm volatile("" ::: "memory");
}

// The same for the whole block.
template <int VM, int LGKM>
__device__ __forceinline__ void landed_barrier() {
  wait_for<VM, LGKM>();
  asm volatile("s_barrier" ::: "memory");
}

// 16-byte chunk c of an LDS row of 128 bytes sits at place c ^ ((row >> 1) & 7):
// 16 neighbouring rows of a fragment read then touch all 64 banks once.  A
// copy fills places in order, so the order is turned on its global side.
__device__ __forceinline__ int place(int c, int row) {
  return c ^ ((row >> 1) & 7);
}

__device__ __forceinline__ v8i join(const v4i& a, const v4i& b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The tile a block works on.  Experts' tiles are numbered expert by expert,
// from device data; every wavefront finds its block's by itself.  Runs of
// consecutive tiles go to one XCD (block b runs on XCD b % 8), and within a
// run eight row tiles share a column of weights, so the 32 CUs of an XCD
// read a window of 8 by 4 tiles through their L2.  TM = kAllRows (every expert
// that holds rows is one tile of them all): a tile's columns one after the
// other, on all XCDs, where tiles differ in what they take and weights are read
// once either way.
struct TileOf {
  int e, m0, n;
  ExpertRows rows;  // of expert e
};

constexpr int kGroupM = 8;

template <int TM>
__device__ __forceinline__ bool find_tile(const MatmulArgs& a, int tiles_n,
                                          TileOf& t) {
  constexpr bool kSpread = TM == kAllRows;
  const int lane = threadIdx.x & 63;
  const int per = (a.E + 63) / 64;  // experts per lane, consecutive
  ExpertRows er{0, 0};
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < a.E) {
      er = expert_rows(a, e);
      mine += row_tiles<TM>(er.count);
    }
    // regions that do not overlap hold 2^24 tiles at most; more, of offsets
    // that no layout makes, must not overflow the sums
    mine = min(mine, 1 << 24);
  }
  int upto = mine;  // row tiles of lanes up to this one
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  const int tiles_m = __builtin_amdgcn_readlane(upto, 63);
  const int64_t total = (int64_t)tiles_m * tiles_n;
  const int64_t run = (total + 7) / 8;
  const int64_t at =
      kSpread ? (int64_t)blockIdx.x
              : (int64_t)(blockIdx.x & 7) * run + (blockIdx.x >> 3);
  if ((!kSpread && (int64_t)(blockIdx.x >> 3) >= run) || at >= total)
    return false;
  constexpr int kGroup = kSpread ? 1 : kGroupM;
  const int64_t group = at / ((int64_t)kGroup * tiles_n);
  const int gm = min(kGroup, tiles_m - (int)group * kGroup);
  const int in = (int)(at - group * kGroup * tiles_n);
  t.n = in / gm;
  const int m = (int)group * kGroup + in % gm;
  const int owner = __ffsll((unsigned long long)__ballot(upto > m)) - 1;
  int first = __builtin_amdgcn_readlane(upto - mine, owner);
  int e = owner * per;
  if (per == 1) {
    // the owner has read its one expert's rows
    const uint64_t f = (uint64_t)er.first;
    er.first = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane(
                             (int)(uint32_t)(f >> 32), owner)
                         << 32 |
                         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)f,
                                                             owner));
    er.count = __builtin_amdgcn_readlane(er.count, owner);
  } else {
    for (int i = 0; i < per; ++i) {
      e = owner * per + i;
      er = expert_rows(a, e);
      const int c = row_tiles<TM>(er.count);
      if (m < first + c) break;
      first += c;
    }
  }
  t.e = __builtin_amdgcn_readfirstlane(e);
  t.m0 = __builtin_amdgcn_readfirstlane((m - first) * TM);
  t.rows = er;
  return true;
}

// ------------------------------------------------------------ end of a tile

constexpr int kStageLd = 260;  // floats per staged token (256 weight rows + pad)

// End of a tile of 64 XF token rows (`rows` of them live, from row0 on) by 256
// weight rows of expert e, from output n0 on.  64 PX token rows (PX fragments
// of each wavefront row) at a time go through LDS as they are, so that a thread
// ends up with eight neighbouring channels of a row: gate and factor meet, a row
// is written in whole lines, and a quantization group lies within a wavefront.
// The arguments come by value: through a reference the compiler asks again for
// what they hold at every store (8-bit weights, 65536 rows, down: 1278 us, not
// 1262).
template <int XF, int OUT, bool GATED, int PX = 2>
__device__ __forceinline__ void finish_tile(const MatmulArgs a, int e,
                                            int64_t row0, int rows, int n0,
                                            const v16f (&acc)[4][XF],
                                            uint8_t* lds) {
  float* stage = reinterpret_cast<float*>(lds);
  constexpr int kOutLanes = GATED ? 16 : 32;  // threads per row
  constexpr int kPerRound = 256 / kOutLanes;  // rows per round of the block
  constexpr int kRounds = 64 * PX / kPerRound;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r32 = lane & 31, g = lane >> 5;
  const int orow = (int)threadIdx.x / kOutLanes;
  const int oc = (int)threadIdx.x % kOutLanes * 8;
  const int col = n0 + oc;
  float b[8], bu[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = bu[j] = 0.0f;
  if (a.bias != nullptr) {
    const float* br = a.bias + (int64_t)e * a.N;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      b[j] = br[min(col + j, a.NO - 1)];
      if (GATED) bu[j] = br[a.NO + min(col + j, a.NO - 1)];
    }
  }
  // where the gate of output oc stands in a staged row; its factor is 64 on
  const int gate_at = GATED ? (oc >> 6) * 128 + (oc & 63) : oc;
  // token (of the tile) of row i of pass p
  auto token = [&](int p, int i) {
    return i / (32 * PX) * 32 * XF + p * 32 * PX + i % (32 * PX);
  };
  constexpr int kPasses = XF / PX;
  // A pass's residual is asked for a pass ahead, the first one's before its
  // staging: the loads are in flight together and behind other work.
  u32x4 res[2][kRounds];
  auto ask = [&](int p) {
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      res[p & 1][i] = load_residual(
          a, row0 + min(token(p, i * kPerRound + orow), rows - 1), col);
  };
  const bool has_res = OUT == kOutBf16 && a.res != nullptr;
  if (has_res) {
    ask(0);
  } else {
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      res[0][i] = res[1][i] = u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    __syncthreads();
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
        for (int x = 0; x < PX; ++x) {
          const v16f& v = acc[f][PX * pass + x];
          *reinterpret_cast<v4f*>(stage +
                                  (wm * 32 * PX + x * 32 + r32) * kStageLd +
                                  wn * 128 + f * 32 + 8 * q4 + 4 * g) =
              v4f{v[4 * q4], v[4 * q4 + 1], v[4 * q4 + 2], v[4 * q4 + 3]};
        }
    __syncthreads();
    if (has_res && pass + 1 < kPasses) ask(pass + 1);
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int at = i * kPerRound + orow;
      const int tok = token(pass, at);
      const float* src = stage + at * kStageLd + gate_at;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = src[j] + b[j];
      if constexpr (GATED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = silu(v[j]) * (src[64 + j] + bu[j]);
      } else if (a.act == kActSilu) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = silu(v[j]);
      }
      store_channels<OUT>(a, row0 + min(tok, rows - 1), col,
                          tok < rows && col < a.NO, v, res[pass & 1][i]);
    }
  }
}

}  // namespace mxq
