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
// registers).  Sums of 7168 products of normal values come out 1.5e-5 of their
// norm off (fp32 additions: 1e-6; bf16's rounding: 1.7e-3).  Everything
// else, the joined parts of K, bias, activation and residual among it, is
// fp32 up to the one rounding at the end of the row.
#include <type_traits>

#include "matmul_device.hpp"
#include "mxq_host.hpp"

namespace {

using namespace mxq;

constexpr int kMaxSteps = MXQ_MAX_HIDDEN / 128;

// ------------------------------------------------------------ few rows
//
// With few rows an expert's weights are read once for all of them (16 at a
// time), and the kernel is bound by that stream.  A block of four wavefronts
// owns 64 NG weight rows of one expert and all rows of that expert; its
// wavefronts take 64 weight rows each and, where NG < 4, split the K axis in
// 4 / NG interleaved parts (neighbouring 128-byte lines are in flight at
// once), joined in LDS at the end.
//
// Each wavefront keeps a ring of three steps of 128 channels of its own in
// LDS, filled by copies that bring whole lines and need no registers: 20 KB
// per wavefront are on their way while a step is multiplied, and no barrier
// orders them.  (Loaded into registers, where a lane's 16 bytes make half
// lines, one token through 8 of 32 experts of 4096 x 7168 took 64 us; this way
// 44.5 us, 5.3 TB/s, with the same 235 MB read again, which the last-level
// cache partly holds, and 51-52 us, 4.6 TB/s, where they come from HBM.)  The
// weight rows are the MFMA's A operand, the token rows its B operand: a lane
// ends up with four neighbouring output channels of one token.
//
// A 16x16x128 step: lane l = 16 g + r holds channels 16 g + [0, 16) and
// 64 + 16 g + [0, 16) of row r; the scale of 32-channel block g of row r
// comes from lane l.
constexpr int kRing = 3;                       // steps held per wavefront
constexpr int kSmallStep = (64 + 16) * 128;    // bytes of one
constexpr int kRingBytes = 4 * kRing * kSmallStep;

inline int small_scale_ld(int groups) { return (groups + 3) / 4 * 4 + 4; }

template <int G, int NG, int OUT>
__global__ __launch_bounds__(256, 1) void matmul_small_kernel(
    MatmulArgs a, int32_t blocks_n, int32_t ld_xs) {
  constexpr int KS = 4 / NG;
  constexpr int NB = 64 * NG;
  constexpr int LDT = NB + 4;  // floats per staged token
  constexpr int kCopies = 10;  // of a step: 64 weight rows, 16 token rows
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
  const int nsteps = (H + 127) / 128;
  const int mine = (nsteps - ks + KS - 1) / KS;  // steps of this wavefront
  const int nws = a.nbk, nwb = (a.N + 127) / 128;
  const int nxs = H / G;
  uint8_t* ring = lds + wave * kRing * kSmallStep;
  uint8_t* xscale = lds + kRingBytes;
  uint8_t* wscale = xscale + 16 * ld_xs;
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
    woff[i] = (uint32_t)((weight_row(ng * 64 + 8 * i + (lane >> 3)) - n0) * H);
  const v4i wbuf = buffer_of(a.w + ((int64_t)e * a.N + n0) * H,
                             (uint32_t)((a.N - n0) * H));
  // scale bytes of the (at most three) 128-row blocks of the weight rows
  const int up_block = (a.NO + n0) / 128;
  for (int i = threadIdx.x; i < 3 * nws; i += 256) {
    const int b = i / nws;
    const int block = b == 0 ? n0 / 128
                      : gated ? up_block + b - 1 : n0 / 128 + b;
    if (block < nwb)
      wscale[b * kMaxSteps + i % nws] =
          a.ws[((int64_t)e * nwb + block) * nws + i % nws];
  }
  int wsoff[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int lr = ng * 64 + f * 16 + r16;
    const int block = weight_row(lr) / 128;
    wsoff[f] = (gated && lr >= nbo ? block - up_block + 1 : block - n0 / 128) *
               kMaxSteps;
  }

  for (int base = 0; base < er.count; base += 16) {
    const int rows = min(er.count - base, 16);
    const int64_t row0 = er.first + base;
    const v4i xbuf = buffer_of(a.q + row0 * a.ld_q,
                               (uint32_t)((rows - 1) * a.ld_q + H));
    uint32_t xoff[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      xoff[i] = (uint32_t)(min(8 * i + (lane >> 3), rows - 1) * (int)a.ld_q);
    // In a last step that ends inside the 128 channels, chunks past H repeat
    // chunk 0 of the step: in bounds, and cleared when they are read.
    auto copy_step = [&](int i) {
      const int k0 = (ks + i * KS) * 128;
      const uint32_t at = ring0 + (uint32_t)(i % kRing) * kSmallStep;
      const int c1 = chunk0 ^ 4;
      const uint32_t o0 = k0 + 16 * chunk0 < H ? 16 * chunk0 : 0;
      const uint32_t o1 = k0 + 16 * c1 < H ? 16 * c1 : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        copy_to_lds(wbuf, at + j * 1024, woff[j] + (j & 1 ? o1 : o0), k0);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        copy_to_lds(xbuf, at + 8192 + j * 1024, xoff[j] + (j & 1 ? o1 : o0),
                    k0);
    };
    for (int i = threadIdx.x; i < 16 * nxs; i += 256) {
      const int r = i / nxs;
      xscale[r * ld_xs + i % nxs] =
          a.s[(row0 + min(r, rows - 1)) * a.ld_s + i % nxs];
    }
#pragma unroll
    for (int i = 0; i < kRing; ++i)
      if (i < mine) copy_step(i);
    landed_barrier<63, 0>();  // the scale bytes are down

    v4f acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = v4f{0, 0, 0, 0};

    for (int i = 0; i < mine; ++i) {
      // this step's copies have landed; later ones may be on their way
      if (i + kRing <= mine)
        wait_for<(kRing - 1) * kCopies, 15>();
      else
        wait_for<0, 15>();
      const int step = ks + i * KS;
      const uint8_t* at = ring + i % kRing * kSmallStep;
      v4i w[4][2], x[2];
      uint32_t sw[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 4 * h + g;
#pragma unroll
        for (int f = 0; f < 4; ++f)
          w[f][h] = *reinterpret_cast<const v4i*>(
              at + (f * 16 + r16) * 128 + place(c, r16) * 16);
        x[h] = *reinterpret_cast<const v4i*>(at + 8192 + r16 * 128 +
                                             place(c, r16) * 16);
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) sw[f] = wscale[wsoff[f] + step];
      // a block past H has no scale: any finite one will do
      const uint32_t sx =
          xscale[r16 * ld_xs +
                 (G == 128 ? step : min(4 * step + g, nxs - 1))];
      wait_for<63, 0>();  // read: the ring's place may be filled again
      if (i + kRing < mine) copy_step(i + kRing);
      if (step * 128 + 128 > H) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (step * 128 + 64 * h + 16 * g < H) continue;
#pragma unroll
          for (int f = 0; f < 4; ++f) w[f][h] = v4i{0, 0, 0, 0};
          x[h] = v4i{0, 0, 0, 0};
        }
      }
#pragma unroll
      for (int f = 0; f < 4; ++f)
        acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            join(w[f][0], w[f][1]), join(x[0], x[1]), acc[f], 0, 0, 0,
            (int)sw[f], 0, (int)sx);
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

// ------------------------------------------------------------ many rows
//
// A block of four wavefronts, one per SIMD, owns TM = 64 XF token rows of one
// expert by 256 weight rows; each wavefront multiplies 32 XF tokens by 128
// weight rows in 32x32x64 steps (64 XF accumulators per lane).  K goes by in
// steps of 128 channels, held in LDS twice: while one step is multiplied, the
// next is on its way from memory straight into LDS.
//
// A step is multiplied in two halves, A with the first half of the wavefront's
// token fragments, B with the second.  B's token fragments are read from LDS
// during A; the next step's weight fragments and first token fragments during
// B, each weight fragment into the registers that its last MFMA has just left.
// So most of a step's buffer is free when A begins and the rest when B does,
// and the copies of the step after the next are dealt out evenly over the
// whole step, one or two steps before they are waited for.  Copied in one half
// only, they ask for 64 bytes a cycle, all that a CU's L1 can bring.
//
// A gated tile takes 128 gate rows and the 128 factor rows of the same
// outputs; a wavefront holds both for 64 outputs.

constexpr int kScaleLd = 36;   // bytes per row of a scale chunk (32 + pad)

template <int XF>
constexpr int tile_lds_bytes() {
  const int loop = 2 * ((64 * XF + 256) * 128 + 64 * XF * kScaleLd) +
                   3 * kMaxSteps;
  const int end = 128 * kStageLd * 4;
  return loop > end ? loop : end;
}

template <int G, int XF, int OUT, bool GATED>
__global__ __launch_bounds__(256, 1) void matmul_tile_kernel(MatmulArgs a,
                                                             int32_t tiles_n) {
  constexpr int TM = 64 * XF;
  constexpr int kX = TM * 128;             // bytes of a step's token rows
  constexpr int kStage = kX + 256 * 128;   // and with its weight rows
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
  const int nsteps = (H + 127) / 128;
  const int nwb = (a.N + 127) / 128;

  // weight row (within the expert's matrix) of local row lr of the tile
  auto weight_row = [&](int lr) {
    if (!GATED) return min(n0 + lr, a.N - 1);
    const int c = min(n0 + (lr >> 7) * 64 + (lr & 63), a.NO - 1);
    return (lr & 64) ? a.NO + c : c;
  };

  // Copies: 8 rows (1 KB) each, lane l fills place l & 7 of row l >> 3.  The
  // 64 rows of fragment f of both wavefront columns are two copies per
  // wavefront, and so are those of fragment x of both wavefront rows.
  const int chunk = place(lane & 7, wave * 8 + (lane >> 3));
  const int crow = wave * 8 + (lane >> 3);
  uint32_t xoff[XF][2], woff[4][2];
  const int64_t wfirst = n0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int x = 0; x < XF; ++x)
      xoff[x][i] = (uint32_t)(min((i * XF + x) * 32 + crow, rows - 1) *
                              (int)a.ld_q + 16 * chunk);
#pragma unroll
    for (int f = 0; f < 4; ++f)
      woff[f][i] = (uint32_t)(
          (weight_row(i * 128 + f * 32 + crow) - wfirst) * H + 16 * chunk);
  }
  const v4i xbuf = buffer_of(a.q + row0 * a.ld_q,
                             (uint32_t)((rows - 1) * a.ld_q + H));
  const v4i wbuf = buffer_of(a.w + ((int64_t)t.e * a.N + wfirst) * H,
                             (uint32_t)((a.N - wfirst) * H > 0xFFFFFFFFll
                                            ? 0xFFFFFFFFll
                                            : (a.N - wfirst) * H));
  const uint32_t lds0 = (uint32_t)(uintptr_t)(
      __attribute__((address_space(3))) uint8_t*)lds;
  // In a last step that ends inside the 128 channels, chunks past H repeat
  // chunk 0 of the step: in bounds, and cleared when they are read.
  auto step_back = [&](int k) {
    return (uint32_t)(k * 128 + 16 * chunk >= H ? 16 * chunk : 0);
  };
  auto copy_w = [&](int k, int f, int i, uint32_t back) {
    copy_to_lds(wbuf,
                lds0 + (k & 1) * kStage + kX + (i * 128 + f * 32) * 128 +
                    wave * 1024,
                woff[f][i] - back, k * 128);
  };
  auto copy_x = [&](int k, int x, int i, uint32_t back) {
    copy_to_lds(xbuf,
                lds0 + (k & 1) * kStage + (i * XF + x) * 32 * 128 +
                    wave * 1024,
                xoff[x][i] - back, k * 128);
  };
  // Copy c of half A of a step (8: weight fragments 0-2, token fragment 0),
  // and of half B (the rest, those that half B reads first).
  constexpr int kCopiesA = 8, kCopiesB = 2 * XF;
  auto copy_a = [&](int k, int c, uint32_t back) {
    if (c < 6)
      copy_w(k, c >> 1, c & 1, back);
    else
      copy_x(k, 0, c & 1, back);
  };
  auto copy_b = [&](int k, int c, uint32_t back) {
    if (XF == 4) {
      if (c < 2)
        copy_x(k, 1, c & 1, back);
      else if (c < 4)
        copy_w(k, 3, c & 1, back);
      else
        copy_x(k, c >> 1, c & 1, back);
    } else {
      if (c < 2)
        copy_w(k, 3, c & 1, back);
      else
        copy_x(k, 1, c & 1, back);
    }
  };
  // Scales.  A step needs one byte of each token row (G = 128) or four
  // (G = 32): fetched step by step they would cost a scattered load per
  // fragment, so thread r brings 32 bytes of row r at a time into LDS (two
  // such chunks, rows 36 bytes apart).  The tile's weight rows lie in at most
  // three 128-row blocks; their scale bytes are all in LDS from the start.
  constexpr int kPer = G == 128 ? 32 : 8;  // steps per chunk
  uint8_t* xscale = lds + 2 * kStage;
  uint8_t* wscale = xscale + 2 * TM * kScaleLd;
  const int nxs = H / G, nws = a.nbk;
  const uint8_t* xs_row =
      a.s + (row0 + min((int)threadIdx.x, rows - 1)) * a.ld_s;
  uint32_t xs_next[8];
  auto fetch_scales = [&](int chunk_no) {
    if (threadIdx.x >= TM) return;
    const uint8_t* p = xs_row + chunk_no * 32;
    const int left = nxs - chunk_no * 32;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      xs_next[j] = 0x7F7F7F7Fu;
      if (4 * j + 4 <= left) {
        __builtin_memcpy(&xs_next[j], p + 4 * j, 4);
      } else {
        for (int i = 4 * j; i < left; ++i)
          xs_next[j] = (xs_next[j] & ~(0xFFu << (8 * (i & 3)))) |
                       ((uint32_t)p[i] << (8 * (i & 3)));
      }
    }
  };
  auto put_scales = [&](int chunk_no) {
    if (threadIdx.x >= TM) return;
    uint32_t* d = reinterpret_cast<uint32_t*>(
        xscale + ((chunk_no & 1) * TM + threadIdx.x) * kScaleLd);
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = xs_next[j];
  };
  const int up_block = (a.NO + n0) / 128;  // of a GATED tile's factor rows
  for (int i = threadIdx.x; i < 3 * nws; i += 256) {
    const int b = i / nws;
    const int block = b == 0 ? n0 / 128
                      : GATED ? up_block + b - 1 : n0 / 128 + b;
    if (block < nwb)
      wscale[b * kMaxSteps + i % nws] =
          a.ws[((int64_t)t.e * nwb + block) * nws + i % nws];
  }
  int wsoff[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int block = weight_row(wn * 128 + f * 32 + r32) / 128;
    wsoff[f] = (GATED && f >= 2 ? block - up_block + 1 : block - n0 / 128) *
               kMaxSteps;
  }
  uint32_t sx[XF], sw[4], sx1[XF], sw1[4];  // of this step and the next one
  auto read_scales = [&](int k) {
    const uint8_t* chunk_at = xscale + ((k / kPer) & 1) * TM * kScaleLd;
#pragma unroll
    for (int x = 0; x < XF; ++x) {
      const uint8_t* p = chunk_at + (wm * 32 * XF + x * 32 + r32) * kScaleLd;
      sx1[x] = G == 128 ? p[k % kPer]
                        : reinterpret_cast<const uint32_t*>(p)[k % kPer];
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) sw1[f] = wscale[wsoff[f] + k];
  };
  auto use_scales = [&]() {
#pragma unroll
    for (int x = 0; x < XF; ++x) sx[x] = G == 128 ? sx1[x] : sx1[x] >> (8 * g);
#pragma unroll
    for (int f = 0; f < 4; ++f) sw[f] = sw1[f];
  };

  v16f acc[4][XF];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int x = 0; x < XF; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][x][i] = 0.0f;

  // fragments of a step, in the 16-byte pieces of its two MFMA steps
  v4i fw[4][4], fx[XF][4];
  auto read_rows = [&](int k, int p, int first_row, auto last) {
    const int c = p * 2 + g;
    v4i v = *reinterpret_cast<const v4i*>(
        lds + (k & 1) * kStage + first_row * 128 + r32 * 128 +
        place(c, r32) * 16);
    if constexpr (decltype(last)::value)
      if (k * 128 + 16 * c >= H) v = v4i{0, 0, 0, 0};
    return v;
  };
  auto read_w = [&](int k, int f, int p, auto last) {
    fw[f][p] = read_rows(k, p, TM + wn * 128 + f * 32, last);
  };
  auto read_x = [&](int k, int x, int p, auto last) {
    fx[x][p] = read_rows(k, p, wm * 32 * XF + x * 32, last);
  };
  constexpr int kXA = XF / 2;  // token fragments of half A, and of half B
  constexpr int kMfma = 8 * kXA;  // of a half
  // MFMA i of a half whose first token fragment is x0: weight fragments one
  // after the other, both channel halves of each
  auto multiply = [&](int i, int x0) {
    const int f = i / (2 * kXA), h = i / kXA % 2, x = x0 + i % kXA;
    if (G == 32 && h == 1)
      // the second half's scales are two bytes further
      acc[f][x] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          join(fw[f][2], fw[f][3]), join(fx[x][2], fx[x][3]), acc[f][x], 0, 0,
          0, (int)sw[f], 2, (int)sx[x]);
    else
      acc[f][x] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          join(fw[f][2 * h], fw[f][2 * h + 1]),
          join(fx[x][2 * h], fx[x][2 * h + 1]), acc[f][x], 0, 0, 0,
          (int)sw[f], 0, (int)sx[x]);
    __builtin_amdgcn_sched_barrier(0);
  };
  using Yes = std::true_type;
  using No = std::false_type;

  fetch_scales(0);
#pragma unroll
  for (int c = 0; c < kCopiesA; ++c) copy_a(0, c, step_back(0));
#pragma unroll
  for (int c = 0; c < kCopiesB; ++c) copy_b(0, c, step_back(0));
  put_scales(0);
  landed_barrier<0, 0>();
  if (nsteps > 1) {
#pragma unroll
    for (int c = 0; c < kCopiesA; ++c) copy_a(1, c, step_back(1));
#pragma unroll
    for (int c = 0; c < kCopiesB; ++c) copy_b(1, c, step_back(1));
  }
  read_scales(0);
  use_scales();
#pragma unroll
  for (int x = 0; x < kXA; ++x)
#pragma unroll
    for (int p = 0; p < 4; ++p) read_x(0, x, p, Yes{});
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int p = 0; p < 4; ++p) read_w(0, f, p, Yes{});
  __builtin_amdgcn_sched_barrier(0);

  // One step.  `more`: another one follows; `copy`: and one after that;
  // `last`: this is, and `next_last`: the next one is, the last.  The waits
  // count the copies that may still be on their way: at barrier A all of the
  // next step's, at barrier B those of its second token fragments and of the
  // step after it.  (Once per chunk of token scales, 32 steps or 8 for G = 32,
  // all of them are waited for: the compiler, which sees no copies, waits for
  // the scales that put_scales writes as for its own last load.)  At barrier A
  // the four reads of weight fragment 3, always the last ones, may be too: its
  // rows are overwritten after barrier B only.
  auto step = [&](int k, auto more_, auto copy_, auto last, auto next_last) {
    constexpr bool more = decltype(more_)::value;
    constexpr bool copy = decltype(copy_)::value;
    const uint32_t back = step_back(k + 2);
    landed_barrier<more ? kCopiesA + kCopiesB : 0, 4>();
#pragma unroll
    for (int i = 0; i < kMfma; ++i) {
      if constexpr (copy) {
#pragma unroll
        for (int c = i * kCopiesA / kMfma; c < (i + 1) * kCopiesA / kMfma; ++c)
          copy_a(k + 2, c, back);
      }
      if (i < 4) {
#pragma unroll
        for (int x = kXA; x < XF; ++x) read_x(k, x, i, last);
      }
      multiply(i, 0);
    }
    if constexpr (more)
      landed_barrier<copy ? kCopiesA + 2 * kXA : 2 * kXA, 0>();
    if constexpr (copy) {
      // one chunk ahead: fetched in a chunk's first step, put down in its
      // second
      const int next = (k / kPer + 1) * kPer;
      if (k % kPer == 0 && next < nsteps) fetch_scales(k / kPer + 1);
      if (k % kPer == 1 && next < nsteps) put_scales(k / kPer + 1);
    }
    if constexpr (more) read_scales(k + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kMfma; ++i) {
      if constexpr (copy) {
#pragma unroll
        for (int c = i * kCopiesB / kMfma; c < (i + 1) * kCopiesB / kMfma; ++c)
          copy_b(k + 2, c, back);
      }
      if constexpr (more) {
        // a weight fragment's registers take the next step's as soon as its
        // MFMAs are issued
        constexpr int kF = 2 * kXA;  // MFMAs of a weight fragment
        if (i < kF) {
#pragma unroll
          for (int p = i * 4 / kF; p < (i + 1) * 4 / kF; ++p)
#pragma unroll
            for (int x = 0; x < kXA; ++x) read_x(k + 1, x, p, next_last);
        } else {
#pragma unroll
          for (int p = i % kF * 4 / kF; p < (i % kF + 1) * 4 / kF; ++p)
            read_w(k + 1, i / kF - 1, p, next_last);
        }
      }
      multiply(i, kXA);
    }
    if constexpr (more) {
      use_scales();
#pragma unroll
      for (int p = 0; p < 4; ++p) read_w(k + 1, 3, p, next_last);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  int k = 0;
  for (; k + 2 < nsteps; ++k) step(k, Yes{}, Yes{}, No{}, No{});
  if (k + 1 < nsteps) step(k++, Yes{}, No{}, No{}, Yes{});
  step(k, No{}, No{}, Yes{}, No{});

  finish_tile<XF, OUT, GATED>(a, t.e, row0, rows, n0, acc, lds);
}

// ------------------------------------------------------------ entry points

template <int G, int NG, int OUT>
mxq_status launch_small(const MatmulArgs& a, hipStream_t s) {
  const int nbo = a.act == kActSiluMul ? 32 * NG : 64 * NG;
  const int64_t bn = ceil_div(a.NO, nbo);
  if (bn * a.E > max_blocks(256)) return MXQ_ERR_UNSUPPORTED;
  const int ld_xs = small_scale_ld(a.H / G);
  const int lds = kRingBytes + 16 * ld_xs + 3 * kMaxSteps;
  static_assert(kRingBytes >= 4 * 16 * (64 + 4) * 4 &&
                    kRingBytes >= 16 * (256 + 4) * 4,
                "the joined K parts fit the rings");
  auto* k = &matmul_small_kernel<G, NG, OUT>;
  if (hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                          hipFuncAttributeMaxDynamicSharedMemorySize,
                          lds) != hipSuccess) {
    (void)hipGetLastError();
    return MXQ_ERR_HIP;
  }
  k<<<(unsigned)(bn * a.E), 256, lds, s>>>(a, (int32_t)bn, ld_xs);
  return launch_status();
}

template <int G, int XF, int OUT>
mxq_status launch_tile(const MatmulArgs& a, hipStream_t s) {
  const int64_t tn = ceil_div(a.NO, a.act == kActSiluMul ? 128 : 256);
  // every expert ends in at most one partial row tile
  const int64_t tm = a.num_rows / (64 * XF) + a.E;
  const int64_t blocks = ceil_div(tm * tn, 8) * 8;
  if (blocks > max_blocks(256)) return MXQ_ERR_UNSUPPORTED;
  constexpr int lds = tile_lds_bytes<XF>();
  auto* k = a.act == kActSiluMul ? &matmul_tile_kernel<G, XF, OUT, true>
                                 : &matmul_tile_kernel<G, XF, OUT, false>;
  if (hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                          hipFuncAttributeMaxDynamicSharedMemorySize,
                          lds) != hipSuccess) {
    (void)hipGetLastError();
    return MXQ_ERR_HIP;
  }
  k<<<(unsigned)blocks, 256, lds, s>>>(a, (int32_t)tn);
  return launch_status();
}

// The kernel for `expected` rows in a busy expert.  Measured with top-8
// routings over 32 experts whose fullest holds 2.6 times the mean, gate/up
// (4096 x 7168, G = 128) and down (7168 x 2048, G = 32), us:
//   mean rows        4         16        64        128       256       512
//   few rows     152, 90   274, 122  765, 326
//   128-row tile 161, 106  178, 112  231, 124  236, 158  386, 227  607, 394
//   256-row tile 186, 126  201, 131  206, 144  285, 159  313, 209  507, 323
// (the weights alone take 177 and 89 us at 5.3 TB/s; gate/up with few rows
// leaves experts without a row out).  A 128-row tile takes 0.6 of a 256-row
// one's time, both one to a CU, so the smaller one is taken where that many
// rounds of the 256 CUs are over sooner: 375 mean rows of 24 experts of 1432 x
// 1376 take 43 against 58 us in two rounds either way, 750 take 80 against 63.
template <int G, int OUT>
mxq_status launch(const MatmulArgs& a, int64_t expected, hipStream_t s) {
  constexpr int64_t kCus = 256;
  if (expected > 12) {
    const int64_t columns =
        a.E * ceil_div(a.NO, a.act == kActSiluMul ? 128 : 256);
    const int64_t rounds4 = ceil_div(columns * ceil_div(expected, 256), kCus);
    const int64_t rounds2 = ceil_div(columns * ceil_div(expected, 128), kCus);
    return rounds2 * 3 <= rounds4 * 5 ? launch_tile<G, 2, OUT>(a, s)
                                      : launch_tile<G, 4, OUT>(a, s);
  }
  // 256 weight rows per block once that makes a block for every CU: longer
  // runs, so a block's start costs less (down, mean 8: 86 against 102 us);
  // else 64, and the K axis is split.  A group of 128 outputs stays in one
  // block: 128 weight rows at least, 256 when gated.
  if (ceil_div(a.N, 256) * a.E >= 256 ||
      (OUT == kOutG128 && a.act == kActSiluMul))
    return launch_small<G, 4, OUT>(a, s);
  return launch_small<G, OUT == kOutG128 ? 2 : 1, OUT>(a, s);
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
  if (expected_m > INT32_MAX) expected_m = INT32_MAX;
  if (act != MXQ_ACT_NONE && act != MXQ_ACT_SILU && act != MXQ_ACT_SILU_MUL)
    return MXQ_ERR_UNSUPPORTED;
  if (E < 1 || E > MXQ_MAX_LOCAL_EXPERTS || N < 1 || H < 1 || H % G != 0 ||
      num_rows < 0 || num_rows > INT32_MAX || expected_m < 0)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (act == MXQ_ACT_SILU_MUL && N % 2 != 0) return MXQ_ERR_INVALID_ARGUMENT;
  const int32_t NO = act == MXQ_ACT_SILU_MUL ? N / 2 : N;
  const int unit = OUT == kOutBf16 ? 4 : OUT == kOutG128 ? 128 : 32;
  if (NO % unit != 0) return MXQ_ERR_INVALID_ARGUMENT;
  // row counts are rounded up to whole tiles in 32 bits
  if (H > MXQ_MAX_HIDDEN || (int64_t)N * H > INT32_MAX ||
      num_rows > MXQ_MAX_MATMUL_ROWS)
    return MXQ_ERR_UNSUPPORTED;
  if (num_rows == 0) return MXQ_OK;
  if (q == nullptr || scales == nullptr || w == nullptr ||
      w_scales == nullptr || offsets == nullptr || counts == nullptr ||
      out == nullptr)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || ld_q % 16 != 0 || ld_q < H || ld_s < H / G ||
      !aligned16(w) || ld_out < NO)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (ld_q > MXQ_MAX_MATMUL_LD || ld_s > MXQ_MAX_MATMUL_LD)
    return MXQ_ERR_UNSUPPORTED;
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
    default:  // quantized rows of e4m3 only
      return MXQ_ERR_UNSUPPORTED;
  }
}
