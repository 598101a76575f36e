// moe_balance_loss, moe_balance_loss_backward: the router's balance loss per
// sequence, its log-sum-exp penalty, and their gradient to the logits.
//
//   p_te  = softmax(l_t)_e, or sigmoid(l_te) over the row's sum of them
//   P_e   = mean of p_te over the sequence's n tokens
//   loss  = E sum_e (c_e / sum_j c_j) P_e       c_e: the sequence's choices of e
//   z     = mean of (log sum_e exp l_te)^2
//   dl_te = grad E / (n sum_j c_j) p_te (c_e - sum_j p_tj c_j)
//           (times 1 - sigmoid(l_te) for sigmoid scores)
//           + grad_z 2 / n lse_t softmax(l_t)_e
//
// A row of E logits is held by L lanes in C chunks of four neighbouring experts
// per lane, so a wavefront works on 64 / L tokens at once, every chunk is one
// load of neighbouring lanes, and a row's maximum and sums are log2 L steps of
// DPP for all of its tokens.  Sums over tokens stay in registers, one per
// expert, until a block is through its share of a sequence; no float atomics,
// so equal calls give equal bytes.  Choices are counted in LDS in whole numbers.
#include <algorithm>
#include <type_traits>

#include "mxq_device.hpp"
#include "mxq_host.hpp"

namespace {

using namespace mxq;

// ------------------------------------------------ reductions over L lanes

template <int CTRL>
__device__ __forceinline__ uint32_t paired(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF,
                                               false);
}

// f over groups of L neighbouring lanes (a power of two from 4 on), for every
// lane of a group: quad permutes, mirrors of 8 and 16 lanes, and swaps of rows.
template <int L, typename F>
__device__ __forceinline__ uint32_t over_group(uint32_t v, F f) {
  v = f(v, paired<0xB1>(v));
  v = f(v, paired<0x4E>(v));
  if constexpr (L >= 8) v = f(v, paired<0x141>(v));
  if constexpr (L >= 16) v = f(v, paired<0x140>(v));
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = f(r[0], r[1]);
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = f(r[0], r[1]);
  }
  return v;
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return __uint_as_float(
      over_group<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
      }));
}

template <int L>
__device__ __forceinline__ float group_maxf(float v) {
  return __uint_as_float(
      over_group<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
      }));
}

template <int L>
__device__ __forceinline__ int group_maxi(int v) {
  return (int)over_group<L>((uint32_t)v, [](uint32_t a, uint32_t b) {
    return (uint32_t)max((int)a, (int)b);
  });
}

// ------------------------------------------------------------- one row

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kFltMax = 3.402823466e38f;

// exp(x) for x <= 0.  The product with log2(e) is rounded once: exp is off by
// a factor of at most 1 + (1.3 |x| + 2) 2^-24, which is little where it is not
// tiny.
__device__ __forceinline__ float exp_neg(float x) {
  return __builtin_amdgcn_exp2f(x * kLog2e);
}

template <int N>
struct Row {
  float p[N];     // shares: softmax, or sigmoids over their sum
  float back[N];  // 1 - sigmoid
  float soft[N];  // softmax of a sigmoid router, where z is wanted
  float top;      // largest logit
  float lse;      // log-sum-exp, 0 of a row without a live logit
};

// Sigmoids are taken times exp(-min(top, 0)): their shares are right also
// where the sigmoids themselves are too small for fp32.
template <int L, int N, bool SIGMOID, bool Z>
__device__ __forceinline__ void row_shares(const float (&l)[N], Row<N>& r) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, l[i]);
  m = group_maxf<L>(m);
  r.top = m;
  m = fmaxf(m, -kFltMax);  // no live logit: every share is 0
  float x[N], total = 0.0f;
  if (!SIGMOID || Z) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = exp_neg(l[i] - m);
      total += x[i];
    }
    total = group_sum<L>(total);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
    if (Z)
      r.lse = total > 0.0f
                  ? m + kLn2 * __builtin_amdgcn_logf(total) : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) (SIGMOID ? r.soft : r.p)[i] = x[i] * inv;
  }
  if (SIGMOID) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float a = exp_neg(-fabsf(l[i]));
      const float q = __builtin_amdgcn_rcpf(1.0f + a);
      const bool pos = l[i] > 0.0f;
      r.back[i] = (pos ? a : 1.0f) * q;
      x[i] = (pos ? 1.0f : a) * q;
    }
    if (__ballot(m < 0.0f) != 0) {
      // below 0 throughout: exp(l - m) in the place of exp(l)
#pragma unroll
      for (int i = 0; i < N; ++i)
        x[i] = m < 0.0f ? exp_neg(l[i] - m) * r.back[i] : x[i];
    }
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) total += x[i];
    total = group_sum<L>(total);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) r.p[i] = x[i] * inv;
  }
}

// The lane's 4 C experts of a row are those from 4 L i + 4 lane, i < C.  VEC:
// rows (and rows of counts) start on four experts' bytes, E % 4 == 0.  What
// lies past E is read from the row's end instead, so that no load hangs on a
// branch, and is then replaced.
template <int L, int C, bool BF16, bool VEC>
__device__ __forceinline__ void load_chunks(const void* row, int E, int lane,
                                            float (&v)[4 * C]) {
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int e = 4 * L * i + 4 * lane;
    if constexpr (VEC) {
      const int at = min(e, E - 4);
      if constexpr (BF16) {
        const uint2 w = *reinterpret_cast<const uint2*>(
            static_cast<const uint16_t*>(row) + at);
        v[4 * i] = bf16_lo(w.x);
        v[4 * i + 1] = bf16_hi(w.x);
        v[4 * i + 2] = bf16_lo(w.y);
        v[4 * i + 3] = bf16_hi(w.y);
      } else {
        const float4 w = *reinterpret_cast<const float4*>(
            static_cast<const float*>(row) + at);
        v[4 * i] = w.x;
        v[4 * i + 1] = w.y;
        v[4 * i + 2] = w.z;
        v[4 * i + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = min(e + j, E - 1);
        if constexpr (BF16)
          v[4 * i + j] = __uint_as_float(
              (uint32_t)static_cast<const uint16_t*>(row)[at] << 16);
        else
          v[4 * i + j] = static_cast<const float*>(row)[at];
      }
    }
  }
}

template <int L, int C, bool VEC>
__device__ __forceinline__ void load_counts(const int32_t* row, int E, int lane,
                                            int (&c)[4 * C]) {
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int e = 4 * L * i + 4 * lane;
    if constexpr (VEC) {
      const int4 w = *reinterpret_cast<const int4*>(row + min(e, E - 4));
      c[4 * i] = w.x;
      c[4 * i + 1] = w.y;
      c[4 * i + 2] = w.z;
      c[4 * i + 3] = w.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) c[4 * i + j] = row[min(e + j, E - 1)];
    }
  }
#pragma unroll
  for (int i = 0; i < 4 * C; ++i)
    if (i / 4 * 4 * L + 4 * lane + i % 4 >= E) c[i] = 0;
}

template <int L, int C, bool BF16, bool VEC>
__device__ __forceinline__ void store_chunks(void* row, int E, int lane,
                                             const float (&g)[4 * C]) {
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int e = 4 * L * i + 4 * lane;
    uint16_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[j] = __builtin_bit_cast(uint16_t, (__bf16)g[4 * i + j]);
    if constexpr (VEC) {
      if (e >= E) continue;
      if constexpr (BF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(row) + e) =
            uint2{(uint32_t)h[0] | ((uint32_t)h[1] << 16),
                  (uint32_t)h[2] | ((uint32_t)h[3] << 16)};
      else
        *reinterpret_cast<float4*>(static_cast<float*>(row) + e) =
            float4{g[4 * i], g[4 * i + 1], g[4 * i + 2], g[4 * i + 3]};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (e + j >= E) continue;
        if constexpr (BF16)
          static_cast<uint16_t*>(row)[e + j] = h[j];
        else
          static_cast<float*>(row)[e + j] = g[4 * i + j];
      }
    }
  }
}

// Logits: -inf for NaN too and past E; +inf counts as the largest finite
// value.
template <int L, int N>
__device__ __forceinline__ void as_logits(float (&v)[N], int E, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool in = i / 4 * 4 * L + 4 * lane + i % 4 < E;
    v[i] = in && v[i] == v[i] ? fminf(v[i], kFltMax) : -__builtin_inff();
  }
}

// ------------------------------------------------------------- sequences

struct BalanceArgs {
  const void* logits;
  int64_t ld;
  const int32_t* ids;  // [T, K]
  int32_t T, E, K, S;
  const int32_t* offsets;  // [S + 1] or null
  const int32_t* lens;     // [S] or null
  float* loss;      // [S]
  float* z;         // [S] or null
  int32_t* counts;  // [S, E]
  float* probs;     // [S, E]
  // two launches: a block's sums of the tokens it has of a sequence
  int32_t chunk;  // tokens per block
  int32_t epad;   // columns of a row of sums
  float* part_p;  // [blocks + S][epad]
  int32_t* part_c;
  float* part_z;  // [blocks + S]
  double* piece;  // [S][column blocks][2]
  uint32_t* done;  // [S]
};

// First token of sequence s and the end of its tokens, inside the batch
// whatever the device data say.
struct Tokens {
  int32_t first, end;
};

__device__ __forceinline__ Tokens sequence(const int32_t* offsets,
                                           const int32_t* lens, int32_t T,
                                           int s) {
  int32_t first = 0, n = T;
  if (offsets != nullptr) {
    first = min(T, max(offsets[s], 0));
    n = max(min(T, max(offsets[s + 1], 0)) - first, 0);
  }
  if (lens != nullptr) n = min(n, max(lens[s], 0));
  return Tokens{first, first + n};
}

// ------------------------------------------------------------- forward

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;

// Sums over tokens [lo, hi) by one block: shares into sum[e], choices into
// cnt[e], squared log-sum-exps into the return value (of every thread).
template <int L, int C, bool BF16, bool VEC, bool SIGMOID, bool Z>
__device__ __forceinline__ float block_sums(const BalanceArgs& a, int32_t lo,
                                            int32_t hi, float* sum /*[waves]
                                            [W]*/, int32_t* cnt,
                                            float* zsum /*[waves]*/) {
  constexpr int TG = 64 / L, W = 4 * L * C, N = 4 * C;
  constexpr int kSlots = kWaves * TG;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int at = lane & (L - 1);
  auto load = [&](int32_t t, float (&v)[N]) {
    load_chunks<L, C, BF16, VEC>(static_cast<const char*>(a.logits) +
                                     min(t, hi - 1) * a.ld * (BF16 ? 2 : 4),
                                 a.E, at, v);
  };
  // the first rows are on their way while choices are counted, the next ones
  // while a row is worked on; a wavefront without a token (a sequence may have
  // none at all) loads nothing
  float next[N];
  int32_t tw = lo + wave * TG;  // the wavefront's first token
  if (tw < hi) load(tw + lane / L, next);
  for (int i = threadIdx.x; i < W; i += kThreads) cnt[i] = 0;
  __syncthreads();
  for (int32_t i = lo * a.K + threadIdx.x; i < hi * a.K; i += kThreads) {
    const int id = a.ids[i];
    if (id >= 0 && id < a.E) atomicAdd(&cnt[id], 1);
  }
  float acc[N], zacc = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  for (; tw < hi; tw += kSlots) {
    const int32_t t = tw + lane / L;
    float l[N];
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = t < hi ? next[i] : -__builtin_inff();
    if (tw + kSlots < hi) load(t + kSlots, next);
    as_logits<L>(l, a.E, at);
    Row<N> r;
    row_shares<L, N, SIGMOID, Z>(l, r);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += r.p[i];
    if (Z) zacc += r.lse * r.lse;
  }
  // tokens of a wavefront, then wavefronts
#pragma unroll
  for (int d = L; d < 64; d <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += __shfl_xor(acc[i], d);
    if (Z) zacc += __shfl_xor(zacc, d);
  }
  if (lane < L) {
#pragma unroll
    for (int i = 0; i < C; ++i)
      *reinterpret_cast<float4*>(sum + wave * W + 4 * L * i + 4 * at) =
          float4{acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]};
  }
  if (Z && lane == 0) zsum[wave] = zacc;
  __syncthreads();
  for (int e = threadIdx.x; e < W; e += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += sum[w * W + e];
    sum[e] = v;  // column e is this thread's alone
  }
  float z = 0.0f;
  if (Z) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) z += zsum[w];
  }
  __syncthreads();
  return z;
}

// One launch: block s has the whole of sequence s.  A chain of dependent steps,
// not bytes: 48 tokens of 16 experts take 3.0 us (2.1 the gradient).
template <int L, int C, bool BF16, bool VEC, bool SIGMOID, bool Z>
__global__ __launch_bounds__(kThreads) void balance_whole_kernel(
    BalanceArgs a) {
  constexpr int W = 4 * L * C;
  __shared__ __attribute__((aligned(16))) float sum[kWaves * W];
  __shared__ int32_t cnt[W];
  __shared__ float zsum[kWaves];
  __shared__ double red[2][kWaves];
  const int s = blockIdx.x;
  const Tokens q = sequence(a.offsets, a.lens, a.T, s);
  const float z = block_sums<L, C, BF16, VEC, SIGMOID, Z>(
      a, q.first, q.end, sum, cnt, zsum);
  const double inv = q.end > q.first ? 1.0 / (q.end - q.first) : 0.0;
  double dot = 0.0, total = 0.0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    const double p = sum[e] * inv;
    a.probs[(int64_t)s * a.E + e] = (float)p;
    a.counts[(int64_t)s * a.E + e] = cnt[e];
    dot += p * cnt[e];
    total += cnt[e];
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    dot += __shfl_xor(dot, d);
    total += __shfl_xor(total, d);
  }
  if ((threadIdx.x & 63) == 0) {
    red[0][threadIdx.x >> 6] = dot;
    red[1][threadIdx.x >> 6] = total;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    dot = total = 0.0;
    for (int w = 0; w < kWaves; ++w) {
      dot += red[0][w];
      total += red[1][w];
    }
    a.loss[s] = total > 0.0 ? (float)(a.E * dot / total) : 0.0f;
    if (Z) a.z[s] = (float)(z * inv);
  }
}

// First of two launches, bound by vector instructions and one round of latency:
// 8192 fp32 rows of 256 experts (8 MB) take 7.5 us, 50000 bf16 rows of 160
// (16 MB) in 23 sequences 12.1.
//
// Block b has tokens [b * chunk, (b + 1) * chunk) and leaves a row of sums for
// each sequence that it has tokens of.  Block and sequence only go up from one
// such row to the next, so row b + s belongs to this pair alone.
template <int L, int C, bool BF16, bool VEC, bool SIGMOID, bool Z>
__global__ __launch_bounds__(kThreads) void balance_part_kernel(
    BalanceArgs a) {
  constexpr int W = 4 * L * C;
  __shared__ __attribute__((aligned(16))) float sum[kWaves * W];
  __shared__ int32_t cnt[W];
  __shared__ float zsum[kWaves];
  const int32_t from = min((int64_t)blockIdx.x * a.chunk, (int64_t)a.T);
  const int32_t to = min((int64_t)from + a.chunk, (int64_t)a.T);
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s < a.S; s += kThreads) a.done[s] = 0;
  __shared__ uint64_t has[kWaves];
  for (int base = 0; base < a.S; base += kThreads) {
    // which of the next sequences have tokens here
    const int mine = base + (int)threadIdx.x;
    const Tokens m = sequence(a.offsets, a.lens, a.T, min(mine, a.S - 1));
    const uint64_t b =
        __ballot(mine < a.S && max(from, m.first) < min(to, m.end));
    if ((threadIdx.x & 63) == 0) has[threadIdx.x >> 6] = b;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) {
      for (uint64_t left = has[w]; left != 0; left &= left - 1) {
        const int s = base + w * 64 + __ffsll((unsigned long long)left) - 1;
        const Tokens q = sequence(a.offsets, a.lens, a.T, s);
        const float z = block_sums<L, C, BF16, VEC, SIGMOID, Z>(
            a, max(from, q.first), min(to, q.end), sum, cnt, zsum);
        const int64_t row = (int64_t)blockIdx.x + s;
        for (int e = threadIdx.x; e < a.E; e += kThreads) {
          a.part_p[row * a.epad + e] = sum[e];
          a.part_c[row * a.epad + e] = cnt[e];
        }
        if (Z && threadIdx.x == 0) a.part_z[row] = z;
        __syncthreads();
      }
    }
    __syncthreads();
  }
}

// Second (6.9 us after 512 blocks, 7.2 with 23 sequences: loads that wait for
// each other): a block joins 32 experts' sums of one sequence, in a fixed order;
// the last block of a sequence joins what they add to its loss.  Eight lanes hold a
// row's 32 columns, so a block has 128 rows in flight, two of each at a time.
constexpr int kCols = 32;
constexpr int kJoinThreads = 1024;
constexpr int kJoinRows = kJoinThreads / 8;
constexpr int kJoinWaves = kJoinThreads / 64;

__global__ __launch_bounds__(kJoinThreads) void balance_join_kernel(
    BalanceArgs a, int32_t ncol) {
  __shared__ double p[kJoinWaves][kCols];
  __shared__ int32_t c[kJoinWaves][kCols];
  __shared__ double zs[kJoinWaves];
  const int s = blockIdx.x / ncol, j = blockIdx.x % ncol;
  const Tokens q = sequence(a.offsets, a.lens, a.T, s);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = threadIdx.x >> 3, c4 = (threadIdx.x & 7) * 4;
  double v[4] = {0.0, 0.0, 0.0, 0.0}, z = 0.0;
  int32_t n[4] = {0, 0, 0, 0};
  if (q.end > q.first) {
    const int b0 = q.first / a.chunk, b1 = (q.end - 1) / a.chunk;
    for (int b = b0 + r; b <= b1; b += 2 * kJoinRows) {
      float4 x[2];
      int4 k[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t row = (int64_t)min(b + i * kJoinRows, b1) + s;
        const int64_t at = row * a.epad + j * kCols + c4;
        x[i] = *reinterpret_cast<const float4*>(a.part_p + at);
        k[i] = *reinterpret_cast<const int4*>(a.part_c + at);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (b + i * kJoinRows > b1) continue;
        v[0] += x[i].x; v[1] += x[i].y; v[2] += x[i].z; v[3] += x[i].w;
        n[0] += k[i].x; n[1] += k[i].y; n[2] += k[i].z; n[3] += k[i].w;
      }
    }
    if (a.z != nullptr && j == 0)
      for (int b = b0 + (int)threadIdx.x; b <= b1; b += kJoinThreads)
        z += a.part_z[(int64_t)b + s];
  }
#pragma unroll
  for (int d = 8; d < 64; d <<= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] += __shfl_xor(v[i], d);
      n[i] += __shfl_xor(n[i], d);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) z += __shfl_xor(z, d);
  if (lane < 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[wave][c4 + i] = v[i];
      c[wave][c4 + i] = n[i];
    }
  }
  if (lane == 0) zs[wave] = z;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  const double inv = q.end > q.first ? 1.0 / (q.end - q.first) : 0.0;
  double dot = 0.0, total = 0.0;
  z = lane < kJoinWaves ? zs[lane] : 0.0;
  const int e = j * kCols + lane;
  if (lane < kCols && e < a.E) {
    double sum = 0.0;
    int32_t k = 0;
#pragma unroll
    for (int i = 0; i < kJoinWaves; ++i) {
      sum += p[i][lane];
      k += c[i][lane];
    }
    sum *= inv;
    a.probs[(int64_t)s * a.E + e] = (float)sum;
    a.counts[(int64_t)s * a.E + e] = k;
    dot = sum * k;
    total = k;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    dot += __shfl_xor(dot, d);
    total += __shfl_xor(total, d);
    z += __shfl_xor(z, d);
  }
  if (lane == 0 && a.z != nullptr && j == 0) a.z[s] = (float)(z * inv);
  if (ncol > 1) {
    double* piece = a.piece + (int64_t)s * ncol * 2;
    uint32_t before = 0;
    if (lane == 0) {
      __hip_atomic_store(piece + 2 * j, dot, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(piece + 2 * j + 1, total, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
      before = __hip_atomic_fetch_add(a.done + s, 1u, __ATOMIC_ACQ_REL,
                                      __HIP_MEMORY_SCOPE_AGENT);
    }
    before = (uint32_t)__builtin_amdgcn_readfirstlane((int)before);
    if (before + 1 != (uint32_t)ncol) return;
    // at most 32 pieces, a lane each
    static_assert(MXQ_MAX_ROUTE_EXPERTS / kCols <= 64, "one piece a lane");
    dot = total = 0.0;
    if (lane < ncol) {
      dot = __hip_atomic_load(piece + 2 * lane, __ATOMIC_RELAXED,
                              __HIP_MEMORY_SCOPE_AGENT);
      total = __hip_atomic_load(piece + 2 * lane + 1, __ATOMIC_RELAXED,
                                __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      dot += __shfl_xor(dot, d);
      total += __shfl_xor(total, d);
    }
  }
  if (lane != 0) return;
  a.loss[s] = total > 0.0 ? (float)(a.E * dot / total) : 0.0f;
}

// ------------------------------------------------------------- backward

struct BalanceBackArgs {
  const float* grad;    // [S] or null
  const float* grad_z;  // [S] or null
  const void* logits;
  int64_t ld;
  const int32_t* counts;  // [S, E]
  int32_t T, E, S;
  const int32_t* offsets;
  const int32_t* lens;
  const void* add;  // [T, ld_add] or null
  int64_t ld_add;
  void* out;
  int64_t ld_out;
  int32_t chunk;  // tokens per block
};

constexpr int kBackWaves = 4;

// 8.0 us for 8192 fp32 rows of 256 experts (16 MB), 16.8 for 50000 bf16 rows of
// 160 (32 MB), where the row's steps bound it, not the bytes.
//
// Counts enter as their differences to the largest logit's expert: the shares
// add up to one, so that takes nothing away, and where one share is nearly all
// of it the others' keep their bits.
template <int L, int C, bool BF16, bool VEC, bool SIGMOID, bool Z>
__global__ __launch_bounds__(kBackWaves * 64) void balance_backward_kernel(
    BalanceBackArgs a) {
  constexpr int TG = 64 / L, kSlots = kBackWaves * TG, N = 4 * C;
  constexpr int kSize = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int at = lane & (L - 1), gid = lane / L;
  const int32_t from = min((int64_t)blockIdx.x * a.chunk, (int64_t)a.T);
  const int32_t to = min((int64_t)from + a.chunk, (int64_t)a.T);
  int have = -1;  // the sequence whose counts and factors these are
  int c[N];
  float coef = 0.0f, zcoef = 0.0f;
  Tokens q{0, 0};
#pragma unroll
  for (int i = 0; i < N; ++i) c[i] = 0;
  // ends of the first 64 sequences: asked for ahead of the rows, so that the
  // search and the loads that follow from it need not wait for those
  int32_t end0 = 0;
  if (a.offsets != nullptr) end0 = a.offsets[min(lane, a.S - 1) + 1];
  for (int32_t tw = from + wave * TG; tw < to; tw += kSlots) {
    const int32_t t = tw + gid;
    const int64_t tc = min(t, to - 1);
    float l[N], add[N];
    load_chunks<L, C, BF16, VEC>(
        static_cast<const char*>(a.logits) + tc * a.ld * kSize, a.E, at, l);
    if (a.add != nullptr) {
      load_chunks<L, C, BF16, VEC>(
          static_cast<const char*>(a.add) + tc * a.ld_add * kSize, a.E, at,
          add);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) add[i] = 0.0f;
    }
    int s = 0;
    if (a.offsets != nullptr) {
      // as many sequences as end at or before the token
      auto count = [&](int base, int32_t end) {
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          const int n = __popcll(__ballot(base + lane < a.S && end <= tw + g));
          if (g == gid) s += n;
        }
      };
      count(0, end0);
      for (int base = 64; base < a.S; base += 64)
        count(base, a.offsets[min(base + lane, a.S - 1) + 1]);
      s = min(s, a.S - 1);  // past the last: not among its tokens
    }
    if (__ballot(s != have) != 0) {
      have = s;
      q = sequence(a.offsets, a.lens, a.T, s);
      const float n = (float)max(q.end - q.first, 1);
      float total = 0.0f;
      if (a.grad != nullptr) {
        load_counts<L, C, VEC>(a.counts + (int64_t)s * a.E, a.E, at, c);
#pragma unroll
        for (int i = 0; i < N; ++i) total += (float)c[i];
        total = group_sum<L>(total);
        coef = total > 0.0f ? a.grad[s] * ((float)a.E / n) / total : 0.0f;
      }
      if (Z) zcoef = 2.0f * a.grad_z[s] / n;
    }
    as_logits<L>(l, a.E, at);
    Row<N> r;
    row_shares<L, N, SIGMOID, Z>(l, r);
    int ct = INT32_MIN;
    float dot = 0.0f, d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) ct = l[i] == r.top ? max(ct, c[i]) : ct;
    ct = group_maxi<L>(ct);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      d[i] = (float)(int)((uint32_t)c[i] - (uint32_t)ct);
      dot += r.p[i] * d[i];
    }
    dot = group_sum<L>(dot);
    const bool mine = t >= q.first && t < q.end;
    const float w = mine ? coef : 0.0f;
    // where 2 grad_z / n lse passes fp32's range, the log-sum-exp meets the
    // share first: a share of 0 then stays 0
    const bool far = Z && fabsf(zcoef * r.lse) > kFltMax;
    const float wz = Z && mine ? zcoef * (far ? 1.0f : r.lse) : 0.0f;
    const float zl = far ? r.lse : 1.0f;
    float g[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      g[i] = w * r.p[i] * (d[i] - dot);
      if (SIGMOID) g[i] *= r.back[i];
      if (Z) g[i] += wz * (zl * (SIGMOID ? r.soft : r.p)[i]);
      g[i] += add[i];
    }
    if (t < to)
      store_chunks<L, C, BF16, VEC>(
          static_cast<char*>(a.out) + t * a.ld_out * kSize, a.E, at, g);
  }
}

// ------------------------------------------------------------ entry points

// Lanes that a row takes.  Four lanes to 16 with one chunk each up to 64
// experts; then as many chunks as it takes up to 256, for a reduction's steps
// serve all tokens of a wavefront (160 experts: three chunks of 16 lanes, of
// which a sixth has nothing, against 64 lanes of which 40 have something);
// above that twice and four times the lanes.
inline int row_lanes(int32_t E) {
  return E <= 16 ? 4 : E <= 32 ? 8 : E <= 256 ? 16 : E <= 512 ? 32 : 64;
}

template <typename F>
void by_row(int32_t E, F&& f) {
  using std::integral_constant;
  auto lanes = [&](auto l, int chunks) {
    switch (chunks) {
      case 1: return f(l, integral_constant<int, 1>{});
      case 2: return f(l, integral_constant<int, 2>{});
      case 3: return f(l, integral_constant<int, 3>{});
      default: return f(l, integral_constant<int, 4>{});
    }
  };
  if (E <= 16)
    f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (E <= 32)
    f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (E <= 256)
    lanes(integral_constant<int, 16>{}, (E + 63) / 64);
  else if (E <= 512)
    f(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  else
    f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
}

template <typename F>
void by_kind(bool bf16, bool vec, bool sigmoid, bool z, F&& f) {
  using Y = std::true_type;
  using N = std::false_type;
  auto kinds = [&](auto b, auto v) {
    if (sigmoid)
      z ? f(b, v, Y{}, Y{}) : f(b, v, Y{}, N{});
    else
      z ? f(b, v, N{}, Y{}) : f(b, v, N{}, N{});
  };
  if (bf16)
    vec ? kinds(Y{}, Y{}) : kinds(Y{}, N{});
  else
    vec ? kinds(N{}, Y{}) : kinds(N{}, N{});
}

// Rows that start on four values' bytes.
inline bool row_of_fours(const void* p, int64_t ld, int64_t esz) {
  return reinterpret_cast<uintptr_t>(p) % (4 * esz) == 0 && ld % 4 == 0;
}

// Blocks of the first of two launches, and whether one launch does: a block
// for every sequence, if no lane then has more than eight rows to read.
struct BalanceGeom {
  bool whole;
  int64_t blocks, chunk;
  int32_t epad, ncol;
};

constexpr int64_t kMaxParts = 512;
constexpr int64_t kMaxTokens = MXQ_MAX_BALANCE_TOKENS;

BalanceGeom balance_geom(int64_t T, int32_t E) {
  const int64_t slots = kThreads / row_lanes(E);
  BalanceGeom g{};
  g.whole = T <= 8 * slots;
  g.blocks = std::min(kMaxParts, std::max<int64_t>(1, ceil_div(T, slots)));
  g.chunk = std::max<int64_t>(1, ceil_div(T, g.blocks));
  g.ncol = (int32_t)ceil_div(E, kCols);
  g.epad = g.ncol * kCols;
  return g;
}

size_t balance_bytes(const BalanceGeom& g, int32_t S) {
  if (g.whole) return 0;
  const size_t rows = (size_t)(g.blocks + S);
  return (size_t)S * g.ncol * 16 + rows * g.epad * 8 + rows * 4 +
         (size_t)S * 4;
}

bool balance_sizes_ok(int64_t T, int32_t E, int32_t S) {
  return T >= 0 && E >= 1 && S >= 1;
}

}  // namespace

extern "C" size_t moe_balance_loss_workspace_bytes(int64_t T, int32_t E,
                                                   int32_t S) {
  if (!balance_sizes_ok(T, E, S) || E > MXQ_MAX_ROUTE_EXPERTS ||
      T > kMaxTokens)
    return 0;
  return balance_bytes(balance_geom(T, E), S);
}

extern "C" mxq_status moe_balance_loss(
    const void* logits, mxq_out_dtype dtype, int64_t ld_logits,
    const int32_t* topk_ids, int64_t T, int32_t E, int32_t K,
    mxq_score_fn score, const int32_t* seq_offsets, const int32_t* seq_lens,
    int32_t S, float* loss, float* z_loss, int32_t* counts, float* probs,
    void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != MXQ_OUT_BF16 && dtype != MXQ_OUT_F32)
    return MXQ_ERR_UNSUPPORTED;
  if (score != MXQ_SCORE_SOFTMAX && score != MXQ_SCORE_SIGMOID)
    return MXQ_ERR_UNSUPPORTED;
  if (!balance_sizes_ok(T, E, S) || K < 1 || K > MXQ_MAX_TOPK ||
      (S > 1 && seq_offsets == nullptr))
    return MXQ_ERR_INVALID_ARGUMENT;
  // tokens and choices are counted in 32 bits, a block's at a time
  if (E > MXQ_MAX_ROUTE_EXPERTS || T > kMaxTokens / K)
    return MXQ_ERR_UNSUPPORTED;
  if (loss == nullptr || counts == nullptr || probs == nullptr ||
      (T > 0 && (logits == nullptr || topk_ids == nullptr)) || ld_logits < E)
    return MXQ_ERR_INVALID_ARGUMENT;
  const BalanceGeom g = balance_geom(T, E);
  const int64_t joins = (int64_t)S * g.ncol;
  if (joins > max_blocks(kJoinThreads) || S > max_blocks(kThreads))
    return MXQ_ERR_UNSUPPORTED;
  BalanceArgs a{};
  a.logits = logits;
  a.ld = ld_logits;
  a.ids = topk_ids;
  a.T = (int32_t)T;
  a.E = E;
  a.K = K;
  a.S = S;
  a.offsets = seq_offsets;
  a.lens = seq_lens;
  a.loss = loss;
  a.z = z_loss;
  a.counts = counts;
  a.probs = probs;
  a.chunk = (int32_t)g.chunk;
  a.epad = g.epad;
  if (!g.whole) {
    if (workspace_bytes < balance_bytes(g, S)) return MXQ_ERR_WORKSPACE;
    if (workspace == nullptr || !aligned16(workspace))
      return MXQ_ERR_INVALID_ARGUMENT;
    const int64_t rows = g.blocks + S;
    a.piece = static_cast<double*>(workspace);
    a.part_p = reinterpret_cast<float*>(a.piece + joins * 2);
    a.part_c = reinterpret_cast<int32_t*>(a.part_p + rows * g.epad);
    a.part_z = reinterpret_cast<float*>(a.part_c + rows * g.epad);
    a.done = reinterpret_cast<uint32_t*>(a.part_z + rows);
  }
  const bool vec =
      E % 4 == 0 &&
      row_of_fours(logits, ld_logits, dtype == MXQ_OUT_BF16 ? 2 : 4);
  hipStream_t s = as_stream(stream);
  by_row(E, [&](auto l, auto p) {
    constexpr int L = decltype(l)::value, C = decltype(p)::value;
    by_kind(dtype == MXQ_OUT_BF16, vec, score == MXQ_SCORE_SIGMOID,
            z_loss != nullptr, [&](auto b, auto v, auto sg, auto z) {
              constexpr bool B = decltype(b)::value, V = decltype(v)::value,
                             SG = decltype(sg)::value,
                             Z = decltype(z)::value;
              if (g.whole)
                balance_whole_kernel<L, C, B, V, SG, Z>
                    <<<(unsigned)S, kThreads, 0, s>>>(a);
              else
                balance_part_kernel<L, C, B, V, SG, Z>
                    <<<(unsigned)g.blocks, kThreads, 0, s>>>(a);
            });
  });
  if (!g.whole)
    balance_join_kernel<<<(unsigned)joins, kJoinThreads, 0, s>>>(a, g.ncol);
  return launch_status();
}

extern "C" mxq_status moe_balance_loss_backward(
    const float* grad_loss, const float* grad_z, const void* logits,
    mxq_out_dtype dtype, int64_t ld_logits, const int32_t* counts, int64_t T,
    int32_t E, mxq_score_fn score, const int32_t* seq_offsets,
    const int32_t* seq_lens, int32_t S, const void* add, int64_t ld_add,
    void* grad_logits, int64_t ld_grad, void* stream) {
  if (dtype != MXQ_OUT_BF16 && dtype != MXQ_OUT_F32)
    return MXQ_ERR_UNSUPPORTED;
  if (score != MXQ_SCORE_SOFTMAX && score != MXQ_SCORE_SIGMOID)
    return MXQ_ERR_UNSUPPORTED;
  if (!balance_sizes_ok(T, E, S) || (S > 1 && seq_offsets == nullptr) ||
      (grad_loss == nullptr && grad_z == nullptr) ||
      (grad_loss != nullptr && counts == nullptr))
    return MXQ_ERR_INVALID_ARGUMENT;
  if (E > MXQ_MAX_ROUTE_EXPERTS || T > kMaxTokens) return MXQ_ERR_UNSUPPORTED;
  if (T == 0) return MXQ_OK;
  if (logits == nullptr || grad_logits == nullptr || ld_logits < E ||
      ld_grad < E || (add != nullptr && ld_add < E))
    return MXQ_ERR_INVALID_ARGUMENT;
  const int64_t esz = dtype == MXQ_OUT_BF16 ? 2 : 4;
  BalanceBackArgs a{};
  a.grad = grad_loss;
  a.grad_z = grad_z;
  a.logits = logits;
  a.ld = ld_logits;
  a.counts = counts;
  a.T = (int32_t)T;
  a.E = E;
  a.S = S;
  a.offsets = seq_offsets;
  a.lens = seq_lens;
  a.add = add;
  a.ld_add = ld_add;
  a.out = grad_logits;
  a.ld_out = ld_grad;
  // up to 2048 blocks, each with whole rounds of its wavefronts
  const int64_t slots = kBackWaves * 64 / row_lanes(E);
  const int64_t rounds = ceil_div(ceil_div(T, slots), 2048);
  a.chunk = (int32_t)(slots * rounds);
  const unsigned blocks = (unsigned)ceil_div(T, a.chunk);
  const bool vec = E % 4 == 0 && row_of_fours(logits, ld_logits, esz) &&
                   row_of_fours(add, ld_add, esz) &&
                   row_of_fours(grad_logits, ld_grad, esz) &&
                   row_of_fours(counts, E, 4);
  hipStream_t s = as_stream(stream);
  by_row(E, [&](auto l, auto p) {
    constexpr int L = decltype(l)::value, C = decltype(p)::value;
    by_kind(dtype == MXQ_OUT_BF16, vec, score == MXQ_SCORE_SIGMOID,
            grad_z != nullptr, [&](auto b, auto v, auto sg, auto z) {
              balance_backward_kernel<L, C, decltype(b)::value,
                                      decltype(v)::value, decltype(sg)::value,
                                      decltype(z)::value>
                  <<<blocks, kBackWaves * 64, 0, s>>>(a);
            });
  });
  return launch_status();
}
