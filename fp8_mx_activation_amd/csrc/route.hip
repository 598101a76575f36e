// moe_route, moe_route_backward: the router in front of the layout.
//
// Forward, per token: scores s_e = softmax(l)_e or 1 / (1 + exp(-l_e));
// choice values c_e = s_e (+ bias_e); the K largest c_e among the experts of
// the best groups, equal values by lowest index; weights from the unbiased
// scores of the chosen.  Backward: the gradient of the weights to the logits
// (the choice itself has none).
//
// One wavefront per token; lane i owns the PER consecutive experts from
// i * PER, so a row is one vector load per lane, and the lowest lane that
// holds the maximum also holds the lowest index.  Each of the K choices is
// one wavefront maximum of ordered integer keys (six v_max with DPP operands
// for 32 bits, twice that for 64; no LDS memory).
//
// Choice values are those of 64 bits wherever they come out of an exponential:
// near a tie two experts' values lie closer than fp32 rounding, and the choice
// would then hang on the rounding of exp.  They are first taken in 32 bits with
// a bound on their error; a token that the bound does not decide (how many do
// not hangs on the values, see choose_in_32_bits) is done again in 64 bits.  A
// softmax without bias or groups keeps the order of its logits, so there the
// fp32 logits themselves are the keys and no exponential is taken for the
// choice.  The weights are computed in 64 bits (at most K exponentials per
// token, one per lane) and rounded once to fp32.
//
// Bound: a row of E logits is 0.5-4 KB, so even 8192 tokens are one or two
// microseconds of HBM time; the kernel is bound by the K dependent reductions
// of one wavefront (some 65 instructions each).  Measured in a replayed graph,
// launches included, 256 experts, top-8: softmax of bf16 logits 2.9 us for one
// token, 6.6 for 8192, 36 for 65536 (3.3, 7.4 and 41 with whole 32-bit keys, as
// for fp32); sigmoid with bias and 4 of 8 groups 5.0, 13-15 and 72-75 us
// (5.5, 15.4 and 96 with 64-bit values throughout); gradients of renormalized
// weights or sigmoids 2.5, 6.1-6.6 and 32-33 us (fp32: 134 MB), of a plain
// softmax over the whole row 3.0, 8.9-9.3 and 52-54 us.  An empty kernel takes
// 2.1 us, a launch 4.2 us of host time.
#include <algorithm>
#include <type_traits>

#include "mxq_device.hpp"
#include "mxq_host.hpp"

namespace {

using namespace mxq;

constexpr float kFltMax = 3.402823466e38f;

// ------------------------------------------------- wavefront reductions

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp32(uint32_t old, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS,
                                               0xF, false);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp64(uint64_t old, uint64_t v) {
  const uint32_t lo = dpp32<CTRL, ROWS>((uint32_t)old, (uint32_t)v);
  const uint32_t hi =
      dpp32<CTRL, ROWS>((uint32_t)(old >> 32), (uint32_t)(v >> 32));
  return ((uint64_t)hi << 32) | lo;
}

// Each step combines a lane with one below it (rows of 16 lanes by shifts of
// 1, 2, 4 and 8, then across rows), so lane 63 ends with the whole
// wavefront's value.  A lane with no source takes 0, the lowest key: a step is
// one v_max with a DPP operand.
template <int CTRL>
__device__ __forceinline__ uint32_t max_step(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF,
                                                      0xF, true));
}

__device__ __forceinline__ uint32_t wave_max_key(uint32_t v) {
  v = max_step<0x111>(v);
  v = max_step<0x112>(v);
  v = max_step<0x114>(v);
  v = max_step<0x118>(v);
  v = max_step<0x142>(v);
  v = max_step<0x143>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// A 64-bit key by halves: the low half decides among the lanes that hold the
// largest high half.
__device__ __forceinline__ uint64_t wave_max_key(uint64_t v) {
  const uint32_t hi = wave_max_key((uint32_t)(v >> 32));
  const uint32_t lo =
      wave_max_key((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ uint64_t from_lane(uint64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
  const uint32_t hi =
      (uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane);
  return ((uint64_t)hi << 32) | lo;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double sum_step(double v) {
  const uint64_t t = dpp64<CTRL, ROWS>(0, __builtin_bit_cast(uint64_t, v));
  return v + __builtin_bit_cast(double, t);
}

__device__ __forceinline__ double wave_sum64(double v) {
  v = sum_step<0x111, 0xF>(v);
  v = sum_step<0x112, 0xF>(v);
  v = sum_step<0x114, 0xF>(v);
  v = sum_step<0x118, 0xF>(v);
  v = sum_step<0x142, 0xA>(v);
  v = sum_step<0x143, 0xC>(v);
  return __builtin_bit_cast(double,
                            from_lane(__builtin_bit_cast(uint64_t, v), 63));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float sum_step(float v) {
  return v + __uint_as_float(dpp32<CTRL, ROWS>(0, __float_as_uint(v)));
}

__device__ __forceinline__ float wave_sum32(float v) {
  v = sum_step<0x111, 0xF>(v);
  v = sum_step<0x112, 0xF>(v);
  v = sum_step<0x114, 0xF>(v);
  v = sum_step<0x118, 0xF>(v);
  v = sum_step<0x142, 0xA>(v);
  v = sum_step<0x143, 0xC>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// ------------------------------------------------------------ ordered keys

// Integer whose unsigned order is the order of the value.  Key 0 stands for
// "not to be chosen": no value above -inf maps to it.
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 is 0
  const uint64_t k = (b >> 63) ? ~b : b | (1ull << 63);
  return v > -__builtin_inf() ? k : 0;
}

__device__ __forceinline__ double value_of(uint64_t k) {
  const uint64_t b = (k >> 63) ? k & ~(1ull << 63) : ~k;
  return __builtin_bit_cast(double, b);
}

__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  const uint32_t k = (b >> 31) ? ~b : b | (1u << 31);
  return v > -__builtin_inff() ? k : 0;
}

__device__ __forceinline__ float value_of(uint32_t k) {
  const uint32_t b = (k >> 31) ? k & ~(1u << 31) : ~k;
  return __builtin_bit_cast(float, b);
}

// The two largest keys of a group: (a1, a2) joined with (b1, b2).
template <typename Key>
__device__ __forceinline__ void join_top2(Key& a1, Key& a2, Key b1, Key b2) {
  const Key lesser = min(a1, b1);
  a1 = max(a1, b1);
  a2 = max(lesser, max(a2, b2));
}

// Joined with the lane that DPP control CTRL pairs this one with.
template <int CTRL>
__device__ __forceinline__ void join_paired(uint64_t& a1, uint64_t& a2) {
  join_top2(a1, a2, dpp64<CTRL, 0xF>(0, a1), dpp64<CTRL, 0xF>(0, a2));
}

template <int CTRL>
__device__ __forceinline__ void join_paired(uint32_t& a1, uint32_t& a2) {
  join_top2(a1, a2, dpp32<CTRL, 0xF>(0, a1), dpp32<CTRL, 0xF>(0, a2));
}

// The same over a group of 1, 2, 4, 8 or 16 neighbouring lanes of a DPP row:
// pairwise (quad permutes, then mirrors of 8 and 16 lanes), all groups at
// once.
template <typename Key>
__device__ __forceinline__ void join_group(int lanes, Key& m1, Key& m2) {
  if (lanes >= 2) join_paired<0xB1>(m1, m2);
  if (lanes >= 4) join_paired<0x4E>(m1, m2);
  if (lanes >= 8) join_paired<0x141>(m1, m2);
  if (lanes >= 16) join_paired<0x140>(m1, m2);
}

// --------------------------------------------------------------- row access

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

template <bool BF16>
__device__ __forceinline__ float logit_at(const void* row, int e) {
  float v;
  if constexpr (BF16)
    v = __uint_as_float(
        (uint32_t)static_cast<const uint16_t*>(row)[e] << 16);
  else
    v = static_cast<const float*>(row)[e];
  return v != v ? -__builtin_inff() : (v > kFltMax ? kFltMax : v);
}

__device__ __forceinline__ double sigmoid64(float l) {
  return 1.0 / (1.0 + exp(-(double)l));
}

// ------------------------------------------------------------------ forward

struct RouteArgs {
  const void* logits;
  int64_t ld;  // elements
  int64_t T;
  int32_t E, K;
  int32_t sigmoid;
  const float* bias;  // or null
  int32_t groups, top_groups;
  int32_t renorm;
  float scale;
  int32_t vec, vec_bias;  // rows (the bias) start on 16 bytes
  int32_t* ids;
  float* weights;
};

constexpr int kMaxGroups = 64;

// Takes the largest of the wavefront's keys (equal ones by lowest index): its
// key, 0 if none is left, and its expert in `id`.
template <int PER, typename Key>
__device__ __forceinline__ Key take_largest(int lane, Key (&key)[PER],
                                            int& id) {
  Key m = key[0];
  int at = 0;  // lowest of the lane's experts that holds m
#pragma unroll
  for (int i = 1; i < PER; ++i) {
    at = key[i] > m ? i : at;
    m = max(m, key[i]);
  }
  const Key best = wave_max_key(m);
  if (best == 0) return best;
  const int from = __ffsll((unsigned long long)__ballot(m == best)) - 1;
  const int taken = __builtin_amdgcn_readlane(at, from);
  id = from * PER + taken;
  const int mark = lane == from ? taken : -1;
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = mark == i ? 0 : key[i];
  return best;
}

// K choices; lane j keeps the j-th.  Ids stay -1 once nothing is left.
template <int PER, typename Key>
__device__ __forceinline__ void choose(int lane, int K, Key (&key)[PER],
                                       int& my_id) {
  for (int j = 0; j < K; ++j) {
    int id = -1;
    if (take_largest<PER>(lane, key, id) == 0) break;
    if (lane == j) my_id = id;
  }
}

// The same for bf16 logits, whose keys have 16 bits to spare: with the expert
// in them (the lower index the larger), the largest key says whose it is and
// is no one else's.  Rounding up keeps the order of the 16 bits, and the
// largest finite fp32 value, which stands for infinity, above bf16's.
template <int PER>
__device__ __forceinline__ void choose_packed(int lane, int K,
                                              uint32_t (&key)[PER],
                                              int& my_id) {
#pragma unroll
  for (int i = 0; i < PER; ++i)
    key[i] = key[i] == 0 ? 0
                         : ((key[i] + 0xFFFFu) & 0xFFFF0000u) |
                               (0xFFFFu - (uint32_t)(lane * PER + i));
  for (int j = 0; j < K; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = max(m, key[i]);
    const uint32_t best = wave_max_key(m);
    if (best == 0) break;
    if (lane == j) my_id = (int)(0xFFFFu - (best & 0xFFFFu));
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = key[i] == best ? 0 : key[i];
  }
}

// A group of gs experts is 1, 2, 4, 8 or 16 whole neighbouring lanes.
__device__ __forceinline__ bool whole_lanes(int gs, int per) {
  const int lanes = gs / per;
  return lanes * per == gs && lanes <= 16 && (lanes & (lanes - 1)) == 0;
}

// The choice in 32 bits, where it is certain to be that of the 64-bit values:
// false if two values that decide it lie too close, and the token goes by 64
// bits.  With u = 2^-24:
//   - a sigmoid is off by less than 4 u (3 u of its own from the sum and the
//     reciprocal, and s (1 - s) times the power's 2 u (|l| + 1)), a softmax by
//     less than 53 u (1 u, and s times 46 u of the sum over the row and 5 u);
//     adding the bias, u |c| more.  Two values that differ by 2^-20 max(1, |c|)
//     for the sigmoid, 2^-17 max(1, |c|) for the softmax, are in order;
//   - a group's value, of two values of at most 16 each, is off by less than
//     256 u: two that differ by 2^-15 are in order;
//   - without a bias the choice within the groups goes by the logits.  Logits
//     that differ by 2^-40 or more (any two beyond 2^-16 do) have scores that
//     differ in 64 bits too, but for sigmoids close to one (l > 16) and what
//     comes near 64 bits' smallest (exp(-700)).
// Where a set is cut off (the groups, the K-th choice) the next one is
// compared too.
//
// Tokens that go by 64 bits, by this rule over drawn rows of 256 experts, top-8:
// sigmoid of normal logits of deviation 2 with a bias of deviation 0.3 and 4 of
// 8 groups 0.15 %, with a bias of 0.01 1.3 %, without a bias 1.3 %; softmax of
// the same logits with a bias of 0.3 0.05 %, of 0.001 1.3 %.  The margins do not
// shrink with the scores, so flat rows mostly go by 64 bits (softmax of logits
// of deviation 0.5 with a bias of 0.001: 13 %, 512 experts and top-10 35 %), and
// so do saturated ones (sigmoid of logits of deviation 6 with a bias: nearly
// all, for the largest scores round to one).
template <int PER>
__device__ __forceinline__ bool choose_in_32_bits(const RouteArgs& a, int lane,
                                                  const float (&l)[PER],
                                                  const float (&bias)[PER],
                                                  float top, int& my_id) {
  constexpr float kLog2e = 1.44269504088896341f;
  const float inf = __builtin_inff();
  const bool biased = a.bias != nullptr;
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = key_of(l[i]);
  if (biased || a.groups > 1) {
    float c[PER];
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        c[i] = __builtin_amdgcn_rcpf(
            1.0f + __builtin_amdgcn_exp2f(-l[i] * kLog2e));
    } else {
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        c[i] = __builtin_amdgcn_exp2f((l[i] - top) * kLog2e);
        part += c[i];
      }
      const float r = __builtin_amdgcn_rcpf(wave_sum32(part));
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] *= r;
    }
    if (biased) {
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] += bias[i];
    }
    uint32_t ck[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) ck[i] = l[i] > -inf ? key_of(c[i]) : 0;
    bool keep = true;
    if (a.groups > 1) {
      const int lanes = a.E / a.groups / PER;
      uint32_t m1 = ck[0], m2 = 0;
#pragma unroll
      for (int i = 1; i < PER; ++i) join_top2<uint32_t>(m1, m2, ck[i], 0);
      join_group(lanes, m1, m2);
      const float v1 = m1 ? value_of(m1) : 0.0f;
      const float v2 = m2 ? value_of(m2) : 0.0f;
      const float value = m1 ? v1 + v2 : -inf;
      // a group's lanes compare it with one other group each
      const int shift = __popc(lanes - 1);  // lanes is a power of two
      const int group = lane >> shift, in = lane & (lanes - 1);
      bool close = !(fabsf(v1) <= 16.0f && fabsf(v2) <= 16.0f);
      int better = 0;
      for (int g0 = 0; g0 < a.groups; g0 += lanes) {
        const int g = g0 + in;
        const float v = __shfl(value, g << shift);
        const bool other = g < a.groups && g != group && v > -inf;
        close |= other && !(fabsf(v - value) > 0x1p-15f);
        const uint64_t above = __ballot(other && v > value);
        better += __popcll(above >> (group << shift) & ((1ull << lanes) - 1));
      }
      if (__ballot(close) != 0) return false;
      keep = better < a.top_groups && m1 != 0;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = !keep ? 0 : biased ? ck[i] : key[i];
  }

  bool sure = true;
  float last = kFltMax;
  const float rel = a.sigmoid ? 0x1p-20f : 0x1p-17f;
  const float low = a.sigmoid ? -700.0f : top - 700.0f;
  const float high = a.sigmoid ? 16.0f : kFltMax;
  for (int j = 0; j <= a.K; ++j) {
    int id = -1;
    const uint32_t best = take_largest<PER>(lane, key, id);
    if (best == 0) break;  // nothing left: ids from here on stay -1
    const float v = value_of(best);
    const float d = last - v;
    if (biased)
      sure &= d > rel * fmaxf(1.0f, fabsf(last));
    else
      sure &= (d > 0x1p-40f || (d == 0.0f && (j < a.K || fabsf(v) >= 0x1p-16f))) &&
              (j == a.K || (v >= low && v <= high));
    if (lane == j && j < a.K) my_id = id;
    last = v;
  }
  return sure;
}

// WIDE: 64-bit choice values; else the logits themselves are the choice.
template <int PER, bool BF16, bool WIDE>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 6) +
                    __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.T) return;
  const int E = a.E;
  const int e0 = lane * PER;
  const char* row = static_cast<const char*>(a.logits) +
                    t * a.ld * (BF16 ? 2 : 4);
  float l[PER];
  load_logits<PER, BF16>(row, E, e0, a.vec != 0, l);
  float bias[PER];
  if (WIDE && a.bias != nullptr)
    load_row<PER, false>(a.bias, E, e0, a.vec_bias != 0, bias);

  // a softmax's largest logit, and the sum of its exponentials where a single
  // one depends on it
  double top = 0.0, z = 1.0;
  if (!a.sigmoid) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = fmaxf(m, l[i]);
    const uint32_t k = wave_max_key(key_of(m));
    top = k ? (double)value_of(k) : 0.0;
  }

  int my_id = -1;  // lane j: the j-th choice
  bool chosen = false;
  if constexpr (WIDE) {
    const int gs = E / a.groups;
    if (a.groups == 1 || whole_lanes(gs, PER))
      chosen = choose_in_32_bits<PER>(a, lane, l, bias, (float)top, my_id);
    if (!chosen) {
      my_id = -1;
      double s[PER];
      if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < PER; ++i) s[i] = sigmoid64(l[i]);
      } else {
        double part = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          s[i] = exp((double)l[i] - top);
          part += s[i];
        }
        z = wave_sum64(part);
#pragma unroll
        for (int i = 0; i < PER; ++i) s[i] = s[i] / z;
      }
      if (a.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < PER; ++i) s[i] += (double)bias[i];
      }
      uint64_t key[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i)
        key[i] = l[i] > -__builtin_inff() ? key_of(s[i]) : 0;
      if (a.groups > 1) {
        // Group value: the sum of the group's two largest choice values.  A
        // group without a live expert has none and is never kept.
        const int gs = E / a.groups;
        const int lanes = gs / PER;  // of a group
        uint64_t value = 0;          // key of the lane's group's value
        int group = 0;
        const bool aligned = lanes * PER == gs && lanes <= 16 &&
                             (lanes & (lanes - 1)) == 0;
        if (aligned) {
          uint64_t m1 = key[0], m2 = 0;
#pragma unroll
          for (int i = 1; i < PER; ++i) join_top2<uint64_t>(m1, m2, key[i], 0);
          join_group(lanes, m1, m2);
          if (m1 != 0)
            value = key_of(value_of(m1) + (m2 ? value_of(m2) : 0.0));
          group = lane / max(lanes, 1);
          // kept: fewer than top_groups others are better (an equal one with a
          // lower index is)
          int better = 0;
          for (int g = 0; g < a.groups; ++g) {
            const uint64_t v = from_lane(value, g * lanes);
            better += v > value || (v == value && g < group);
          }
          const bool keep = better < a.top_groups && value != 0;
#pragma unroll
          for (int i = 0; i < PER; ++i) key[i] = keep ? key[i] : 0;
        } else {
          uint64_t mine = 0;  // lane g: the key of group g's value
          for (int g = 0; g < a.groups; ++g) {
            const int lo = g * gs, hi = lo + gs;
            uint64_t m1 = 0, m2 = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i)
              if (e0 + i >= lo && e0 + i < hi)
                join_top2<uint64_t>(m1, m2, key[i], 0);
            const uint64_t first = wave_max_key(m1);
            if (first == 0) continue;
            // the lowest lane that holds it offers its second instead
            const int owner =
                __ffsll((unsigned long long)__ballot(m1 == first)) - 1;
            const uint64_t second = wave_max_key(lane == owner ? m2 : m1);
            const uint64_t gk =
                key_of(value_of(first) + (second ? value_of(second) : 0.0));
            if (lane == g) mine = gk;
          }
          uint64_t kept = 0;  // bit g: group g may be chosen from
          for (int n = 0; n < a.top_groups; ++n) {
            const uint64_t best = wave_max_key(mine);
            if (best == 0) break;
            const int g =
                __ffsll((unsigned long long)__ballot(mine == best)) - 1;
            kept |= 1ull << g;
            if (lane == g) mine = 0;
          }
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int g = min((e0 + i) / gs, kMaxGroups - 1);
            if (!((kept >> g) & 1)) key[i] = 0;
          }
        }
      }
      choose<PER>(lane, a.K, key, my_id);
    }
  } else {
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = key_of(l[i]);
    if constexpr (BF16)
      choose_packed<PER>(lane, a.K, key, my_id);
    else
      choose<PER>(lane, a.K, key, my_id);
    chosen = true;
  }
  // a softmax's own score takes the sum over the row
  if (chosen && !a.sigmoid && !a.renorm) {
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) part += exp((double)l[i] - top);
    z = wave_sum64(part);
  }

  double p = 0.0;
  if (my_id >= 0) {
    const float mine = logit_at<BF16>(row, my_id);
    p = a.sigmoid ? sigmoid64(mine) : exp((double)mine - top);
  }
  if (a.renorm) {
    const double total = wave_sum64(p);
    p = total > 0.0 ? p / total : 0.0;
  } else {
    p = z > 0.0 ? p / z : 0.0;  // 0: no live expert
  }
  if (lane < a.K) {
    a.ids[t * a.K + lane] = my_id;
    a.weights[t * a.K + lane] = (float)((double)a.scale * p);
  }
}

// ----------------------------------------------------------------- backward

struct RouteBackArgs {
  const float* grad;  // [T, K]
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  int64_t T;
  int32_t E, K;
  int32_t sigmoid, renorm;
  float scale;
  int32_t vec_in, vec_out;
  void* out;
  int64_t ld_out;
};

// The value v of the lowest lane that holds the wavefront's largest l.
__device__ __forceinline__ double of_largest(float l, double v) {
  const uint32_t k = key_of(l);
  const int lane =
      __ffsll((unsigned long long)__ballot(k == wave_max_key(k))) - 1;
  return __builtin_bit_cast(double,
                            from_lane(__builtin_bit_cast(uint64_t, v), lane));
}

// With q_j the chosen scores over their sum: renormalized weights give
// s_j ds_j = scale * q_j * (g_j - sum_i q_i g_i), others scale * s_j * g_j.
// Sigmoid scores: dl_j = s_j ds_j (1 - s_j), with 1 - s_j = exp(-l_j) s_j, for
// the difference leaves nothing of it near one.  Softmax scores: the
// renormalized form depends on the chosen logits alone, dl_j = s_j ds_j; the
// other reads the whole row, dl_e = scale * p_e * (G_e - sum_i p_i G_i), G_e
// the sum of an expert's g_j (0 unless chosen).  The scores add up to one, so
// gradients may be taken against any one: against the largest score's, the
// sum is of what the others add and keeps its bits however little that is.
// In 64 bits, rounded to fp32 and from there to bf16.
template <int PER, bool BF16>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBackArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 6) +
                    __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.T) return;
  const int E = a.E;
  const int e0 = lane * PER;
  const char* row = static_cast<const char*>(a.logits) +
                    t * a.ld * (BF16 ? 2 : 4);
  char* out = static_cast<char*>(a.out) + t * a.ld_out * (BF16 ? 2 : 4);
  int id = -1;
  double g = 0.0;
  float lj = -__builtin_inff();
  if (lane < a.K) {
    id = a.ids[t * a.K + lane];
    if (id < 0 || id >= E) {
      id = -1;
    } else {
      g = (double)a.grad[t * a.K + lane];
      lj = logit_at<BF16>(row, id);
    }
  }
  const bool has = lj > -__builtin_inff();
  double d = 0.0;  // gradient of the lane's chosen logit
  float res[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) res[i] = 0.0f;
  if (a.sigmoid) {
    const double x = exp(-(double)lj);  // infinite below -709.8: s is 0
    const double s = has ? 1.0 / (1.0 + x) : 0.0;
    const double rest = s > 0.0 ? x * s : 1.0;  // 1 - s
    double ds = (double)a.scale * s * g;
    if (a.renorm) {
      // s over the sum, whose reciprocal may be beyond 64 bits
      const double total = wave_sum64(s);
      const double q = total > 0.0 ? s / total : 0.0;
      const double dg = g - of_largest(lj, g);
      ds = (double)a.scale * q * (dg - wave_sum64(q * dg));
    }
    d = has ? ds * rest : 0.0;
  } else if (a.renorm) {
    const uint32_t k = wave_max_key(key_of(lj));
    const double top = k ? (double)value_of(k) : 0.0;
    const double x = has ? exp((double)lj - top) : 0.0;
    const double total = wave_sum64(x);
    const double q = total > 0.0 ? x / total : 0.0;
    const double dg = g - of_largest(lj, g);
    d = (double)a.scale * q * (dg - wave_sum64(q * dg));
  } else {
    float l[PER];
    load_logits<PER, BF16>(row, E, e0, a.vec_in != 0, l);
    float m = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = fmaxf(m, l[i]);
    const uint32_t k = wave_max_key(key_of(m));
    const double top = k ? (double)value_of(k) : 0.0;
    double part = 0.0;
    double x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      x[i] = exp((double)l[i] - top);
      part += x[i];
    }
    const double z = wave_sum64(part);
    const double inv = z > 0.0 ? 1.0 / z : 0.0;
    double G[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) G[i] = 0.0;
    for (int j = 0; j < a.K; ++j) {
      const int idj = __builtin_amdgcn_readlane(id, j);
      const double gj = __builtin_bit_cast(
          double, from_lane(__builtin_bit_cast(uint64_t, g), j));
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (idj == e0 + i) G[i] += gj;
    }
    double mine = G[0];  // of an expert with the lane's largest logit
#pragma unroll
    for (int i = 1; i < PER; ++i) mine = l[i] == m ? G[i] : mine;
    const double largest = of_largest(m, mine);
    double dot = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      G[i] -= largest;
      dot += x[i] * G[i];
    }
    dot = wave_sum64(dot) * inv;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      res[i] = (float)((double)a.scale * (x[i] * inv) * (G[i] - dot));
    store_row<PER, BF16>(out, E, e0, a.vec_out != 0, res);
    return;
  }
  // An id that occurs twice adds up.
  const float df = (float)d;
  for (int j = 0; j < a.K; ++j) {
    const int idj = __builtin_amdgcn_readlane(id, j);
    const float dj = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, df), j));
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (idj == e0 + i) res[i] += dj;
  }
  store_row<PER, BF16>(out, E, e0, a.vec_out != 0, res);
}

// Wavefronts per block: four once there are more tokens than CUs; below
// that one, so that every token has a CU of its own.
inline int route_waves(int64_t T) { return T > 256 ? 4 : 1; }

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

template <typename F>
void by_experts(int32_t E, F&& f) {
  if (E <= 64)
    f(std::integral_constant<int, 1>{});
  else if (E <= 128)
    f(std::integral_constant<int, 2>{});
  else if (E <= 256)
    f(std::integral_constant<int, 4>{});
  else if (E <= 512)
    f(std::integral_constant<int, 8>{});
  else
    f(std::integral_constant<int, 16>{});
}

}  // namespace

extern "C" mxq_status moe_route(const void* logits, mxq_out_dtype dtype,
                                int64_t ld_logits, int64_t T, int32_t E,
                                int32_t K, mxq_score_fn score,
                                const float* bias, int32_t num_groups,
                                int32_t top_groups, int32_t renormalize,
                                float weight_scale, int32_t* topk_ids,
                                float* topk_weights, void* stream) {
  if (dtype != MXQ_OUT_BF16 && dtype != MXQ_OUT_F32)
    return MXQ_ERR_UNSUPPORTED;
  if (score != MXQ_SCORE_SOFTMAX && score != MXQ_SCORE_SIGMOID)
    return MXQ_ERR_UNSUPPORTED;
  if (T < 0 || T > INT32_MAX || E < 1 || K < 1 || K > MXQ_MAX_TOPK || K > E ||
      num_groups < 1 || num_groups > E || E % num_groups != 0 ||
      top_groups < 1 || top_groups > num_groups ||
      K > E / num_groups * top_groups)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (E > MXQ_MAX_ROUTE_EXPERTS || num_groups > kMaxGroups)
    return MXQ_ERR_UNSUPPORTED;
  if (T == 0) return MXQ_OK;
  if (logits == nullptr || topk_ids == nullptr || topk_weights == nullptr ||
      ld_logits < E)
    return MXQ_ERR_INVALID_ARGUMENT;
  const int64_t esz = dtype == MXQ_OUT_BF16 ? 2 : 4;
  const int waves = route_waves(T);
  RouteArgs a{logits,     ld_logits,  T,
              E,          K,          score == MXQ_SCORE_SIGMOID,
              bias,       num_groups, top_groups,
              renormalize != 0, weight_scale,
              row_vec(logits, ld_logits, esz),
              aligned16(bias),
              topk_ids,   topk_weights};
  hipStream_t s = as_stream(stream);
  // a softmax keeps the order of its logits
  const bool wide = a.sigmoid || bias != nullptr || num_groups > 1;
  by_launches(T, waves, [&](int64_t t, int64_t n, unsigned blocks) {
    a.logits = static_cast<const char*>(logits) + t * ld_logits * esz;
    a.T = n;
    a.ids = topk_ids + t * K;
    a.weights = topk_weights + t * K;
    by_experts(E, [&](auto per) {
      constexpr int kPer = decltype(per)::value;
      if (dtype == MXQ_OUT_BF16)
        wide ? route_kernel<kPer, true, true><<<blocks, waves * 64, 0, s>>>(a)
             : route_kernel<kPer, true, false>
                   <<<blocks, waves * 64, 0, s>>>(a);
      else
        wide ? route_kernel<kPer, false, true><<<blocks, waves * 64, 0, s>>>(a)
             : route_kernel<kPer, false, false>
                   <<<blocks, waves * 64, 0, s>>>(a);
    });
  });
  return launch_status();
}

extern "C" mxq_status moe_route_backward(
    const float* grad_weights, const void* logits, mxq_out_dtype dtype,
    int64_t ld_logits, const int32_t* topk_ids, int64_t T, int32_t E,
    int32_t K, mxq_score_fn score, int32_t renormalize, float weight_scale,
    void* grad_logits, int64_t ld_grad, void* stream) {
  if (dtype != MXQ_OUT_BF16 && dtype != MXQ_OUT_F32)
    return MXQ_ERR_UNSUPPORTED;
  if (score != MXQ_SCORE_SOFTMAX && score != MXQ_SCORE_SIGMOID)
    return MXQ_ERR_UNSUPPORTED;
  if (T < 0 || T > INT32_MAX || E < 1 || K < 1 || K > MXQ_MAX_TOPK)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (E > MXQ_MAX_ROUTE_EXPERTS) return MXQ_ERR_UNSUPPORTED;
  if (T == 0) return MXQ_OK;
  if (grad_weights == nullptr || logits == nullptr || topk_ids == nullptr ||
      grad_logits == nullptr || ld_logits < E || ld_grad < E)
    return MXQ_ERR_INVALID_ARGUMENT;
  const int64_t esz = dtype == MXQ_OUT_BF16 ? 2 : 4;
  const int waves = route_waves(T);
  RouteBackArgs a{grad_weights, logits, ld_logits, topk_ids, T, E, K,
                  score == MXQ_SCORE_SIGMOID, renormalize != 0, weight_scale,
                  row_vec(logits, ld_logits, esz),
                  row_vec(grad_logits, ld_grad, esz), grad_logits, ld_grad};
  hipStream_t s = as_stream(stream);
  by_launches(T, waves, [&](int64_t t, int64_t n, unsigned blocks) {
    a.grad = grad_weights + t * K;
    a.logits = static_cast<const char*>(logits) + t * ld_logits * esz;
    a.ids = topk_ids + t * K;
    a.T = n;
    a.out = static_cast<char*>(grad_logits) + t * ld_grad * esz;
    by_experts(E, [&](auto per) {
      constexpr int kPer = decltype(per)::value;
      if (dtype == MXQ_OUT_BF16)
        route_backward_kernel<kPer, true><<<blocks, waves * 64, 0, s>>>(a);
      else
        route_backward_kernel<kPer, false><<<blocks, waves * 64, 0, s>>>(a);
    });
  });
  return launch_status();
}
