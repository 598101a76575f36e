// moe_scatter_rows_backward, moe_combine_backward: the gradients of the
// expert sort and of the weighted way back.
//
// Sort (row d = src2dst[t, j] of the layout takes token row t): the token's
// gradient is the sum of its rows' gradients, dx[t] = sum_j drows[d].
// Combine (out[t] = sum_j w[t, j] y[d]): dy[d] = w[t, j] dout[t] and
// dw[t, j] = <dout[t], y[d]>.  Assignments without a row add nothing and
// have dw = 0; rows that are no destination are not written.
//
// Both move every row once and are bound by HBM: the sort's gradient reads K
// rows and writes one per token, the combine's reads one row and K rows and
// writes K.  All sums are in fp32, in a fixed order.  Measured at 8192 tokens,
// top-8, hidden 7168, bf16: sort 176-180 us (5.9 TB/s, a large copy's rate),
// combine 370-392 us (5.1-5.4 TB/s; its writes are half of the traffic), the
// gradient of its rows alone 210 us (writes), of its weights alone 155 us.  An
// expert-parallel rank's share, 512 tokens with an eighth of the assignments
// here: 5.1 us (6.2 with one wavefront per row).
#include <algorithm>

#include "mxq_device.hpp"
#include "mxq_host.hpp"

namespace {

using namespace mxq;

__device__ __forceinline__ uint32_t bf16x2_rne(float lo, float hi) {
  const uint32_t a = __builtin_bit_cast(uint16_t, (__bf16)lo);
  const uint32_t b = __builtin_bit_cast(uint16_t, (__bf16)hi);
  return a | (b << 16);
}

// Eight consecutive channels as floats.
template <bool F32>
struct Ch8;
template <>
struct Ch8<false> {
  u32x4 v;
  __device__ __forceinline__ void load_nt(const char* p) { v = load16_nt(p); }
  __device__ __forceinline__ void load(const char* p) { v = load16(p); }
  __device__ __forceinline__ void clear() { v = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = bf16_lo(v.x);
    f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y);
    f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z);
    f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w);
    f[7] = bf16_hi(v.w);
  }
};
template <>
struct Ch8<true> {
  u32x4 a, b;
  __device__ __forceinline__ void load_nt(const char* p) {
    a = load16_nt(p);
    b = load16_nt(p + 16);
  }
  __device__ __forceinline__ void load(const char* p) {
    a = load16(p);
    b = load16(p + 16);
  }
  __device__ __forceinline__ void clear() {
    a = u32x4{0, 0, 0, 0};
    b = u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = __uint_as_float(a.x);
    f[1] = __uint_as_float(a.y);
    f[2] = __uint_as_float(a.z);
    f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x);
    f[5] = __uint_as_float(b.y);
    f[6] = __uint_as_float(b.z);
    f[7] = __uint_as_float(b.w);
  }
};

template <bool F32>
__device__ __forceinline__ void store8_nt(char* p, const float (&f)[8]) {
  if constexpr (F32) {
    store16_nt(p, u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]),
                        __float_as_uint(f[2]), __float_as_uint(f[3])});
    store16_nt(p + 16, u32x4{__float_as_uint(f[4]), __float_as_uint(f[5]),
                             __float_as_uint(f[6]), __float_as_uint(f[7])});
  } else {
    store16_nt(p, u32x4{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]),
                        bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7])});
  }
}

// One block per token and slice of channels, eight channels per lane, the
// rows of eight assignments in flight before they are added (j ascending):
// the combine's access pattern without its weights.
template <bool F32_IN, bool F32_OUT>
__global__ __launch_bounds__(1024) void scatter_rows_backward_kernel(
    const char* __restrict__ rows, int64_t ld, int64_t num_rows,
    const int32_t* __restrict__ src2dst, int32_t K, int32_t H, int32_t slice,
    char* __restrict__ out, int64_t ld_out) {
  constexpr int kIn = F32_IN ? 4 : 2, kOut = F32_OUT ? 4 : 2;
  const int64_t t = blockIdx.x;
  // unsigned: a slice's end and a block's stride past it stay below 2^32
  const uint32_t c_lo = blockIdx.y * (uint32_t)slice;
  const uint32_t c_hi = min((uint32_t)H, c_lo + (uint32_t)slice);
  const int lane = threadIdx.x & 63;
  const int32_t d_lane =
      K > 0 ? src2dst[t * K + min(lane, K - 1)] : -1;
  for (uint32_t col = c_lo + threadIdx.x * 8; col < c_hi;
       col += blockDim.x * 8) {
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < K; j0 += 8) {
      Ch8<F32_IN> v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int j = j0 + u;
        const int64_t d =
            j < K ? (int64_t)__builtin_amdgcn_readlane(d_lane, j) : -1;
        if (d >= 0 && d < num_rows)
          v[u].load_nt(rows + (d * ld + col) * kIn);
        else
          v[u].clear();
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        float f[8];
        v[u].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += f[i];
      }
    }
    store8_nt<F32_OUT>(out + (t * ld_out + col) * kOut, acc);
  }
}

// One block of eight wavefronts per token.  The token's gradient row is staged
// in LDS once, then each wavefront takes one of the assignments that have a
// row, and the eighth after it: it reads row d of y, adds up the product with
// the staged row and writes row d of dy on the same pass, so y and dy are
// touched once and the dot product needs one wavefront reduction per
// assignment and no barrier.  Where fewer than five assignments have a row
// (an expert-parallel rank's share), two, four or eight wavefronts take
// vectors of a row in turn and join their sums in LDS; a token without any
// is done before its gradient is read.
constexpr int kCombineBackWaves = 8;
constexpr int kCombineBackThreads = 64 * kCombineBackWaves;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

template <bool F32_G, bool NEED_Y, bool NEED_W>
__global__ __launch_bounds__(kCombineBackThreads) void combine_backward_kernel(
    const char* __restrict__ g, int64_t ld_g, const uint16_t* __restrict__ y,
    int64_t ld_y, int64_t num_rows, const int32_t* __restrict__ src2dst,
    const float* __restrict__ w, int32_t K, int32_t H,
    uint16_t* __restrict__ dy, int64_t ld_dy, float* __restrict__ dw) {
  constexpr int kG = F32_G ? 4 : 2;
  extern __shared__ __attribute__((aligned(16))) char staged[];
  __shared__ float joined[kCombineBackWaves];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int jl = min(lane, K - 1);
  const int32_t d_lane = src2dst[t * K + jl];
  const int32_t w_lane = NEED_Y ? __float_as_int(w[t * K + jl]) : 0;
  const bool has = lane < K && d_lane >= 0 && d_lane < num_rows;
  const uint64_t rows = __ballot(has);
  if (NEED_W && wave == 0 && lane < K && !has) dw[t * K + lane] = 0.0f;
  if (rows == 0) return;
  const char* gr = g + t * ld_g * kG;
  for (int c = threadIdx.x * 16; c < H * kG; c += blockDim.x * 16)
    *reinterpret_cast<u32x4*>(staged + c) = load16(gr + c);
  __syncthreads();
  const int n = __popcll(rows);
  const int share = n == 1 ? 8 : n == 2 ? 4 : n <= 4 ? 2 : 1;  // of a row
  const int part = wave & (share - 1);
  uint64_t left = rows;
  for (int i = wave / share; i > 0; --i) left &= left - 1;
  while (left != 0) {
    const int j = __ffsll((unsigned long long)left) - 1;
    const int64_t d = __builtin_amdgcn_readlane(d_lane, j);
    const float wj = __int_as_float(__builtin_amdgcn_readlane(w_lane, j));
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    const char* yr = reinterpret_cast<const char*>(y + d * ld_y);
    char* dyr = reinterpret_cast<char*>(dy + d * ld_dy);
    // four vectors of 512 channels in flight per wavefront
    const int step = share * 512;
    for (int c0 = part * 512 + lane * 8; c0 < H; c0 += 4 * step) {
      Ch8<false> v[4];
      if constexpr (NEED_W) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int c = c0 + u * step;
          if (c < H)
            v[u].load_nt(yr + c * 2);
          else
            v[u].clear();
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + u * step;
        if (c >= H) continue;
        Ch8<F32_G> gv;
        gv.load(staged + c * kG);
        float gf[8];
        gv.get(gf);
        if constexpr (NEED_W) {
          float yf[8];
          v[u].get(yf);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = fmaf(gf[i], yf[i], sum[i]);
        }
        if constexpr (NEED_Y) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = wj * gf[i];
          store8_nt<false>(dyr + c * 2, o);
        }
      }
    }
    if constexpr (NEED_W) {
      const float s = wave_sum(((sum[0] + sum[1]) + (sum[2] + sum[3])) +
                               ((sum[4] + sum[5]) + (sum[6] + sum[7])));
      if (lane == 0) {
        if (share == 1)
          dw[t * K + j] = s;
        else
          joined[wave] = s;
      }
    }
    if (share > 1) break;  // a row per group of wavefronts
#pragma unroll
    for (int i = 0; i < kCombineBackWaves; ++i) left &= left - 1;
  }
  if constexpr (NEED_W) {
    if (share == 1) return;
    __syncthreads();
    if (left != 0 && part == 0 && lane == 0) {
      float s = joined[wave] + joined[wave + 1];
      if (share >= 4) s += joined[wave + 2] + joined[wave + 3];
      if (share == 8)
        s += (joined[wave + 4] + joined[wave + 5]) +
             (joined[wave + 6] + joined[wave + 7]);
      dw[t * K + __ffsll((unsigned long long)left) - 1] = s;
    }
  }
}

// As in the combine: below this many tokens a row is dealt to blocks of
// kBackSlice channels (more, where a grid's second dimension would pass
// 65535).
constexpr int64_t kBackSliceMaxTokens = 192;
constexpr int32_t kBackSlice = 1024;

inline bool f32_or_bf16(mxq_out_dtype d) {
  return d == MXQ_OUT_BF16 || d == MXQ_OUT_F32;
}

inline bool row_ok(const void* p, int64_t ld, int64_t H, int64_t esz) {
  return p != nullptr && ld >= H && aligned16(p) && (ld * esz) % 16 == 0;
}

}  // namespace

extern "C" mxq_status moe_scatter_rows_backward(
    const void* grad_rows, mxq_out_dtype rows_dtype, int64_t ld_rows,
    int64_t num_rows, const int32_t* src2dst, int64_t T, int32_t K, int32_t H,
    void* grad_x, int64_t ld_x, mxq_out_dtype x_dtype, void* stream) {
  if (!f32_or_bf16(rows_dtype) || !f32_or_bf16(x_dtype))
    return MXQ_ERR_UNSUPPORTED;
  if (T < 0 || T > INT32_MAX || K < 0 || K > MXQ_MAX_TOPK || H <= 0 ||
      H % 8 != 0 || num_rows < 0 || num_rows > INT32_MAX)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (T == 0) return MXQ_OK;
  const int64_t in = rows_dtype == MXQ_OUT_F32 ? 4 : 2;
  const int64_t on = x_dtype == MXQ_OUT_F32 ? 4 : 2;
  if (!row_ok(grad_x, ld_x, H, on) || (K > 0 && src2dst == nullptr) ||
      (num_rows > 0 && !row_ok(grad_rows, ld_rows, H, in)))
    return MXQ_ERR_INVALID_ARGUMENT;
  int32_t slice = H;
  if (T <= kBackSliceMaxTokens && H > kBackSlice)
    slice = (int32_t)std::max<int64_t>(
        kBackSlice, ceil_div(ceil_div(H, 65535), 8) * 8);
  const int threads = row_block_threads(slice, 8);
  const int64_t most = max_blocks(threads);  // tokens of a launch
  hipStream_t s = as_stream(stream);
  const char* r = static_cast<const char*>(grad_rows);
  char* o = static_cast<char*>(grad_x);
  auto go = [&](auto fin, auto fout) {
    for (int64_t t = 0; t < T; t += most)
      scatter_rows_backward_kernel<decltype(fin)::value,
                                   decltype(fout)::value>
          <<<dim3((unsigned)std::min(most, T - t),
                  (unsigned)ceil_div(H, slice)),
             threads, 0, s>>>(r, ld_rows, num_rows, src2dst + t * K, K, H,
                              slice, o + t * ld_x * on, ld_x);
  };
  using Y = std::true_type;
  using N = std::false_type;
  if (in == 4)
    on == 4 ? go(Y{}, Y{}) : go(Y{}, N{});
  else
    on == 4 ? go(N{}, Y{}) : go(N{}, N{});
  return launch_status();
}

extern "C" mxq_status moe_combine_backward(
    const void* grad_out, mxq_out_dtype grad_dtype, int64_t ld_g,
    const void* y_bf16, int64_t ld_y, int64_t num_rows,
    const int32_t* src2dst, const float* topk_weights, int64_t T, int32_t K,
    int32_t H, void* grad_y_bf16, int64_t ld_gy, float* grad_weights,
    void* stream) {
  if (!f32_or_bf16(grad_dtype)) return MXQ_ERR_UNSUPPORTED;
  if (T < 0 || T > INT32_MAX || K < 0 || K > MXQ_MAX_TOPK || H <= 0 ||
      H % 8 != 0 || num_rows < 0 || num_rows > INT32_MAX)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (H > MXQ_MAX_HIDDEN) return MXQ_ERR_UNSUPPORTED;
  if (grad_y_bf16 == nullptr && grad_weights == nullptr)
    return MXQ_ERR_INVALID_ARGUMENT;
  if (T == 0 || K == 0) return MXQ_OK;
  const int64_t esz = grad_dtype == MXQ_OUT_F32 ? 4 : 2;
  if (src2dst == nullptr || !row_ok(grad_out, ld_g, H, esz))
    return MXQ_ERR_INVALID_ARGUMENT;
  const bool need_y = grad_y_bf16 != nullptr;
  const bool need_w = grad_weights != nullptr;
  if (num_rows > 0) {
    if (need_y && (topk_weights == nullptr ||
                   !row_ok(grad_y_bf16, ld_gy, H, 2)))
      return MXQ_ERR_INVALID_ARGUMENT;
    if (need_w && !row_ok(y_bf16, ld_y, H, 2))
      return MXQ_ERR_INVALID_ARGUMENT;
  }
  if (need_y && topk_weights == nullptr) return MXQ_ERR_INVALID_ARGUMENT;
  const size_t lds = (size_t)(H * esz);
  hipStream_t s = as_stream(stream);
  auto go = [&](auto f32, auto ny, auto nw) -> mxq_status {
    auto* k = &combine_backward_kernel<decltype(f32)::value,
                                       decltype(ny)::value,
                                       decltype(nw)::value>;
    // more than 64 KB, with the joined sums, needs the kernel's limit raised
    if (lds + kCombineBackWaves * sizeof(float) > 65536 &&
        hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                            hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)lds) != hipSuccess) {
      (void)hipGetLastError();
      return MXQ_ERR_HIP;
    }
    const int64_t most = max_blocks(kCombineBackThreads);  // of a launch
    for (int64_t t = 0; t < T; t += most)
      k<<<(unsigned)std::min(most, T - t), kCombineBackThreads, lds, s>>>(
          static_cast<const char*>(grad_out) + t * ld_g * esz, ld_g,
          static_cast<const uint16_t*>(y_bf16), ld_y, num_rows,
          src2dst + t * K, need_y ? topk_weights + t * K : nullptr, K, H,
          static_cast<uint16_t*>(grad_y_bf16), ld_gy,
          need_w ? grad_weights + t * K : nullptr);
    return launch_status();
  };
  using Y = std::true_type;
  using N = std::false_type;
  if (esz == 4) {
    if (need_y && need_w) return go(Y{}, Y{}, Y{});
    return need_y ? go(Y{}, Y{}, N{}) : go(Y{}, N{}, Y{});
  }
  if (need_y && need_w) return go(N{}, Y{}, Y{});
  return need_y ? go(N{}, Y{}, N{}) : go(N{}, N{}, Y{});
}
