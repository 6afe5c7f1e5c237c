// combine_grad.hip -- gradient of the weighted combine out_t = residual_t + sum_j w_tj y_tj:
//   dw_tj = sum_c dout_tc y_tjc      dy_tjc = w_tj dout_tc      (the residual's gradient is dout itself)
//
// One pass: a token's dout is read once into registers and meets each of its k rows of y, whose loads are all issued
// before the first product; dy is written from the same registers.  HBM bounds it: T k H (read + write) elements.
// Sums in fp32, over columns in an order that depends on H alone, so a token's dw does not depend on its neighbours
// and two calls give the same bits.
#include <algorithm>
#include <type_traits>

#include "wave_dev.hpp"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int C>
struct Cols {
  float v[C];
};
// C consecutive columns (C = 4 or 8) of an fp32 or bf16 row, kept as loaded until they are used.
template <typename T, int C>
struct Raw {
  static constexpr int kWords = C * (int)sizeof(T) / 4;
  uint32_t w[kWords];
};
template <typename T, int C>
__device__ __forceinline__ Raw<T, C> load_raw(const T* p) {
  Raw<T, C> r;
  if constexpr (Raw<T, C>::kWords == 2) {
    const u32x2 q = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    r.w[0] = q.x; r.w[1] = q.y;
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T, C>::kWords; i += 4) {
      const u32x4 q = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p) + i / 4);
      r.w[i] = q.x; r.w[i + 1] = q.y; r.w[i + 2] = q.z; r.w[i + 3] = q.w;
    }
  }
  return r;
}
template <typename T, int C>
__device__ __forceinline__ Cols<C> widen(const Raw<T, C>& r) {
  Cols<C> o;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if constexpr (sizeof(T) == 4) o.v[i] = __uint_as_float(r.w[i]);
    else o.v[i] = __uint_as_float(i & 1 ? r.w[i / 2] & 0xFFFF0000u : r.w[i / 2] << 16);
  }
  return o;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __bf16 x = (__bf16)a, y = (__bf16)b;
  return (uint32_t)__builtin_bit_cast(uint16_t, x) | (uint32_t)__builtin_bit_cast(uint16_t, y) << 16;
}
template <int C>
__device__ __forceinline__ void store_cols(float* p, const Cols<C>& v) {
#pragma unroll
  for (int i = 0; i < C; i += 4)
    reinterpret_cast<float4*>(p)[i / 4] = make_float4(v.v[i], v.v[i + 1], v.v[i + 2], v.v[i + 3]);
}
template <int C>
__device__ __forceinline__ void store_cols(uint16_t* p, const Cols<C>& v) {
  if constexpr (C == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v.v[0], v.v[1]), pack_bf16(v.v[2], v.v[3]),
                                              pack_bf16(v.v[4], v.v[5]), pack_bf16(v.v[6], v.v[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v.v[0], v.v[1]), pack_bf16(v.v[2], v.v[3]));
}

constexpr int kThreads = 256;

// Grid: (tokens, k / J rounded up, T / tokens rounded up), as one dimension holds less than 2^32 threads; workgroup
// (t, b) takes rows b J ... of token t.  Thread i owns columns C i ... of each 256 C-column stretch.
template <typename YT, typename GT, int C, int J>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(const YT* __restrict__ y, const float* __restrict__ w,
                                                                    const GT* __restrict__ dout, int T, int k, int H,
                                                                    float* __restrict__ dw, YT* __restrict__ dy) {
  __shared__ float s_dot[kThreads / 64][J];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const size_t t = (size_t)blockIdx.z * gridDim.x + blockIdx.x;
  if (t >= (size_t)T) return;
  const int j0 = blockIdx.y * J, nj = min(J, k - j0);
  const size_t row0 = t * k + j0;
  float wj[J], dot[J];
#pragma unroll
  for (int j = 0; j < J; ++j) wj[j] = dot[j] = 0.0f;
  if (dy) {  // (w may be null without dy)
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (j < nj) wj[j] = w[row0 + j];
  }
  for (int c = tid * C; c < H; c += kThreads * C) {
    Raw<YT, C> rows[J];
    const Raw<GT, C> graw = load_raw<GT, C>(dout + t * H + c);
    if (dw) {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (j < nj) rows[j] = load_raw<YT, C>(y + (row0 + j) * H + c);
    }
    const Cols<C> g = widen<GT, C>(graw);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (j >= nj) continue;
      if (dy) {
        Cols<C> o;
#pragma unroll
        for (int i = 0; i < C; ++i) o.v[i] = wj[j] * g.v[i];
        store_cols<C>(dy + (row0 + j) * H + c, o);
      }
      if (dw) {
        const Cols<C> v = widen<YT, C>(rows[j]);
#pragma unroll
        for (int i = 0; i < C; ++i) dot[j] = __builtin_fmaf(g.v[i], v.v[i], dot[j]);
      }
    }
  }
  if (!dw) return;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float v = wave_sum(dot[j]);
    if (lane == 0) s_dot[wave][j] = v;
  }
  __syncthreads();
  if (tid < nj) {
    float v = s_dot[0][tid];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) v += s_dot[i][tid];
    dw[row0 + tid] = v;
  }
}

// Rows of a token per workgroup: all of them, so that dout is read once, unless the tokens are too few to fill the card
// (12 tokens of 10 x 2,048 fp32: 9.4 us with 10 rows, 3.4 with 2).
template <typename YT, typename GT, int C>
void launch_c(const YT* y, const float* w, const GT* dout, int T, int k, int H, float* dw, YT* dy, hipStream_t s) {
  constexpr int kTokens = 1 << 22;
  auto go = [&](auto kernel, int rows) {
    const dim3 grid((unsigned)std::min(T, kTokens), (unsigned)ceil_div(k, rows), (unsigned)ceil_div(T, kTokens));
    launch_k(MOE_KERNEL_COMBINE_BACKWARD, kernel, grid, dim3(kThreads), 0, s, y, w, dout, T, k, H, dw, dy);
  };
  if (T < 256 && k > 2) go(combine_backward_kernel<YT, GT, C, 2>, 2);
  else if (k > 8) go(combine_backward_kernel<YT, GT, C, kMaxK>, kMaxK);
  else go(combine_backward_kernel<YT, GT, C, 8>, 8);
}

template <typename YT, typename GT>
void launch_t(const void* y, const float* w, const void* dout, int T, int k, int H, float* dw, void* dy,
              hipStream_t s) {
  auto go = [&](auto c) {
    launch_c<YT, GT, decltype(c)::value>((const YT*)y, w, (const GT*)dout, T, k, H, dw, (YT*)dy, s);
  };
  if (H % 8 == 0) go(std::integral_constant<int, 8>{});
  else go(std::integral_constant<int, 4>{});
}

}  // namespace

moe_status launch_combine_backward(const void* y, moe_dtype y_t, const float* w, const void* dout, moe_dtype dout_t,
                                   int T, int k, int H, float* dw, void* dy, hipStream_t s) {
  if (y_t == MOE_BF16)
    dout_t == MOE_BF16 ? launch_t<uint16_t, uint16_t>(y, w, dout, T, k, H, dw, dy, s)
                       : launch_t<uint16_t, float>(y, w, dout, T, k, H, dw, dy, s);
  else
    dout_t == MOE_BF16 ? launch_t<float, uint16_t>(y, w, dout, T, k, H, dw, dy, s)
                       : launch_t<float, float>(y, w, dout, T, k, H, dw, dy, s);
  return check_launch("combine_backward");
}

}  // namespace moe
