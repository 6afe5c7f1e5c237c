// quantize_dev.hpp -- values to 8-bit codes: a row's scale is s = max(amax / 127, 2^-126) in fp32, its codes q = rint(x / s),
// the real quotient to the nearest integer, ties to even.
//
// The quotient comes from a product with 1 / s, which is off by less than 127 (2^-24 + 2^-24) < 2^-15, so q is certain
// unless the product lies that close to a border between two integers.  There x - q s is compared with s / 2, which a
// fused multiply-add does exactly: for |q| > 1 the difference is a multiple of s's last place and no larger than about
// s / 2, so it fits 24 bits; for |q| <= 1 it is x itself, or one whose rounding to s / 2 leads to the same even code.
#pragma once

#include "wave_dev.hpp"

namespace moe {

constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126, fp32's smallest normal value: s and s / 2 stay exact

struct RowScale {
  float s, inv, half;
};
// From the largest magnitude of a row as bits, which order as unsigned integers with infinity and NaN on top.  A row
// that holds one of those has scale NaN; its codes are 0 (the callers see to that), so all that comes of it is NaN.
__device__ __forceinline__ bool finite_bits(uint32_t amax) { return amax < 0x7F800000u; }
__device__ __forceinline__ RowScale row_scale(uint32_t amax) {
  RowScale r;
  r.s = finite_bits(amax) ? fmaxf(__uint_as_float(amax) / 127.0f, kLeastScale) : __uint_as_float(0x7FC00000u);
  r.inv = finite_bits(amax) ? 1.0f / r.s : 0.0f;
  r.half = 0.5f * r.s;
  return r;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
// Maximum over the wave, in every lane (as wave_all does for floats).
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp_u32<0x111, 0xF>(v));
  v = max(v, dpp_u32<0x112, 0xF>(v));
  v = max(v, dpp_u32<0x114, 0xF>(v));
  v = max(v, dpp_u32<0x118, 0xF>(v));
  v = max(v, dpp_u32<0x142, 0xA>(v));
  v = max(v, dpp_u32<0x143, 0xC>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Adding 1.5 * 2^23 rounds to an integer, whose low byte is then the sum's.
constexpr float kRound = 12582912.0f, kNear = 0.5f - 0x1p-15f;

// The sum's bits moved to the right code where the product with 1 / s cannot tell.
__device__ __forceinline__ uint32_t settle(float x, uint32_t bits, const RowScale& r) {
  const float q = __uint_as_float(bits) - kRound;
  const float d = __builtin_fmaf(-q, r.s, x);
  const bool move = fabsf(d) > r.half || (fabsf(d) == r.half && (bits & 1));
  return move ? bits + (d > 0.0f ? 1 : -1) : bits;
}

// Eight values to eight codes.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], const RowScale& r) {
  uint32_t b[8];
  float worst = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = x[i] * r.inv, t = v + kRound;
    b[i] = __float_as_uint(t);
    worst = fmaxf(worst, fabsf(v - (t - kRound)));
  }
  if (worst > kNear) {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = settle(x[i], b[i], r);
  }
  auto pack = [&](int i) {
    const uint32_t lo = __builtin_amdgcn_perm(b[i + 1], b[i], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[i + 3], b[i + 2], 0x0C0C0400u);
    return lo | hi << 16;
  };
  return make_uint2(pack(0), pack(4));
}

// Eight consecutive values, `i` a multiple of 8 elements from a 16-byte boundary.
template <bool F32>
struct Eight;
template <>
struct Eight<false> {
  uint4 q;
  __device__ __forceinline__ void load(const void* x, size_t i) {
    q = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + i);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Eight<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* x, size_t i) {
    a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + i);
    b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + i + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <bool F32>
__device__ __forceinline__ uint32_t amax_bits(const Eight<F32>& e) {
  float v[8];
  e.get(v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

}  // namespace moe
