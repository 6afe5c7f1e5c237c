// wave_dev.hpp -- sums and maxima over a wave on the vector ALU.
#pragma once

#include "internal.hpp"

namespace moe {

constexpr float kNegInf = -__builtin_huge_valf();

// Sum or maximum over the wave, in every lane: four shifts within rows of 16 lanes, two broadcasts across rows, all on
// the vector ALU (butterflies through LDS took the loss of an 8,192 x 512 chunk 18.6 us, these 7).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v, float other) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(other), __float_as_uint(v), CTRL, ROWS, 0xF, false));
}
template <typename Op>
__device__ __forceinline__ float wave_all(float v, float unit, Op op) {
  v = op(v, dpp<0x111, 0xF>(v, unit));  // row_shr:1
  v = op(v, dpp<0x112, 0xF>(v, unit));
  v = op(v, dpp<0x114, 0xF>(v, unit));
  v = op(v, dpp<0x118, 0xF>(v, unit));
  v = op(v, dpp<0x142, 0xA>(v, unit));  // lane 15 of rows 0 and 2 to rows 1 and 3
  v = op(v, dpp<0x143, 0xC>(v, unit));  // lane 31 to rows 2 and 3
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_all(v, 0.0f, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_all(v, kNegInf, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace moe
