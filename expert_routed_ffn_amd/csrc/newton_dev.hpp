// newton_dev.hpp -- what the two ways to an orthogonalised update share (orthogonalize.hip, orthogonalize_small.hip).
#pragma once

#include "linear_dev.hpp"

namespace moe {

struct Update {
  const void* g;
  float* moment;  // null: the update is g
  int g_bf16, nesterov;
  float beta, rest;  // rest = 1 - beta
  int R, K;
};

// u from g and the moment after this step.
__device__ __forceinline__ float update_of(const Update& u, float g, float m) {
  return !u.moment ? g : u.nesterov ? __builtin_fmaf(u.beta, m, u.rest * g) : m;
}

// 1 / (norm + eps) from the sum of squares (which are 0 in 64 bits for zeros alone): 0 for a zero matrix, which stays zero
// however small eps is, and NaN for one with an infinity or a NaN, which becomes NaN throughout.
__device__ __forceinline__ double inverse_norm(double squares, double eps) {
  const double total = sqrt(squares) + eps;
  return squares == 0.0 ? 0.0 : total < __builtin_huge_val() ? 1.0 / total : __builtin_nan("");
}

// Four values of u from row r, column k on; zeros past the matrix.  MOMENT: the moment is brought up to date on the way.
template <bool MOMENT>
__device__ __forceinline__ void load_update(const Update& u, int64_t base, int r, int k, float (&v)[4]) {
  float g[4] = {0.f, 0.f, 0.f, 0.f}, m[4] = {0.f, 0.f, 0.f, 0.f};
  const int64_t i = base + (int64_t)r * u.K + k;
  if (r < u.R && k + 4 <= u.K) {
    load4(u.g, u.g_bf16, i, g);
    if (u.moment) {
      load4(u.moment, 0, i, m);
      if constexpr (MOMENT) {
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = __builtin_fmaf(u.beta, m[e], u.rest * g[e]);
        store4(u.moment, 0, i, m);
      }
    }
  } else if (r < u.R) {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (k + e < u.K) {
        g[e] = load_any(u.g, u.g_bf16, i + e);
        if (u.moment) {
          m[e] = u.moment[i + e];
          if constexpr (MOMENT) u.moment[i + e] = m[e] = __builtin_fmaf(u.beta, m[e], u.rest * g[e]);
        }
      }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = update_of(u, g[e], m[e]);
}

// Matrices whose shorter side is at most 64: see orthogonalize_small.hip.
bool newton_is_small(int R, int K, int steps, const float* coef);
size_t newton_small_ws_bytes(int B, int R, int K);
moe_status launch_newton_small(const Update& u, int B, int steps, const float* coef, double eps, void* o, moe_dtype o_t,
                               void* ws, hipStream_t s);

}  // namespace moe
