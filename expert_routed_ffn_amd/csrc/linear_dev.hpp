// linear_dev.hpp -- device pieces shared by the dense product and its gradient: bf16 conversions, activations, the
// epilogue, and the description of one product for the tiled kernel.
#pragma once

#include "internal.hpp"

namespace moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  return (uint32_t)f32_to_bf16(a) | (uint32_t)f32_to_bf16(b) << 16;
}

// An fp32 value as a sum of up to three bf16 terms, each the nearest bf16 of what is left: 8 + 8 + 8 significant bits,
// so three terms hold every finite value of normal size exactly and two hold 16 to 17 bits.  A value that rounds
// past the largest bf16 is cut instead; infinities and NaN stand in the first term alone.
__device__ __forceinline__ void bf16_terms(float f, uint16_t (&t)[3]) {
  uint16_t h = f32_to_bf16(f);
  const bool finite = (__float_as_uint(f) & 0x7F800000u) != 0x7F800000u;
  if (finite && (h & 0x7F80u) == 0x7F80u) h = (uint16_t)(__float_as_uint(f) >> 16);
  t[0] = h;
  const float r = finite ? f - bf16_to_f32(h) : 0.0f;
  t[1] = f32_to_bf16(r);
  t[2] = f32_to_bf16(r - bf16_to_f32(t[1]));
}

// Two values as TERMS packed bf16 terms each, for uses that take all of them: what does not fit a term, infinities and NaN
// included, is left to the next (no term but the last exceeds the largest bf16), which costs fewer steps than testing
// for them.
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
template <int TERMS>
__device__ __forceinline__ void split_terms(float a, float b, uint32_t (&t)[TERMS]) {
  constexpr float kMax = 3.38953139e38f;  // 0x7F7F0000
#pragma unroll
  for (int k = 0; k < TERMS; ++k) {
    f32x2_t v = {a, b};
    if (k < TERMS - 1) v = f32x2_t{__builtin_amdgcn_fmed3f(a, -kMax, kMax), __builtin_amdgcn_fmed3f(b, -kMax, kMax)};
    t[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
    a -= __uint_as_float(t[k] << 16);
    b -= __uint_as_float(t[k] & 0xFFFF0000u);
  }
}
// Four values at x + 4 i to the term planes, `plane` elements apart.
template <int TERMS>
__device__ __forceinline__ void write_terms(const float* x, int64_t i, uint16_t* planes, int64_t plane) {
  const float4 q = reinterpret_cast<const float4*>(x)[i];
  uint32_t lo[TERMS], hi[TERMS];
  split_terms<TERMS>(q.x, q.y, lo);
  split_terms<TERMS>(q.z, q.w, hi);
#pragma unroll
  for (int k = 0; k < TERMS; ++k) reinterpret_cast<uint2*>(planes + k * plane)[i] = make_uint2(lo[k], hi[k]);
}

// 1 / (1 + e^-z): z -> -inf gives 0, z -> inf gives 1, NaN stays NaN.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}
// tanh form of GELU: z (1 + tanh(v)) / 2 = z sigmoid(2 v), v = sqrt(2/pi) (z + 0.044715 z^3).
constexpr float kGeluA2 = 1.59576912f, kGeluB = 0.044715f;  // 2 sqrt(2/pi)
__device__ __forceinline__ float gelu_gate(float z) {
  return sigmoid(kGeluA2 * z * __builtin_fmaf(kGeluB * z, z, 1.0f));
}
__device__ __forceinline__ float act_value(int act, float z) {
  if (act == MOE_ACT_GELU) return z * gelu_gate(z);
  if (act == MOE_ACT_SILU) return z * sigmoid(z);
  return z;
}
__device__ __forceinline__ float act_slope(int act, float z) {
  if (act == MOE_ACT_GELU) {
    // From |z| = 32 on h is 0 or 1 and the slope is h; z^2 is kept from growing past fp32's range there, as 0 times an
    // infinity is NaN (a NaN z stays one through h).
    const float h = gelu_gate(z), c = __builtin_amdgcn_fmed3f(z, -32.0f, 32.0f);
    return __builtin_fmaf(c * h * (1.0f - h), kGeluA2 * __builtin_fmaf(3.0f * kGeluB * c, c, 1.0f), h);
  }
  if (act == MOE_ACT_SILU) {
    const float h = sigmoid(z);
    return h * __builtin_fmaf(z, 1.0f - h, 1.0f);
  }
  return 1.0f;
}

// Four or eight consecutive elements of a row at any element boundary: global memory takes 8- and 16-byte accesses at
// addresses that are only aligned to their elements, so rows of odd length cost no more than others.  (Element by
// element, an 8,192 x 1,001 result took 66 us against 44 with 1,000 columns, and its gradient's first launch 47 against
// 20.)
typedef uint32_t u32x2_at2_t __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_at2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_at4_t __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ void load4(const void* p, int bf16, size_t i, float (&v)[4]) {
  if (bf16) {
    const u32x2_at2_t q = *reinterpret_cast<const u32x2_at2_t*>(reinterpret_cast<const uint16_t*>(p) + i);
    v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xFFFF0000u);
    v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xFFFF0000u);
  } else {
    const u32x4_at4_t q = *reinterpret_cast<const u32x4_at4_t*>(reinterpret_cast<const float*>(p) + i);
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y); v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
  }
}
__device__ __forceinline__ void store4(void* p, int bf16, size_t i, const float (&v)[4]) {
  if (bf16)
    *reinterpret_cast<u32x2_at2_t*>(reinterpret_cast<uint16_t*>(p) + i) =
        u32x2_at2_t{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])};
  else
    *reinterpret_cast<u32x4_at4_t*>(reinterpret_cast<float*>(p) + i) =
        u32x4_at4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
}

// What becomes of an element z of the product: y = act(z + bias) + residual, z + bias kept in `pre`.
struct Epi {
  const float* bias;  // [R] or null
  const void* res;    // [M x N] or null
  void* y;            // [M x N]
  void* pre;          // [M x R] of y's type, or null
  int N, R;           // output columns; product columns (2 N for SwiGLU, else N)
  int act;
  int res_bf16, y_bf16;
};

__device__ __forceinline__ float load_any(const void* p, int bf16, size_t i) {
  return bf16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_any(void* p, int bf16, size_t i, float v) {
  if (bf16) reinterpret_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
  else reinterpret_cast<float*>(p)[i] = v;
}
// What the epilogue of one element reads, so that it can be read before the product is there.
struct EpiIn {
  float b = 0.0f, bu = 0.0f, res = 0.0f;
};
__device__ __forceinline__ EpiIn epi_in(const Epi& e, int m, int n) {
  EpiIn in;
  if (e.bias) {
    in.b = e.bias[n];
    if (e.act == MOE_ACT_SWIGLU) in.bu = e.bias[e.N + n];
  }
  if (e.res) in.res = load_any(e.res, e.res_bf16, (size_t)m * e.N + n);
  return in;
}
// One element; zu is the up value of a SwiGLU pair.
__device__ __forceinline__ void epi_one(const Epi& e, int m, int n, float z, float zu, const EpiIn& in) {
  const bool pair = e.act == MOE_ACT_SWIGLU;
  z += in.b;
  zu += in.bu;
  if (e.pre) {
    store_any(e.pre, e.y_bf16, (size_t)m * e.R + n, z);
    if (pair) store_any(e.pre, e.y_bf16, (size_t)m * e.R + e.N + n, zu);
  }
  float v = pair ? z * sigmoid(z) * zu : act_value(e.act, z);
  const size_t i = (size_t)m * e.N + n;
  v += in.res;
  store_any(e.y, e.y_bf16, i, v);
}
// Columns n .. n + 3 (n < N; those past N are left out) of rows m, m + STEP, ...: `rows` rows from m on, whose products
// value(d, z, zu) gives for row m + d.  Addresses advance by a constant and the flags are the same for all threads, so
// what a row costs is its loads, its stores and the activation; residuals of four rows are read ahead.  (With addresses
// computed for each row, 64-bit products among them, the epilogue of an 8,192 x 1,024 result took 9 us longer.)
template <bool PAIR, int STEP, int ACT, typename Value>
__device__ __forceinline__ void epi_rows_act(const Epi& e, int m, int n, int rows, Value value) {
  float b[4] = {0.f, 0.f, 0.f, 0.f}, bu[4] = {0.f, 0.f, 0.f, 0.f};
  if (e.bias) {
    load4(e.bias, 0, n, b);
    if constexpr (PAIR) load4(e.bias, 0, (size_t)e.N + n, bu);
  }
  size_t i = (size_t)m * e.N + n, ip = (size_t)m * e.R + n;
  const size_t di = (size_t)STEP * e.N, dp = (size_t)STEP * e.R;
  for (int d = 0; d < rows; d += 4 * STEP) {
    float res[4][4] = {};
    if (e.res) {  // (rows past the last read the first of the four: a load under a condition is waited for at its end)
      size_t at[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) at[k] = i + (d + k * STEP < rows ? k * di : 0);
      if (e.res_bf16) {
#pragma unroll
        for (int k = 0; k < 4; ++k) load4(e.res, 1, at[k], res[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) load4(e.res, 0, at[k], res[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (d + k * STEP < rows) {
        float z[4], zu[4], v[4];
        value(d + k * STEP, z, zu);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          z[r] += b[r];
          if constexpr (PAIR) zu[r] += bu[r];
        }
        if (e.pre) {
          store4(e.pre, e.y_bf16, ip, z);
          if constexpr (PAIR) store4(e.pre, e.y_bf16, ip + e.N, zu);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (PAIR) v[r] = z[r] * sigmoid(z[r]) * zu[r];
          else v[r] = act_value(ACT, z[r]);
          v[r] += res[k][r];
        }
        store4(e.y, e.y_bf16, i, v);
      }
      i += di;
      ip += dp;
    }
  }
}
template <bool PAIR, int STEP, typename Value>
__device__ __forceinline__ void epi_rows(const Epi& e, int m, int n, int rows, Value value) {
  if (n + 4 > e.N) {  // the last columns of rows whose length is no multiple of 4
    for (int d = 0; d < rows; d += STEP) {
      float z[4], zu[4] = {0.f, 0.f, 0.f, 0.f};
      value(d, z, zu);
#pragma unroll
      for (int r = 0; r < 3; ++r)
        if (n + r < e.N) epi_one(e, m + d, n + r, z[r], zu[r], epi_in(e, m + d, n + r));
    }
  } else if (PAIR) {
    epi_rows_act<PAIR, STEP, MOE_ACT_SWIGLU>(e, m, n, rows, value);
  } else if (e.act == MOE_ACT_GELU) {
    epi_rows_act<PAIR, STEP, MOE_ACT_GELU>(e, m, n, rows, value);
  } else if (e.act == MOE_ACT_SILU) {
    epi_rows_act<PAIR, STEP, MOE_ACT_SILU>(e, m, n, rows, value);
  } else {
    epi_rows_act<PAIR, STEP, MOE_ACT_NONE>(e, m, n, rows, value);
  }
}

// One product C[m][n] = sum over segments and k of A(m, k) B(n, k); which operand lies [index][k] and which [k][index]
// is the kernel's.  A segment names one term plane of each operand (see bf16_terms): planes are `a_plane` / `b_plane`
// elements apart.
struct Prob {
  const uint16_t *A, *B;
  int64_t a_plane, b_plane;
  int lda, ldb;            // elements per stored row, multiples of 8
  int M, R, K;             // C is M x R, K the reduction (a multiple of 8 where an operand is [index][k])
  int nseg;                // of a plan of kDirect 1
  int terms;               // kDirect: A is fp32 and enters as so many bf16 terms
  uint32_t sa, sb;         // two bits per segment: its plane of A and of B
  int split;               // parts of the reduction, each a workgroup
  float* partial;          // [split][M][ldp] when split > 1
  int ldp;                 // elements per row of a part
  Epi epi;
};
struct DbSum {  // column sums of dz from the parts that the prep launch left; db null: not wanted
  const float* part;  // [rows][n]
  float* db;          // [n]
  int rows, n;
};
struct Join {  // sums of the parts of up to two products, or db's
  Prob p[2];
  int n0, n1;  // workgroups of each product (0: not split)
  DbSum db;
};

// Sizes of a product, and how a launch of up to two cuts them.
struct Shape {
  int M, R, K, nseg;
  bool f32;      // A is fp32 in memory, its terms the segments: kDirect may split it as it reads it
  int turns;     // launches that its term planes take otherwise, each with its share of the rows
};
constexpr int kDirect = 3;
struct Plan {
  int shape;     // 64, 128 or 256 squared tiles, or (kDirect) 64 squared ones of fp32 A
  int split[2];
};
Plan plan_products(const Shape* s, int count);
int tile_side(const Plan& plan);
// Launches a forward product (`grad` false, count = 1) or the gradient's (dW first where both are there) with db's sum,
// then what joins the products' parts.
moe_status launch_products(int kid, const Plan& plan, Prob* p, int count, bool grad, bool first_is_dw, const DbSum& db,
                           hipStream_t s, const char* what);

}  // namespace moe
