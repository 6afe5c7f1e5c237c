// linear.hip -- dense product with bias, activation and residual in its epilogue:
//   z = x W^T + b,  y = act(z) + residual,  SwiGLU: y = silu(z_gate) z_up + residual with W's first N rows the gate.
//
// Up to 64 tokens: linear_few_kernel, weights straight from memory into matrix operands, the reduction split over the
// waves of a workgroup.  More: the tiled product of product.hip.  Sums in fp32.  fp32 activations enter
// as bf16 terms (split_terms in linear_dev.hpp): three, which hold them exactly, when y is fp32 or the tokens are few; two,
// which leave at most 2^-17 of each value (2^-9 of the half step that y's rounding costs), when y is bf16 and the product is
// tiled.  (One term there was off by up to 2^-8 of each value, as much again as y's rounding, and gave a token another
// value in a batch of more than 64.)
#include <algorithm>

#include "linear_dev.hpp"

namespace moe {
namespace {

// ---- up to 64 tokens --------------------------------------------------------------------

constexpr int kFewT = 64, kFewWaves = 8;

template <bool XF32>
struct FewX;  // 8 consecutive activations of one token
template <>
struct FewX<false> {
  uint4 q;
  __device__ __forceinline__ void load(const void* x, size_t i) {
    q = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + i);
  }
  __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
};
template <>
struct FewX<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* x, size_t i) {
    a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + i);
    b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + i + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
};

// Grid: one workgroup per 16 rows of W (8 gate and 8 up rows for SwiGLU), 8 waves.  v_mfma_f32_16x16x32_bf16 takes
// the 16 rows as its first operand and 16 tokens as its second; TF such token fragments share each weight fragment.
// Wave w works through its eighth of the K-steps with the loads of U steps in flight, then the eight sums of an element
// are added through LDS in wave order.  fp32 activations are split as they are used; the steps of that are many, and the
// code of more than a few of them costs more than it saves (2,048 -> 1,024 from one fp32 token: 7.8 us with four steps
// unrolled and a split that tests for infinities, 4.9 with this one).  Rows of W past R and tokens past T read the last
// valid one and are not stored.
template <bool XF32, int TF>
__global__ __launch_bounds__(64 * kFewWaves) void linear_few_kernel(const void* __restrict__ x,
                                                                    const uint16_t* __restrict__ w, int T, int K, Epi e) {
  constexpr int U = XF32 ? (TF == 1 ? 2 : 1) : TF == 4 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) float red[kFewWaves][TF][64][4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool pair = e.act == MOE_ACT_SWIGLU;
  const int fr = lane & 15, fq = lane >> 4;
  int row;
  if (pair) {
    row = min((int)blockIdx.x * 8 + (fr & 7), e.N - 1) + (fr >= 8 ? e.N : 0);
  } else {
    row = min((int)blockIdx.x * 16 + fr, e.N - 1);
  }
  const uint16_t* wrow = w + (size_t)row * K + fq * 8;
  size_t xoff[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) xoff[f] = (size_t)min(16 * f + fr, T - 1) * K + fq * 8;

  // The results this thread will finish, with their bias and residual, which are read here beside the first weights.
  constexpr int kElems = (TF * 256 + 64 * kFewWaves - 1) / (64 * kFewWaves);
  struct {
    int t, n, r;  // t < 0: none
    EpiIn in;
  } el[kElems];
#pragma unroll
  for (int i = 0; i < kElems; ++i) {
    const int at = i * 64 * kFewWaves + threadIdx.x;
    el[i].r = at & 15;
    el[i].n = blockIdx.x * (pair ? 8 : 16) + el[i].r;
    const bool has = at < TF * 256 && at >> 4 < T && el[i].n < e.N && !(pair && el[i].r >= 8);
    el[i].t = has ? at >> 4 : -1;
    if (has) el[i].in = epi_in(e, el[i].t, el[i].n);
  }

  f32x4_t acc[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int steps = K / 32;
  const int s0 = steps * wave / kFewWaves, s1 = steps * (wave + 1) / kFewWaves;
  struct Stage {
    uint4 w[U];
    FewX<XF32> x[U][TF];
  };
  auto load = [&](Stage& st, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u < s1) {
        st.w[u] = *reinterpret_cast<const uint4*>(wrow + (s + u) * 32);
#pragma unroll
        for (int f = 0; f < TF; ++f) st.x[u][f].load(x, xoff[f] + (size_t)(s + u) * 32);
      } else {
        st.w[u] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int f = 0; f < TF; ++f) st.x[u][f].zero();
      }
    }
  };
  auto multiply = [&](const Stage& st) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bf16x8_t wf = __builtin_bit_cast(bf16x8_t, st.w[u]);
#pragma unroll
      for (int f = 0; f < TF; ++f) {
        if constexpr (XF32) {
          const float4 a = st.x[u][f].a, b = st.x[u][f].b;
          uint32_t t[4][3];
          split_terms<3>(a.x, a.y, t[0]);
          split_terms<3>(a.z, a.w, t[1]);
          split_terms<3>(b.x, b.y, t[2]);
          split_terms<3>(b.z, b.w, t[3]);
#pragma unroll
          for (int q = 0; q < 3; ++q)
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                wf, __builtin_bit_cast(bf16x8_t, make_uint4(t[0][q], t[1][q], t[2][q], t[3][q])), acc[f], 0, 0, 0);
        } else {
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8_t, st.x[u][f].q), acc[f], 0, 0, 0);
        }
      }
    }
  };
  for (int s = s0; s < s1; s += U) {
    Stage st;
    load(st, s);
    multiply(st);
  }
  // lane: token 16 f + (lane & 15), rows 4 (lane >> 4) + r
#pragma unroll
  for (int f = 0; f < TF; ++f)
    *reinterpret_cast<f32x4_t*>(red[wave][f][lane]) = acc[f];
  __syncthreads();
  auto total = [&](int f, int r, int tk) {  // row r of the workgroup's 16, token tk of fragment f
    const int l = 16 * (r >> 2) + tk;
    float v = red[0][f][l][r & 3];
#pragma unroll
    for (int i = 1; i < kFewWaves; ++i) v += red[i][f][l][r & 3];
    return v;
  };
#pragma unroll
  for (int i = 0; i < kElems; ++i) {
    if (el[i].t < 0) continue;
    const int f = el[i].t >> 4, tk = el[i].t & 15;
    epi_one(e, el[i].t, el[i].n, total(f, el[i].r, tk), pair ? total(f, el[i].r + 8, tk) : 0.0f, el[i].in);
  }
}

// ---- more tokens ---------------------------------------------------------------------------

// fp32 activations to bf16 term planes, `plane` elements apart.
template <int TERMS>
__global__ __launch_bounds__(256) void terms_kernel(const float* __restrict__ x, int64_t n4, uint16_t* __restrict__ planes,
                                                    int64_t plane) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256)
    write_terms<TERMS>(x, i, planes, plane);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct LinearPlan {
  bool few;
  int terms;
  bool split_first;  // fp32 x becomes term planes by a launch of its own
  Plan plan;
  int rows;          // tokens at a time: all, or half of them
  size_t planes, partial, bytes;  // offsets and size of the workspace
  int R, ldp;
};
LinearPlan linear_plan(int T, int K, int N, int act, moe_dtype x_t, moe_dtype y_t) {
  LinearPlan p{};
  p.R = act == MOE_ACT_SWIGLU ? 2 * N : N;
  p.ldp = (p.R + 3) / 4 * 4;
  p.few = T <= kFewT;
  if (p.few) return p;
  p.terms = x_t == MOE_BF16 ? 1 : y_t == MOE_F32 ? 3 : 2;
  // Two planes are made and used for half of the tokens at a time, so that they take the memory of x in bf16 beside a bf16 y.
  const int turns = p.terms == 2 ? 2 : 1;
  const Shape shape{T, p.R, K, p.terms, x_t == MOE_F32, turns};
  p.plan = plan_products(&shape, 1);
  p.split_first = x_t == MOE_F32 && p.plan.shape != kDirect;
  p.rows = p.split_first ? (int)ceil_div(T, turns) : T;
  size_t o = 0;
  p.planes = o;
  if (p.split_first) o = up256(o + (size_t)p.terms * p.rows * K * 2);
  p.partial = o;
  if (p.plan.split[0] > 1) o = up256(o + (size_t)p.plan.split[0] * p.rows * p.ldp * 4);
  p.bytes = o;
  return p;
}

}  // namespace

static moe_status launch_terms(const float* x, int64_t n, uint16_t* planes, int64_t plane, int terms, hipStream_t s) {
  const dim3 grid((unsigned)std::min<int64_t>(2048, ceil_div(n / 4, 256)));
  if (terms == 2) terms_kernel<2><<<grid, 256, 0, s>>>(x, n / 4, planes, plane);
  else terms_kernel<3><<<grid, 256, 0, s>>>(x, n / 4, planes, plane);
  return check_launch("linear");
}

size_t linear_ws_bytes(int T, int K, int N, int act, moe_dtype x_t, moe_dtype y_t) {
  return linear_plan(T, K, N, act, x_t, y_t).bytes;
}

void linear_form(int T, int K, int N, int act, moe_dtype x_t, moe_dtype y_t, int32_t form[4]) {
  const LinearPlan p = linear_plan(T, K, N, act, x_t, y_t);
  form[0] = p.few ? 0 : tile_side(p.plan);
  form[1] = p.few ? 1 : p.plan.split[0];
  form[2] = !p.few ? p.terms : x_t == MOE_F32 ? 3 : 1;
  form[3] = p.split_first ? (int)ceil_div(T, p.rows) : 0;
}

moe_status launch_linear(const void* x, moe_dtype x_t, const uint16_t* w, const float* bias, int act,
                         const void* residual, moe_dtype r_t, int T, int K, int N, void* y, moe_dtype y_t, void* pre,
                         void* ws, hipStream_t s) {
  const LinearPlan pl = linear_plan(T, K, N, act, x_t, y_t);
  Epi e{bias, residual, y, pre, N, pl.R, act, r_t == MOE_BF16, y_t == MOE_BF16};
  if (pl.few) {
    const dim3 grid((unsigned)ceil_div(N, act == MOE_ACT_SWIGLU ? 8 : 16));
    auto go = [&](auto kernel) { launch_k(MOE_KERNEL_LINEAR, kernel, grid, dim3(64 * kFewWaves), 0, s, x, w, T, K, e); };
    const bool f = x_t == MOE_F32;
    if (T <= 16) f ? go(linear_few_kernel<true, 1>) : go(linear_few_kernel<false, 1>);
    else if (T <= 32) f ? go(linear_few_kernel<true, 2>) : go(linear_few_kernel<false, 2>);
    else f ? go(linear_few_kernel<true, 4>) : go(linear_few_kernel<false, 4>);
    return check_launch("linear");
  }
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  for (int t = 0; t < T; t += pl.rows) {
    const int n = std::min(pl.rows, T - t);
    auto from = [&](const void* q, size_t row_bytes) {  // row t of a buffer, or null
      return q ? reinterpret_cast<const uint8_t*>(q) + (size_t)t * row_bytes : nullptr;
    };
    const size_t by = y_t == MOE_F32 ? 4 : 2;
    Prob p{};
    p.A = reinterpret_cast<const uint16_t*>(from(x, (size_t)K * (x_t == MOE_F32 ? 4 : 2)));
    if (pl.split_first) {
      uint16_t* planes = reinterpret_cast<uint16_t*>(base + pl.planes);
      p.a_plane = (int64_t)n * K;
      if (moe_status st = launch_terms(reinterpret_cast<const float*>(p.A), (int64_t)n * K, planes, p.a_plane, pl.terms, s))
        return st;
      p.A = planes;
    }
    p.B = w;
    p.lda = p.ldb = K;
    p.M = n;
    p.R = pl.R;
    p.K = K;
    p.nseg = pl.plan.shape == kDirect ? 1 : pl.terms;
    p.terms = pl.terms;
    p.sa = 0 | 1u << 2 | 2u << 4;
    p.sb = 0;
    p.split = pl.plan.split[0];
    p.partial = reinterpret_cast<float*>(base + pl.partial);
    p.ldp = pl.ldp;
    p.epi = e;
    p.epi.res = from(residual, (size_t)N * (r_t == MOE_F32 ? 4 : 2));
    p.epi.y = const_cast<uint8_t*>(from(y, (size_t)N * by));
    p.epi.pre = const_cast<uint8_t*>(from(pre, (size_t)pl.R * by));
    if (moe_status st = launch_products(MOE_KERNEL_LINEAR, pl.plan, &p, 1, false, false, DbSum{}, s, "linear")) return st;
  }
  return MOE_OK;
}

}  // namespace moe
