// orthogonalize_small.hip -- Newton-Schulz steps of matrices whose shorter side m is at most 64 (routers of few experts),
// in three launches instead of two and three for each step.
//
// Every step multiplies X by a polynomial of its Gram matrix, all of them are polynomials of the first one and commute, so
// they can be gathered on the shorter side: with A = X X^T,
//   S = b A + c A^2,  P = a I + S,  Q' = P Q = a Q + S Q,  A' = P A P = a^2 A + 2 a S A + S (S A),
// and o = Q X in the end.  X (m x n) is read twice whatever the number of steps, and one workgroup holds A, S, S A and Q of
// a matrix in LDS through all of them.
//
// What is near 0 in A, and the noise beside it, grows by a^2 a step, 19,800 over the four that matter of five, where X's own
// steps have 3.44 each.  A is therefore summed in 64 bits, and steps run in 64 bits until A's rounding to fp32 grows by no
// more than 144 in the steps that are left, and what the first fp32 step adds by no more than 16 in those behind it: two of five for
// a bf16 result, all for an fp32 one.  On matrices of one or a few strong directions over noise of 0.01 to 1 of them, sides 8
// to 64, a bf16 result was then off by 8e-4 of its norm at most before its rounding (1.66e-3); with the first step alone in 64 bits
// by 6e-3, with none by 6e-2; with three by 1.1e-4, 3 us slower.  (The bound of 16 alone lets the fp32 steps begin with one of
// any a: with a = 15 there results were 5e-3 to 2.6e-2 off.  Tiles are stored on both sides of the diagonal, so products that should
// commute leave their noise on A.)  Coefficients whose growth 64 bits do not hold go the way of orthogonalize.hip.
//
// One 60 x 544 matrix: 4.8 us for its Gram matrix, 26.6 for the steps (34 in 64 bits throughout; one workgroup, whose products,
// barriers and trips through LDS follow one another) and 4.6 for Q X; by the launches of orthogonalize.hip 74 in all.
//
// v_mfma_f32_16x16x4_f32 and v_mfma_f64_16x16x4_f64: lane l holds row l % 16 and k = l / 16 of an operand; of the result
// column l % 16, rows 4 (l / 16) + i in fp32 and 4 i + l / 16 in 64 bits.
#include <algorithm>
#include <cmath>

#include "newton_dev.hpp"

namespace moe {
namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));
constexpr int kSide = 64, kTiles = 10;  // 16 x 16 tiles on and above the diagonal of a 64 x 64 matrix
constexpr int kMaxParts = 32;           // workgroups that share a matrix's Gram matrix
constexpr int kMaxSteps = 16;

template <typename F>
struct Mat;
template <>
struct Mat<float> {
  typedef f32x4_t Acc;
  static constexpr int kStride = 68, kLong = 80;  // values per row in LDS: the lanes of a read fall on different banks
  static __device__ __forceinline__ Acc mma(float a, float b, Acc c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }
  static __device__ __forceinline__ int row(int i, int q) { return 4 * q + i; }
};
template <>
struct Mat<double> {
  typedef f64x4_t Acc;
  static constexpr int kStride = 66, kLong = 80;
  static __device__ __forceinline__ Acc mma(double a, double b, Acc c) { return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0); }
  static __device__ __forceinline__ int row(int i, int q) { return 4 * i + q; }
};

// Tile number to its place, column by column of the upper triangle.
__device__ __forceinline__ void tile_at(int t, int& i, int& j) {
  j = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0;
  i = t - j * (j + 1) / 2;
}

// 64 x 64 values of u (rows from r0, columns from k0 on) to v: thread t holds columns 4 (t % 16) of rows t / 16 + 16 i.
template <bool MOMENT>
__device__ __forceinline__ void load_tile(const Update& u, int64_t base, int r0, int k0, float (&v)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) load_update<MOMENT>(u, base, r0 + 16 * i + (threadIdx.x >> 4), k0 + (threadIdx.x & 15) * 4, v[i]);
}

// Parts of the Gram matrices: a workgroup takes `subs` stretches of 64 along the longer side, brings the moment up to
// date there, and leaves the ten tiles of its sum as the lanes of the next kernel hold them.
__global__ __launch_bounds__(256) void small_gram_kernel(Update u, int parts, int subs, double* __restrict__ out) {
  __shared__ float xs[kSide * 80];
  const int matrix = blockIdx.x / parts, part = blockIdx.x - matrix * parts;
  const int64_t base = (int64_t)matrix * u.R * u.K;
  const bool turned = u.R > u.K;
  const int n = max(u.R, u.K), tiles = (min(u.R, u.K) + 15) / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
  const int count = tiles * (tiles + 1) / 2;
  // u lies in LDS as in memory: [short][long] at a stride of 68, or [long][short] at 80
  const int along_m = turned ? 1 : 68, along_n = turned ? 80 : 1, stride = turned ? 80 : 68;
  f64x4_t acc[3] = {};
  float v[4][4];
  const int first = part * subs, last = min(first + subs, (n + kSide - 1) / kSide);
  load_tile<true>(u, base, turned ? first * kSide : 0, turned ? 0 : first * kSide, v);
  for (int c = first; c < last; ++c) {
    if (c > first) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(xs + (16 * i + (threadIdx.x >> 4)) * stride + (threadIdx.x & 15) * 4) =
          make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
    __syncthreads();
    if (c + 1 < last) load_tile<true>(u, base, turned ? (c + 1) * kSide : 0, turned ? 0 : (c + 1) * kSide, v);
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      const int t = wave + 4 * s;
      if (t >= count) break;
      int ti, tj;
      tile_at(t, ti, tj);
      const float* a = xs + (16 * ti + r) * along_m + q * along_n;
      const float* b = xs + (16 * tj + r) * along_m + q * along_n;
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[s] = Mat<double>::mma(a[4 * k * along_n], b[4 * k * along_n], acc[s]);
    }
  }
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const int t = wave + 4 * s;
    if (t >= count) break;
    double* to = out + ((int64_t)blockIdx.x * kTiles + t) * 256;
#pragma unroll
    for (int i = 0; i < 4; ++i) to[lane * 4 + i] = acc[s][i];
  }
}

struct Coefs {
  float v[3 * kMaxSteps];
};

// A symmetric matrix of TILES x TILES tiles in LDS that several waves write tile by tile and multiply.  (fp32 values as three bf16 terms on
// v_mfma_f32_16x16x32_bf16 need a third of the matrix units' time, but cutting them into terms took as long again.)
template <typename F, int TILES>
struct Held {
  typedef Mat<F> M;
  typedef typename M::Acc Acc;
  static constexpr int kS = M::kStride;
  F v[16 * TILES * kS] __attribute__((aligned(16)));
  __device__ __forceinline__ void store(int ti, int tj, const Acc& t) {
    const int r = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;
    const int col = 16 * tj + r;
    if constexpr (sizeof(F) == 4) {  // four neighbouring rows
      *reinterpret_cast<Acc*>(v + col * kS + 16 * ti + 4 * q) = t;
      if (ti == tj) return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * ti + M::row(i, q);
      v[row * kS + col] = t[i];
      if constexpr (sizeof(F) == 8) v[col * kS + row] = t[i];
    }
  }
  // The tile of x y, and with TWO that of x z: x's values are read once, and independent sums follow each other on the
  // matrix unit.
  template <bool TWO>
  static __device__ __forceinline__ void products(const Held& x, const Held& y, const Held& z, int ti, int tj, Acc& xy,
                                                  Acc& xz) {
    const int r = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;
    const int at = (16 * ti + r) * kS + q, bt = (16 * tj + r) * kS + q;
    Acc u = {}, w = {};
#pragma unroll
    for (int k = 0; k < 4 * TILES; ++k) {
      const F p = x.v[at + 4 * k];
      u = M::mma(p, y.v[bt + 4 * k], u);
      if constexpr (TWO) w = M::mma(p, z.v[bt + 4 * k], w);
    }
    xy = u;
    if constexpr (TWO) xz = w;
  }
};

template <typename F, int TILES>
struct Work {  // of the steps, in LDS
  Held<F, TILES> as, ss, ts, qs;
};

// Steps from ... to - 1 of `steps`: wave t has tile t of the upper triangle of every matrix, and stores it on both sides.  A is
// in w.as, too, and from the second step on Q in w.qs.
template <typename F, int TILES>
__device__ __forceinline__ void run_steps(Work<F, TILES>& w, const Coefs& coef, int from, int to, int steps, int ti, int tj,
                                          typename Mat<F>::Acc& A, typename Mat<F>::Acc& Q) {
  typedef Mat<F> M;
  typedef typename M::Acc Acc;
  typedef Held<F, TILES> H;
  const int r = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;
  for (int k = from; k < to; ++k) {
    const F a = coef.v[3 * k], b = coef.v[3 * k + 1], c = coef.v[3 * k + 2];
    Acc S = {}, T = {}, z = {};
    H::template products<false>(w.as, w.as, w.as, ti, tj, S, z);
#pragma unroll
    for (int i = 0; i < 4; ++i) S[i] = b * A[i] + c * S[i];
    w.ss.store(ti, tj, S);
    __syncthreads();
    const bool last = k + 1 == steps;
    if (k == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) Q[i] = ti == tj && M::row(i, q) == r ? S[i] + a : S[i];
      if (!last) H::template products<false>(w.ss, w.as, w.as, ti, tj, T, z);
    } else {
      if (last) H::template products<false>(w.ss, w.qs, w.qs, ti, tj, z, T);
      else H::template products<true>(w.ss, w.qs, w.as, ti, tj, z, T);
#pragma unroll
      for (int i = 0; i < 4; ++i) Q[i] = a * Q[i] + z[i];
    }
    if (last) break;
    __syncthreads();  // Q's old values have been read
    w.qs.store(ti, tj, Q);
    w.ts.store(ti, tj, T);
    __syncthreads();
    H::template products<false>(w.ss, w.ts, w.ts, ti, tj, z, S);
#pragma unroll
    for (int i = 0; i < 4; ++i) A[i] = a * (a * A[i] + (F)2 * T[i]) + z[i];
    w.as.store(ti, tj, A);
    __syncthreads();
  }
}

// All steps of one matrix, the first `wide` of them in 64 bits.  Leaves Q [64][64] (of which the tiles in use are written) and
// 1 / (norm + eps).
template <typename F, int TILES>
__global__ __launch_bounds__(32 * TILES * (TILES + 1)) void small_steps_kernel(const double* __restrict__ parts, int count,
                                                                                int steps, int wide, Coefs coef, double eps,
                                                                                F* __restrict__ q_out,
                                                                                double* __restrict__ inv_out) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[sizeof(Work<double, TILES>)];
  constexpr int kWaves = TILES * (TILES + 1) / 2;
  __shared__ double red[kWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
  int ti, tj;
  tile_at(wave, ti, tj);
  f64x4_t g = {};
  const double* p = parts + (((int64_t)blockIdx.x * count * kTiles + wave) * 64 + lane) * 4;
  for (int first = 0; first < count; first += 8) {
    f64x4_t v[8];  // (loads past the last part bring it again and are left out)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = *reinterpret_cast<const f64x4_t*>(p + (int64_t)min(first + e, count - 1) * kTiles * 256);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (first + e < count) g += v[e];
  }
  double trace = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (ti == tj && Mat<double>::row(i, q) == r) trace += g[i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) trace += __shfl_xor(trace, d);
  if (lane == 0) red[wave] = trace;
  __syncthreads();
  double squares = 0.0;
#pragma unroll
  for (int i = 0; i < TILES; ++i) squares += red[i * (i + 3) / 2];  // (the tiles on the diagonal)
  const double inv = inverse_norm(squares, eps);
  if (threadIdx.x == 0) inv_out[blockIdx.x] = inv;

  Work<double, TILES>& w = *reinterpret_cast<Work<double, TILES>*>(lds);
  f64x4_t A = {}, Q = {};
  A = g * inv * inv;
  w.as.store(ti, tj, A);
  __syncthreads();
  run_steps<double, TILES>(w, coef, 0, wide, steps, ti, tj, A, Q);
  auto leave = [&](const auto& tile, auto of) {
    F* to = q_out + (int64_t)blockIdx.x * kSide * kSide;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * ti + decltype(of)::row(i, q), col = 16 * tj + r;
      to[row * kSide + col] = (F)tile[i];
      if (ti != tj) to[col * kSide + row] = (F)tile[i];
    }
  };
  if (sizeof(F) == 8 || wide == steps) {
    leave(Q, Mat<double>{});
  } else if constexpr (sizeof(F) == 4) {  // the lanes hold other rows of an fp32 tile: A and Q come back out of LDS
    Work<float, TILES>& n = *reinterpret_cast<Work<float, TILES>*>(lds);
    f32x4_t an = {}, qn = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = (16 * ti + Mat<float>::row(i, q)) * Held<double, TILES>::kS + 16 * tj + r;
      an[i] = (float)w.as.v[at];
      qn[i] = wide ? (float)w.qs.v[at] : 0.0f;
    }
    __syncthreads();
    n.as.store(ti, tj, an);
    n.qs.store(ti, tj, qn);
    __syncthreads();
    run_steps<float, TILES>(n, coef, wide, steps, steps, ti, tj, an, qn);
    leave(qn, Mat<float>{});
  }
}

// o = Q u / (norm + eps), 64 values along the longer side per workgroup; wave w has rows 16 w ... of Q.
template <typename F>
__global__ __launch_bounds__(256) void small_apply_kernel(Update u, int chunks, const F* __restrict__ q_in,
                                                          const double* __restrict__ inv_in, void* o, int o_bf16) {
  typedef Mat<F> M;
  constexpr int kS = M::kStride, kL = M::kLong;
  __shared__ F qs[kSide * kS], xs[kSide * kL];
  const int matrix = blockIdx.x / chunks, chunk = blockIdx.x - matrix * chunks;
  const int64_t base = (int64_t)matrix * u.R * u.K;
  const bool turned = u.R > u.K;
  const int m = min(u.R, u.K), n = max(u.R, u.K), tiles = (m + 15) / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
  float v[4][4];
  load_tile<false>(u, base, turned ? chunk * kSide : 0, turned ? 0 : chunk * kSide, v);
  typedef F F4 __attribute__((ext_vector_type(4)));
  const F4* from = reinterpret_cast<const F4*>(q_in + (int64_t)matrix * kSide * kSide);
  F4 part[4];  // (rows and columns past the tiles in use hold what they held before; nothing reads them)
#pragma unroll
  for (int i = 0; i < 4; ++i) part[i] = from[256 * i + threadIdx.x];
  const double inv = inv_in[matrix];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) qs[(16 * i + (threadIdx.x >> 4)) * kS + (threadIdx.x & 15) * 4 + e] = part[i][e];
  const int stride = turned ? kS : kL;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      xs[(16 * i + (threadIdx.x >> 4)) * stride + (threadIdx.x & 15) * 4 + e] = (F)((double)v[i][e] * inv);
  __syncthreads();
  if (wave >= tiles) return;
  const int along_m = turned ? 1 : kL, along_n = turned ? kS : 1;
  typename M::Acc acc[4] = {};
  const F* a = qs + (16 * wave + r) * kS + q;
  const F* b = xs + q * along_m + r * along_n;
  for (int t = 0; t < tiles; ++t) {
#pragma unroll
    for (int k = 4 * t; k < 4 * t + 4; ++k) {
      const F x = a[4 * k];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = M::mma(x, b[4 * k * along_m + 16 * j * along_n], acc[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * wave + M::row(i, q), col = chunk * kSide + 16 * j + r;
      if (row < m && col < n)
        store_any(o, o_bf16, base + (turned ? (int64_t)col * u.K + row : (int64_t)row * u.K + col), (float)acc[j][i]);
    }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct SmallPlan {
  int chunks, parts, subs;  // stretches of 64; workgroups that share a Gram matrix, and the stretches of each
  size_t gram, q, inv, bytes;
};
SmallPlan small_plan(int64_t B, int R, int K) {
  SmallPlan p{};
  p.chunks = (int)ceil_div(std::max(R, K), kSide);
  p.subs = (int)ceil_div(p.chunks, kMaxParts);
  p.parts = (int)ceil_div(p.chunks, p.subs);
  size_t o = 0;
  p.gram = o; o = up256(o + (size_t)B * p.parts * kTiles * 256 * 8);
  p.q = o; o = up256(o + (size_t)B * kSide * kSide * 8);
  p.inv = o; o = up256(o + (size_t)B * 8);
  p.bytes = o;
  return p;
}

// What A's smallest eigenvalues, and the noise beside them, grow by in steps first ... steps - 2, before the last step uses them.
double growth(int first, int steps, const float* coef) {
  double g = 1.0;
  for (int i = first; i + 1 < steps; ++i) g *= std::max(1.0, (double)coef[3 * i] * coef[3 * i]);
  return g;
}
constexpr double kGrowthA = 144.0, kGrowthStep = 16.0, kGrowth64 = 268435456.0;

}  // namespace

bool newton_is_small(int R, int K, int steps, const float* coef) {
  return std::min(R, K) <= kSide && (!coef || growth(0, steps, coef) <= kGrowth64);
}

size_t newton_small_ws_bytes(int B, int R, int K) {
  return std::min(R, K) <= kSide ? small_plan(B, R, K).bytes : 0;
}

moe_status launch_newton_small(const Update& u, int B, int steps, const float* coef, double eps, void* o, moe_dtype o_t,
                               void* ws, hipStream_t s) {
  const SmallPlan p = small_plan(B, u.R, u.K);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  double* gram = reinterpret_cast<double*>(base + p.gram);
  double* inv = reinterpret_cast<double*>(base + p.inv);
  const int tiles = (std::min(u.R, u.K) + 15) / 16;
  Coefs c{};
  std::copy(coef, coef + 3 * steps, c.v);
  int wide = steps;  // steps in 64 bits: all that leave an A whose noise would grow
  if (o_t == MOE_BF16)
    while (wide > 0 && growth(wide, steps, coef) <= kGrowthStep && growth(wide - 1, steps, coef) <= kGrowthA) --wide;
  small_gram_kernel<<<dim3((unsigned)(B * p.parts)), 256, 0, s>>>(u, p.parts, p.subs, gram);
  if (moe_status st = check_launch("orthogonalize")) return st;
  const dim3 all((unsigned)((int64_t)B * p.chunks));
  auto go = [&](auto zero) {
    using F = decltype(zero);
    F* q = reinterpret_cast<F*>(base + p.q);
    auto run = [&](auto kernel) {
      launch_k(MOE_KERNEL_ORTHOGONALIZE, kernel, dim3((unsigned)B), dim3((unsigned)(32 * tiles * (tiles + 1))), 0, s, gram, p.parts, steps, wide, c, eps, q, inv);
    };
    if (tiles == 1) run(small_steps_kernel<F, 1>);
    else if (tiles == 2) run(small_steps_kernel<F, 2>);
    else if (tiles == 3) run(small_steps_kernel<F, 3>);
    else run(small_steps_kernel<F, 4>);
    small_apply_kernel<F><<<all, 256, 0, s>>>(u, p.chunks, q, inv, o, o_t == MOE_BF16);
  };
  if (o_t == MOE_BF16) go(0.0f);
  else go(0.0);
  return check_launch("orthogonalize");
}

}  // namespace moe
