// orthogonalize.hip -- an update made orthogonal by Newton-Schulz steps:
//   X = u / (|u|_F + eps);  each step: A = X X^T, P = b A + c A^2, X = a X + P X  (on the shorter side m x n, m <= n)
// which takes each singular value s of X to a s + b s^3 + c s^5 and leaves the singular vectors as they are.
//
// Products run on v_mfma_f32_16x16x32_f16.  fp16 holds 11 bits where bf16 holds 8, and its range is enough: X, A and P of a
// normalised matrix stay within a few units, and are stored times 2^13, 2^12 and 2^11, so that what lies below fp16's
// normal range is below 2^-25 of the largest value.  X's singular values below 4 and P's eigenvalues below 16, as the call asks for,
// leave X's values below 4, P's below 16, and A's off its diagonal at no more than 8 (A has no negative eigenvalue), all
// at about half of fp16's largest value.
//
// What the roundings do: a step multiplies a small singular value by a = 3.44, five of them by 485, and noise beside
// it as much, so X rounded to 11 bits before each step leaves results of low-rank gradients 1 to 7% off, and bf16 20%
// or more.  X is therefore kept as two fp16 terms (22 bits): the sum a X takes both, and only the product P X, whose P is
// nearly 0 on the weak directions, takes the first alone.  The diagonals of A and P, the largest of their values where the spectrum
// is even or few rows are not 0, stay in fp32 beside them: A^2 = E^2 + D E + E D + D^2, E off the diagonal D, and
// diag P X.  (With A's diagonal in 11 bits, too, gradients of a few rows were up to 6e-3 off; in fp32 it costs 0.5 to 2%.)
// The result is 0.1 to 1.2e-3 of its norm off on matrices of 128 to 4,096 rows from Gaussian ones to one strong direction
// over noise, 1.2 to 1.9e-3 where few rows are not 0, 0.9 to 2.5e-3 where all singular values are equal; a bf16
// result's own rounding is 1.66e-3.  Matrices of one value in each row and column, whose roundings do not average out, come to
// 7e-3 where the values are equal and to 1.8e-2 with two or three of the worst sizes.  An fp32 result takes two terms of X,
// A and P in every product (three passes of the matrix units), and is as near as an fp32 computation.
//
// A and P are symmetric: only tiles on and above the diagonal are computed, and stored twice.  All matrices of a
// call share each launch.  m and n are padded to multiples of 64 with zeros, which stay zeros.
#include "newton_dev.hpp"
#include "product_dev.hpp"

namespace moe {
namespace {

// A tile shape besides those of product_dev.hpp: 192 x 192 (12 waves, 64 x 48 each), for symmetric products whose 256 x 256
// tiles leave half of the CUs without one.
using Mid = Tile<192, 192, 3, 4>;
// Small tiles for launches of few of them, whose time is latency: an epilogue of few values per thread and short ways to
// it, 76 -> 57 us for all of a 128 x 128 matrix, 104 -> 79 for 512 x 512.  A K-step brings two pieces of each operand: of
// one term 128 k, of two terms both planes of 64 k, which the three products of the terms then share (1,001 x 777 in two
// terms: 232 -> 160 us).  Rings of three buffers measured better than longer ones, which leave fewer workgroups to a CU.
template <typename T, int RING>
struct Paired : T {
  static constexpr int kRing = RING, kPair = 2 * T::kStage;  // words of a buffer: A's two pieces, then B's
  static constexpr int kBuffers = kRing * kPair * 2, kLds = std::max(kBuffers, T::TM * T::TN * 4);
  static_assert(kBuffers <= 160 * 1024, "LDS of a CU");
};
template <typename T>
struct IsPaired : std::false_type {};
template <typename T, int RING>
struct IsPaired<Paired<T, RING>> : std::true_type {};
using Nano = Paired<Tile<32, 32, 2, 2>, 3>;  // symmetric products
using Flat = Paired<Tile<32, 64, 2, 2>, 3>;  // P X
using Wide = Paired<Tile<64, 64, 2, 2, 3, 2>, 3>;

constexpr float kXScale = 8192.0f, kGScale = 4096.0f, kPScale = 2048.0f;  // of X, A and P

__device__ __forceinline__ uint16_t f32_to_f16(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
__device__ __forceinline__ float f16_to_f32(uint32_t h) { return (float)__builtin_bit_cast(_Float16, (uint16_t)h); }

// Four values as 8 bytes of fp16 and what they leave, rounded again.
__device__ __forceinline__ void terms4(const float (&v)[4], uint2& hi, uint2& lo) {
  uint16_t h[4], l[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    h[r] = f32_to_f16(v[r]);
    l[r] = f32_to_f16(v[r] - f16_to_f32(h[r]));
  }
  hi = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
  lo = make_uint2(l[0] | (uint32_t)l[1] << 16, l[2] | (uint32_t)l[3] << 16);
}
__device__ __forceinline__ void unpack4(uint2 q, float (&v)[4]) {
  v[0] = f16_to_f32(q.x & 0xFFFF); v[1] = f16_to_f32(q.x >> 16);
  v[2] = f16_to_f32(q.y & 0xFFFF); v[3] = f16_to_f32(q.y >> 16);
}

// P X reads X's first term twice, the second time while the L2 may still hold it, and its second term once, whose loads
// are therefore marked as not to be kept (16 matrices of 1,024 x 2,048: 1,239 -> 1,202 us; not in launches of few tiles: one of
// 512 x 2,048 111 -> 113).  What it writes is read by the next launches, from the 256 MB cache where X's terms, old and
// new, fit there; else its stores are marked, too (48 of 512 x 2,048: 1,164 -> 1,119 us, 100 of 256 x 2,048: 991 -> 964; 24 of
// 512 x 2,048, which fit: 631 -> 661), and it goes through the batch from the back, as A before it has just read the last X (100
// of 512 x 2,048: 2,306 -> 2,272; where X fits this costs more than it gives, 8 of 512 x 2,048: 255 -> 271).
constexpr size_t kKept = 256u << 20;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint2 load_once(const uint16_t* p) {
  const u32x2_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(p));
  return make_uint2(v.x, v.y);
}
__device__ __forceinline__ void store_past(uint16_t* p, uint2 v) {
  __builtin_nontemporal_store(u32x2_t{v.x, v.y}, reinterpret_cast<u32x2_t*>(p));
}

// ---- the update and its norm -----------------------------------------------------------

// Values that a workgroup of the next kernel has under way at once; up to 1,024 workgroups a matrix.  (With one load of four
// values a thread at a time and 8,192 values a workgroup 512 x 2,048 took 113 us in all instead of 110, 48 of them 1,128 instead
// of 1,110, 4,096 x 4,096 1,487 instead of 1,480.)
constexpr int kNormValues = 2048, kNormBlocks = 1024;

// The moment m = beta m + (1 - beta) g, and per workgroup the sum of u^2.  In 64 bits: squares of fp32 values neither
// overflow nor vanish there.  48 matrices of 512 x 2,048, bf16 with momentum: 503 MB in 74 us (98 at a copy's rate; part of what
// is written stays in the 256 MB cache).
__global__ __launch_bounds__(256) void newton_moment_kernel(Update u, int blocks, double* __restrict__ parts) {
  __shared__ double red[4];
  const int matrix = blockIdx.x / blocks, block = blockIdx.x - matrix * blocks;
  const int64_t n = (int64_t)u.R * u.K, base = matrix * n;
  double sum = 0.0;
  for (int64_t first = (int64_t)block * kNormValues; first < n; first += (int64_t)blocks * kNormValues) {
    if (first + kNormValues <= n) {
      float g[kNormValues / 1024][4], m[kNormValues / 1024][4] = {};
      const int64_t at = base + first + threadIdx.x * 4;
#pragma unroll
      for (int e = 0; e < kNormValues / 1024; ++e) load4(u.g, u.g_bf16, at + e * 1024, g[e]);
      if (u.moment) {
#pragma unroll
        for (int e = 0; e < kNormValues / 1024; ++e) load4(u.moment, 0, at + e * 1024, m[e]);
#pragma unroll
        for (int e = 0; e < kNormValues / 1024; ++e) {
#pragma unroll
          for (int r = 0; r < 4; ++r) m[e][r] = __builtin_fmaf(u.beta, m[e][r], u.rest * g[e][r]);
          store4(u.moment, 0, at + e * 1024, m[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < kNormValues / 1024; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const double v = update_of(u, g[e][r], m[e][r]);
          sum += v * v;
        }
    } else {
      for (int64_t i = first + threadIdx.x; i < n; i += 256) {
        const float gv = load_any(u.g, u.g_bf16, base + i);
        float mv = 0.0f;
        if (u.moment) {
          mv = __builtin_fmaf(u.beta, u.moment[base + i], u.rest * gv);
          u.moment[base + i] = mv;
        }
        const double v = update_of(u, gv, mv);
        sum += v * v;
      }
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) parts[blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

struct Planes {  // of fp16 terms, `plane` words apart, matrices `step` words apart
  uint16_t* p;
  int64_t plane, step;
};

// X in two terms, padded with zeros, transposed where R > K: a workgroup brings 64 x 64 values of u through LDS.  The norm has
// to be known before a value is rounded, so g and the moment are read again: 503 MB in 94 us for the 48 matrices above.  They
// come from the back, as the caches still hold the last of what the kernel before has read (11 us of 1,106).
__global__ __launch_bounds__(256) void newton_start_kernel(Update u, int blocks, const double* __restrict__ parts, double eps,
                                                           int tr, int tk, Planes x, int ld) {
  __shared__ float tile[64][65];
  __shared__ double red[4];
  const int item = gridDim.x - 1 - blockIdx.x, per = tr * tk, matrix = item / per, t = item - matrix * per;
  const int r0 = t / tk * 64, k0 = t % tk * 64;
  const int64_t base = (int64_t)matrix * u.R * u.K;
  double sum = 0.0;
  for (int i = threadIdx.x; i < blocks; i += 256) sum += parts[(int64_t)matrix * blocks + i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  const int c = (threadIdx.x & 15) * 4, k = k0 + c;
  float v[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 16 * i + (threadIdx.x >> 4);
    load_update<false>(u, base, r, k, v[i]);
  }
  __syncthreads();
  const double inv = kXScale * inverse_norm((red[0] + red[1]) + (red[2] + red[3]), eps);
  const bool turned = u.R > u.K;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 16 * i + (threadIdx.x >> 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i][e] = (float)(v[i][e] * inv);
    if (turned) {
#pragma unroll
      for (int e = 0; e < 4; ++e) tile[c + e][r] = v[i][e];
    }
  }
  if (turned) __syncthreads();
  uint16_t* to = x.p + matrix * x.step + (turned ? (int64_t)k0 * ld + r0 : (int64_t)r0 * ld + k0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 16 * i + (threadIdx.x >> 4);
    if (turned) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = tile[r][c + e];
    }
    uint2 hi, lo;
    terms4(v[i], hi, lo);
    uint16_t* at = to + (int64_t)r * ld + c;
    *reinterpret_cast<uint2*>(at) = hi;
    *reinterpret_cast<uint2*>(at + x.plane) = lo;
  }
}

// The products of a tile by a Paired shape (see product_loop for the ring): K is a multiple of 64.
template <typename T, bool BK, int TERMS, typename RowA, typename RowB>
__device__ __forceinline__ void paired_loop(const Mats& p, int m0, int n0, RowA row_a, RowB row_b, uint8_t* lds,
                                            f32x4_t (&acc)[T::kFM][T::kFN]) {
  constexpr int kFM = T::kFM, kFN = T::kFN, WM = T::WM, WN = T::WN, kPieceA = T::kStageA, kPieceB = T::kStage - T::kStageA;
  const int wave = uniform(threadIdx.x >> 6), kg = wave / (WM * WN), wm = wave / WN % WM, wn = wave % WN;
  Operand<T::TM, T::kThreads, false> A;
  Operand<T::TN, T::kThreads, BK> B;
  A.init(p.lda, p.lda - m0, row_a);
  B.init(p.ldb, p.ldb - n0, row_b);
  const int steps = p.K / kBK, phases = TERMS == 2 ? steps : (steps + 1) / 2;
  uint16_t* const base = reinterpret_cast<uint16_t*>(lds);
  const int64_t step_a = kBK, step_b = BK ? (int64_t)kBK * p.ldb : kBK;
  const uint16_t *src_a = A.at(p.A, m0, 0, p.lda), *src_b = B.at(p.B, n0, 0, p.ldb);
  int next = 0;  // the phase that is loaded next
  auto load = [&](int buf) {
    uint16_t* la = base + buf * T::kPair;
    uint16_t* lb = la + 2 * kPieceA;
    A.load(src_a, p.lda, la, 64 * wave);
    B.load(src_b, p.ldb, lb, 64 * wave);
    // (one term and an odd number of steps: the last has no second piece, and its first one again is not multiplied)
    const bool pair = TERMS == 2 || 2 * next + 1 < steps;
    A.load(src_a + (TERMS == 2 ? p.a_plane : pair ? step_a : 0), p.lda, la + kPieceA, 64 * wave);
    B.load(src_b + (TERMS == 2 ? p.b_plane : pair ? step_b : 0), p.ldb, lb + kPieceB, 64 * wave);
    if (next + 1 < phases) {  // (past the end the last phase is loaded again, into a buffer that nobody reads)
      ++next;
      src_a += (TERMS == 2 ? 1 : 2) * step_a;
      src_b += (TERMS == 2 ? 1 : 2) * step_b;
    }
  };
#pragma unroll
  for (int i = 0; i < kFM; ++i)
#pragma unroll
    for (int j = 0; j < kFN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  constexpr int kPer = 2 * (decltype(A)::kLoads + decltype(B)::kLoads), kLeft = (T::kRing - 2) * kPer;
  static_assert(kLeft < 64, "vmcnt's bits");
#pragma unroll
  for (int i = 0; i < T::kRing - 1; ++i) load(i);
  int now = 0, free = T::kRing - 1;
  for (int s = 0; s < phases; ++s) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (kLeft & 15) | (kLeft >> 4) << 14);  // vmcnt(kLeft) lgkmcnt(0): this phase's loads have landed
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    load(free);
    const uint16_t* la = base + now * T::kPair;
    const uint16_t* lb = la + 2 * kPieceA;
#pragma unroll
    for (int half = 0; half < 2 / T::KG; ++half) {
      const int kk = T::KG == 2 ? kg : half;
      bf16x8_t af[2][kFM], bf[2][kFN];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        B.template read<kFN>(lb + w * kPieceB, (T::TN / WN) * wn, kk, bf[w]);
        A.template read<kFM>(la + w * kPieceA, (T::TM / WM) * wm, kk, af[w]);
      }
      auto mma = [&](int x, int y) {
#pragma unroll
        for (int i = 0; i < kFM; ++i)
#pragma unroll
          for (int j = 0; j < kFN; ++j) acc[i][j] = KindF16::mma(bf[y][j], af[x][i], acc[i][j]);
      };
      mma(0, 0);
      if constexpr (TERMS == 2) {
        mma(0, 1);
        mma(1, 0);
      } else {
        if (2 * s + 1 < steps) mma(1, 1);
      }
    }
    now = now + 1 == T::kRing ? 0 : now + 1;
    free = free + 1 == T::kRing ? 0 : free + 1;
  }
}

// ---- the steps' products ------------------------------------------------------------------

enum Stage { kGram, kPoly, kApply, kApplyPast, kLast };  // kApplyPast: X goes past the caches

struct Step {
  Mats mats;                // of the first matrix
  int64_t a_step, b_step;   // words from one matrix to the next
  int tiles;                // per matrix
  Planes in, out;           // kPoly: A -> P;  kApply: X -> X;  kGram: -> A;  kLast: X
  float* gram_diag;         // [matrix][M] A's diagonal (0 in its planes): written by kGram, read by kPoly
  float* diag;              // [matrix][M] P's diagonal (0 in its planes): written by kPoly, read by kApply and kLast
  float a, b, c;            // b and c take A's scale to P's
  void* o;                  // kLast: [matrix][rows][cols], where X is [cols][rows] if `turned`
  int o_bf16, turned, rows, cols;
};

// One tile of one matrix.  SYM stages compute the tiles on and above the diagonal.
//
// What bounds it, per launch: for one 4,096 x 4,096 matrix the matrix units (A 73 to 77 us and P 75 to 79 on 192 x 192 tiles,
// 22 x 23 / 2 of them in one round, 0.95 to 1.05 PFLOP/s; P X 122 to 127 us, 1.13 PFLOP/s) and the epilogue behind them; for 48 of
// 512 x 2,048 memory in P X (X's terms in and out, 409 MB or more in 106 us) and the tiles' loads out of the L2 in A (46 us,
// 480 tiles of which each brings 32 KB per K-step); for one of 512 x 2,048 latency (A 6.6 us, P 3.6, P X 5.5, of 17 launches in a row).
template <typename T, int STAGE, int TERMS>
__global__ __launch_bounds__(T::kThreads, 2) void newton_product_kernel(Step st) {
  constexpr bool SYM = STAGE == kGram || STAGE == kPoly;
  constexpr int TM = T::TM, TN = T::TN, WM = T::WM, WN = T::WN, kFM = T::kFM, kFN = T::kFN, kThreads = T::kThreads;
  __shared__ __attribute__((aligned(16))) uint8_t lds[T::kLds];
  const int forward = die_item(blockIdx.x, gridDim.x);
  const int item = STAGE == kApplyPast ? (int)gridDim.x - 1 - forward : forward;
  const int matrix = uniform(item / st.tiles), t = uniform(item - matrix * st.tiles);
  Mats p = st.mats;
  p.A += matrix * st.a_step;
  p.B += matrix * st.b_step;
  int m0, n0;
  if constexpr (SYM) {  // column j of tiles holds j + 1 of them
    static_assert(TM == TN, "square tiles");
    int j = (int)((__builtin_sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while ((j + 1) * (j + 2) / 2 <= t) ++j;
    while (j * (j + 1) / 2 > t) --j;
    n0 = uniform(j * TN);
    m0 = uniform((t - j * (j + 1) / 2) * TM);
  } else {  // bands of 8 row tiles, walked column by column
    const int tm = (p.M + TM - 1) / TM, tn = (p.R + TN - 1) / TN;
    const int band = t / (8 * tn), in_band = t - band * 8 * tn, band_rows = min(8, tm - band * 8);
    m0 = uniform((band * 8 + in_band % band_rows) * TM);
    n0 = uniform(in_band / band_rows * TN);
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int kg = wave / (WM * WN), wm = T::KG == 1 ? wave / WN : wave / WN % WM, wn = wave % WN;
  // Through LDS, so that loads and stores run along rows: 16-byte pieces, piece c of row m at c ^ (m % 16)
  // (of 32 columns, m % 8).
  float* tile_c = reinterpret_cast<float*>(lds);
  constexpr int kPieces = TN / 4, kTurn = std::min(16, kPieces) - 1, kPassRows = TM / T::kPasses, kStep = kThreads / kPieces;
  // What the epilogue reads is loaded before the products where the registers hold it, else four rows ahead.
  constexpr bool kEarly = STAGE != kGram && TM <= 128;
  constexpr int kAhead = kEarly ? kPassRows / kStep : std::min(4, kPassRows / kStep);
  static_assert(kThreads % kPieces == 0 && kPassRows % 32 == 0 && kPassRows % (std::min(4, kAhead) * kStep) == 0, "rows come by 64");
  const int r16 = lane & 15, q = lane >> 4;
  const int ld = p.R;
  const uint16_t* in = st.in.p + matrix * st.in.step;
  uint16_t* out = st.out.p + matrix * st.out.step;
  float* gram_diag = st.gram_diag + (int64_t)matrix * p.M;
  float* diag = st.diag + (int64_t)matrix * p.M;
  const int o = tid % kPieces, n = n0 + 4 * o, r0 = tid / kPieces;
  const bool cols_in = n < p.R;
  uint2 hi[kAhead], lo[kAhead];
  float dg[kAhead];
  float4 dc = make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (STAGE == kPoly) dc = *reinterpret_cast<const float4*>(gram_diag + (cols_in ? n : 0));
  auto ahead = [&](int first) {  // of rows first + k kStep; those past the end read the first row, columns the first ones
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int m = first + k * kStep;
      const uint16_t* at = in + (int64_t)(m < p.M ? m : m0) * ld + (cols_in ? n : 0);
      if constexpr (STAGE != kGram) hi[k] = *reinterpret_cast<const uint2*>(at);
      if constexpr (!SYM || (STAGE == kPoly && TERMS == 2))
        lo[k] = IsPaired<T>::value ? *reinterpret_cast<const uint2*>(at + st.in.plane) : load_once(at + st.in.plane);
      if constexpr (STAGE != kGram) dg[k] = (STAGE == kPoly ? gram_diag : diag)[m < p.M ? m : m0];
    }
  };
  if constexpr (kEarly) ahead(m0 + r0);
  const int steps = p.K / kBK * p.nseg;
  f32x4_t acc[kFM][kFN];
  // rows past the end read the last one and are not stored
  const auto row_a = [&](int r) { return min(m0 + r, p.M - 1) - m0; };
  const auto row_b = [&](int r) { return min(n0 + r, p.R - 1) - n0; };
  if constexpr (IsPaired<T>::value) paired_loop<T, !SYM, TERMS>(p, m0, n0, row_a, row_b, lds, acc);
  else product_loop<T, false, !SYM, 0, KindF16>(p, m0, n0, 0, steps, row_a, row_b, lds, acc);

#pragma unroll
  for (int pass = 0; pass < T::kPasses; ++pass) {
    hand_over();
    auto put = [&](auto add) {
#pragma unroll
      for (int i = 0; i < kFM; ++i)
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
          const int m = (T::kPasses == 1 ? (TM / WM) * wm : 0) + 16 * i + r16, c = (TN / WN / 4) * wn + 4 * j + q;
          f32x4_t* at = reinterpret_cast<f32x4_t*>(tile_c + (m * kPieces + (c ^ (m & kTurn))) * 4);
          *at = decltype(add)::value ? acc[i][j] + *at : acc[i][j];
        }
    };
    static_assert(T::KG == 1 || T::kPasses == 1, "groups of waves are added once");
    if constexpr (T::KG == 2) {
      if (kg == 1) put(std::false_type{});
      hand_over();
      if (kg == 0) put(std::true_type{});
    } else {
      if (T::kPasses == 1 || wm == pass) put(std::false_type{});
    }
    hand_over();
    const int mp = m0 + pass * kPassRows;       // the pass's first row
    const int rows = min(kPassRows, p.M - mp);  // (a multiple of 64, or below 1)
    const bool mirrored = (SYM && m0 != n0) || (STAGE == kLast && st.turned);
    for (int d = r0; d < rows; d += kAhead * kStep) {
      if constexpr (!kEarly) ahead(mp + d);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = d + k * kStep, m = mp + r;
        if (kEarly && r >= rows) break;
        float4* at = reinterpret_cast<float4*>(tile_c + (r * kPieces + (o ^ (r & kTurn))) * 4);
        const float4 s = *at;
        const float z[4] = {s.x, s.y, s.z, s.w};
        float h[4], l[4], v[4];
        if constexpr (STAGE != kGram) unpack4(hi[k], h);
        if constexpr (!SYM || (STAGE == kPoly && TERMS == 2)) unpack4(lo[k], l);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (STAGE == kGram) {
            v[e] = z[e] * (kGScale / (kXScale * kXScale));
            if (m == n + e) {
              gram_diag[m] = v[e] * (1.0f / kGScale);
              v[e] = 0.0f;
            }
          } else if constexpr (STAGE == kPoly) {
            // A = E + D with E off the diagonal: A^2 = E^2 + D E + E D + D^2
            float g = TERMS == 2 ? h[e] + l[e] : h[e];
            float sq = __builtin_fmaf(g, dg[k] + (e == 0 ? dc.x : e == 1 ? dc.y : e == 2 ? dc.z : dc.w), z[e] * (1.0f / kGScale));
            if (m == n + e) {
              g = kGScale * dg[k];
              sq = __builtin_fmaf(g, dg[k], sq);
            }
            v[e] = __builtin_fmaf(st.b, g, st.c * sq);
            if (m == n + e) {
              diag[m] = v[e] * (1.0f / kPScale);
              v[e] = 0.0f;
            }
          } else {
            const float x = h[e] + l[e], by = TERMS == 2 ? x : h[e];
            v[e] = __builtin_fmaf(st.a, x, __builtin_fmaf(dg[k], by, z[e] * (1.0f / kPScale)));
          }
        }
        if constexpr (STAGE == kLast) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= 1.0f / kXScale;
        }
        if (mirrored) *at = make_float4(v[0], v[1], v[2], v[3]);
        if constexpr (STAGE == kLast) {
          if (!st.turned && m < st.rows) {
            const size_t i = ((size_t)matrix * st.rows + m) * st.cols + n;
            if (n + 4 <= st.cols) {
              store4(st.o, st.o_bf16, i, v);
            } else {
#pragma unroll
              for (int e = 0; e < 3; ++e)
                if (n + e < st.cols) store_any(st.o, st.o_bf16, i + e, v[e]);
            }
          }
        } else if (cols_in) {
          uint2 a, b;
          terms4(v, a, b);
          uint16_t* to = out + (int64_t)m * ld + n;
          if constexpr (STAGE == kApplyPast) {
            store_past(to, a);
            store_past(to + st.out.plane, b);
          } else {
            *reinterpret_cast<uint2*>(to) = a;
            if constexpr (STAGE == kApply || TERMS == 2) *reinterpret_cast<uint2*>(to + st.out.plane) = b;
          }
        }
      }
    }
    if constexpr (SYM || STAGE == kLast) {
      if (mirrored) {  // the tile's transpose: a thread takes four rows of a column
        hand_over();
        constexpr int kRowPieces = kPassRows / 4;
        static_assert(kThreads % kRowPieces == 0, "rows per thread");
        const int rq = tid % kRowPieces * 4, m = mp + rq;
        for (int c = tid / kRowPieces; c < TN; c += kThreads / kRowPieces) {
          if (rq >= rows || n0 + c >= p.R) continue;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = tile_c[((rq + e) * kPieces + ((c >> 2) ^ ((rq + e) & kTurn))) * 4 + (c & 3)];
          if constexpr (STAGE == kLast) {
            if (n0 + c < st.rows) {
              const size_t i = ((size_t)matrix * st.rows + n0 + c) * st.cols + m;
              if (m + 4 <= st.cols) {
                store4(st.o, st.o_bf16, i, v);
              } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                  if (m + e < st.cols) store_any(st.o, st.o_bf16, i + e, v[e]);
              }
            }
          } else {
            uint2 a, b;
            terms4(v, a, b);
            uint16_t* to = out + (int64_t)(n0 + c) * ld + m;
            *reinterpret_cast<uint2*>(to) = a;
            if constexpr (TERMS == 2) *reinterpret_cast<uint2*>(to + st.out.plane) = b;
          }
        }
      }
    }
  }
}

// ---- sizes ------------------------------------------------------------------------------------

size_t up256(size_t v) { return (v + 255) / 256 * 256; }
int up64(int v) { return (v + 63) / 64 * 64; }

// Shapes; the last two are Mid and Nano in symmetric products, Flat (twice) in P X.
enum { kTiny, kSmall, kLarge, kWide, kMid, kNano, kShapes };

// Time of a launch in microseconds, from traces of 1 to 4,096 tiles of 2 to 64 K-steps: a workgroup costs a start and an
// epilogue (most of a short reduction's time) and its K-steps, less of each while it has a CU to itself.
//   P X, 8 K-steps (48 matrices of 512 x 2,048): 128 x 128 tiles 124 us, 256 x 256 114; of 8 matrices 21 and 26, 64 x 64 27
//   P X, 5 K-steps (24 matrices of 300 x 700): 64 x 64 18 us, 128 x 128 16 (64 x 128 14, not built)
//   A, 64 K-steps of 4,096 x 4,096: 64 x 64 168 us, 128 x 128 110, 192 x 192 77, 256 x 256 108
//   A, 32 K-steps of 512 x 2,048: Nano 7.6 us, 64 x 64 10.5, 128 x 128 25.8
struct Rates {
  int rows, cols, slots;           // of a tile; workgroups at once
  double start, step;              // with the slots taken
  double start_alone, step_alone;  // up to half of them
};
// A paired shape's step is 64 k of all terms, by one term and by two; the others take each pass of the terms by itself.
constexpr Rates kSymRates[2][kShapes] = {
    {{64, 64, 512, 5.0, 0.42, 4.5, 0.19}, {128, 128, 512, 18.0, 1.12, 12.0, 0.43}, {256, 256, 256, 28.0, 1.30, 24.0, 1.07},
     {64, 64, 256, 5.4, 0.18, 5.4, 0.18}, {192, 192, 256, 14.0, 1.00, 12.5, 0.65}, {32, 32, 768, 4.5, 0.25, 3.3, 0.13}},
    {{64, 64, 512, 5.0, 0.42, 4.5, 0.19}, {128, 128, 512, 18.0, 1.12, 12.0, 0.43}, {256, 256, 256, 28.0, 1.30, 24.0, 1.07},
     {64, 64, 256, 5.4, 0.36, 5.4, 0.36}, {192, 192, 256, 14.0, 1.00, 12.5, 0.65}, {32, 32, 768, 5.5, 0.38, 3.6, 0.20}}};
constexpr Rates kApplyRates[2][kShapes - 1] = {
    {{64, 64, 512, 4.3, 0.40, 4.2, 0.20}, {128, 128, 512, 12.5, 0.97, 9.0, 0.68}, {256, 256, 256, 25.0, 1.60, 17.0, 1.18},
     {64, 64, 256, 3.5, 0.28, 4.0, 0.20}, {32, 64, 512, 3.4, 0.40, 3.4, 0.20}},
    {{64, 64, 512, 4.3, 0.40, 4.2, 0.20}, {128, 128, 512, 12.5, 0.97, 9.0, 0.68}, {256, 256, 256, 25.0, 1.60, 17.0, 1.18},
     {64, 64, 256, 4.2, 0.45, 4.2, 0.40}, {32, 64, 512, 3.8, 0.68, 3.8, 0.30}}};
double launch_cost(const Rates& r, int64_t tiles, int64_t steps) {
  const int64_t whole = tiles / r.slots, rest = tiles % r.slots;
  const double full = r.start + r.step * steps, alone = r.start_alone + r.step_alone * steps;
  return whole * full + (rest == 0 ? 0.0 : rest <= r.slots / 2 ? alone : full);
}

int64_t triangle(int64_t t) { return t * (t + 1) / 2; }

struct NewtonPlan {
  int m, n;           // padded
  int terms, blocks;  // fp16 terms of products; workgroups of the norm per matrix
  int shape[2];       // tile shapes of the symmetric products (A and P alike) and of P X
  size_t xa, xb, gram, poly, gram_diag, diag, parts, bytes;
};
const Rates& rates_of(const NewtonPlan& p, bool sym, int shape) {
  return sym ? kSymRates[p.terms - 1][shape] : kApplyRates[p.terms - 1][std::min(shape, kShapes - 2)];
}
int64_t newton_tiles(const NewtonPlan& p, bool sym, int shape) {
  const Rates& r = rates_of(p, sym, shape);
  const int64_t tm = ceil_div(p.m, r.rows);
  return sym ? triangle(tm) : tm * ceil_div(p.n, r.cols);
}
NewtonPlan newton_plan(int64_t B, int R, int K, moe_dtype o_t) {
  NewtonPlan p{};
  p.m = up64(std::min(R, K));
  p.n = up64(std::max(R, K));
  p.terms = o_t == MOE_F32 ? 2 : 1;
  p.blocks = (int)std::min<int64_t>(kNormBlocks, ceil_div((int64_t)R * K, kNormValues));
  for (int sym = 0; sym < 2; ++sym) {
    double least = 0;
    for (int shape = 0; shape < kShapes - !sym; ++shape) {
      const Rates& r = rates_of(p, sym, shape);
      const int64_t tiles = B * newton_tiles(p, sym, shape);
      const int64_t passes = p.terms == 2 && !(shape == kWide || shape == kNano || (!sym && shape > kWide)) ? 3 : 1;
      double c = launch_cost(r, tiles, passes * p.m / kBK);
      if (sym) c += launch_cost(r, tiles, passes * p.n / kBK);  // A's and P's products share a choice
      if (least == 0 || c < least) {
        least = c;
        p.shape[sym ? 0 : 1] = shape;
      }
    }
  }
  size_t o = 0;
  const size_t x = (size_t)B * p.m * p.n * 2, s = (size_t)B * p.m * p.m * 2;
  p.xa = o; o = up256(o + 2 * x);
  p.xb = o; o = up256(o + 2 * x);
  p.gram = o; o = up256(o + p.terms * s);
  p.poly = o; o = up256(o + p.terms * s);
  p.gram_diag = o; o = up256(o + (size_t)B * p.m * 4);
  p.diag = o; o = up256(o + (size_t)B * p.m * 4);
  p.parts = o; o = up256(o + (size_t)B * p.blocks * 8);
  p.bytes = o;
  return p;
}

template <int STAGE>
moe_status launch_stage(const NewtonPlan& pl, int64_t B, Step st, hipStream_t s) {
  const int shape = pl.shape[STAGE == kGram || STAGE == kPoly ? 0 : 1];
  st.tiles = (int)newton_tiles(pl, STAGE == kGram || STAGE == kPoly, shape);
  const dim3 grid((unsigned)(B * st.tiles));
  auto go = [&](auto tile) {
    using T = decltype(tile);
    const dim3 threads((unsigned)T::kThreads);
    if (pl.terms == 2) launch_k(MOE_KERNEL_ORTHOGONALIZE, newton_product_kernel<T, STAGE, 2>, grid, threads, 0, s, st);
    else launch_k(MOE_KERNEL_ORTHOGONALIZE, newton_product_kernel<T, STAGE, 1>, grid, threads, 0, s, st);
  };
  if (shape == kTiny) go(Tiny{});
  else if (shape == kSmall) go(Small{});
  else if (shape == kLarge) go(Large{});
  else if (shape == kWide) go(Wide{});
  else if constexpr (STAGE == kGram || STAGE == kPoly) shape == kMid ? go(Mid{}) : go(Nano{});
  else go(Flat{});
  return check_launch("orthogonalize");
}

}  // namespace

// (which way a call takes depends on its coefficients, which the query does not know)
size_t orthogonalize_ws_bytes(int B, int R, int K, moe_dtype o_t) {
  return std::max(newton_plan(B, R, K, o_t).bytes, newton_small_ws_bytes(B, R, K));
}

void orthogonalize_form(int B, int R, int K, moe_dtype o_t, int32_t form[4]) {
  if (newton_is_small(R, K, 5, nullptr)) {
    form[0] = form[1] = form[2] = form[3] = 0;
    return;
  }
  const NewtonPlan p = newton_plan(B, R, K, o_t);
  form[0] = rates_of(p, true, p.shape[0]).rows;
  form[1] = rates_of(p, false, p.shape[1]).rows;
  form[2] = p.shape[0] == kWide || p.shape[0] == kNano;
  form[3] = p.shape[1] >= kWide;
}

moe_status launch_orthogonalize(const void* g, moe_dtype g_t, float* momentum, double beta, int nesterov, int B, int R, int K,
                                int steps, const float* coef, double eps, void* o, moe_dtype o_t, void* ws, hipStream_t s) {
  const Update u{g, momentum, g_t == MOE_BF16, nesterov, (float)beta, (float)(1.0 - beta), R, K};
  if (newton_is_small(R, K, steps, coef)) return launch_newton_small(u, B, steps, coef, eps, o, o_t, ws, s);
  const NewtonPlan pl = newton_plan(B, R, K, o_t);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  const int64_t xs = (int64_t)pl.m * pl.n, gs = (int64_t)pl.m * pl.m;
  auto planes = [&](size_t at, int64_t step) { return Planes{reinterpret_cast<uint16_t*>(base + at), B * step, step}; };
  Planes x = planes(pl.xa, xs), next = planes(pl.xb, xs);
  const Planes gram = planes(pl.gram, gs), poly = planes(pl.poly, gs);
  double* parts = reinterpret_cast<double*>(base + pl.parts);
  newton_moment_kernel<<<dim3((unsigned)((int64_t)B * pl.blocks)), 256, 0, s>>>(u, pl.blocks, parts);
  if (moe_status st = check_launch("orthogonalize")) return st;
  const int tr = (int)ceil_div(R, 64), tk = (int)ceil_div(K, 64);
  newton_start_kernel<<<dim3((unsigned)((int64_t)B * tr * tk)), 256, 0, s>>>(u, pl.blocks, parts, eps, tr, tk, x, pl.n);
  if (moe_status st = check_launch("orthogonalize")) return st;

  Step st{};
  // the passes of two terms: first x first, first x second, second x first
  st.mats.nseg = pl.terms == 2 ? 3 : 1;
  st.mats.sa = 1u << 4;
  st.mats.sb = 1u << 2;
  st.mats.M = pl.m;
  st.gram_diag = reinterpret_cast<float*>(base + pl.gram_diag);
  st.diag = reinterpret_cast<float*>(base + pl.diag);
  st.o = o;
  st.o_bf16 = o_t == MOE_BF16;
  st.turned = R > K;
  st.rows = R;
  st.cols = K;
  auto operands = [&](const Planes& a, int lda, const Planes& b, int ldb, int cols, int k) {
    st.mats.A = a.p;
    st.mats.B = b.p;
    st.mats.a_plane = a.plane;
    st.mats.b_plane = b.plane;
    st.mats.lda = lda;
    st.mats.ldb = ldb;
    st.mats.R = cols;
    st.mats.K = k;
    st.a_step = a.step;
    st.b_step = b.step;
  };
  const bool past = (size_t)B * xs * 8 > kKept;
  for (int i = 0; i < steps; ++i) {
    st.a = coef[3 * i];
    st.b = coef[3 * i + 1] * (kPScale / kGScale);
    st.c = coef[3 * i + 2] * (kPScale / kGScale);
    operands(x, pl.n, x, pl.n, pl.m, pl.n);
    st.in = gram;  // (not read)
    st.out = gram;
    if (moe_status e = launch_stage<kGram>(pl, B, st, s)) return e;
    operands(gram, pl.m, gram, pl.m, pl.m, pl.m);
    st.in = gram;
    st.out = poly;
    if (moe_status e = launch_stage<kPoly>(pl, B, st, s)) return e;
    operands(poly, pl.m, x, pl.n, pl.n, pl.m);
    st.in = x;
    st.out = next;
    if (moe_status e = i + 1 == steps ? launch_stage<kLast>(pl, B, st, s)
                       : past         ? launch_stage<kApplyPast>(pl, B, st, s)
                                      : launch_stage<kApply>(pl, B, st, s))
      return e;
    std::swap(x, next);
  }
  return MOE_OK;
}

}  // namespace moe
