// linear.hip -- dense product with bias, activation and residual in its epilogue:
//   z = x W^T + b,  y = act(z) + residual,  SwiGLU: y = silu(z_gate) z_up + residual with W's first N rows the gate.
//
// Up to 64 tokens: linear_few_kernel, weights straight from memory into matrix operands, the reduction split over the
// waves of a workgroup.  More: product_kernel, a tiled product through LDS.  Sums in fp32.  fp32 activations enter
// as bf16 terms (bf16_terms in linear_dev.hpp): three, which hold them exactly, when y is fp32; one, a rounding by at
// most 2^-9 relative that y's own rounding to bf16 matches, when y is bf16 and the product is tiled.
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
// Wave w works through its eighth of the K-steps with the loads of U steps in flight, then the eight sums of an
// element are added through LDS in wave order.  Rows of W past R and tokens past T read the last valid one and are
// not stored.
template <bool XF32, int TF>
__global__ __launch_bounds__(64 * kFewWaves) void linear_few_kernel(const void* __restrict__ x,
                                                                    const uint16_t* __restrict__ w, int T, int K, Epi e) {
  constexpr int U = TF == 4 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) float red[kFewWaves][TF][64][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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

  f32x4_t acc[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int steps = K / 32;
  const int s0 = steps * wave / kFewWaves, s1 = steps * (wave + 1) / kFewWaves;
  for (int s = s0; s < s1; s += U) {
    uint4 wv[U];
    FewX<XF32> xv[U][TF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u < s1) {
        wv[u] = *reinterpret_cast<const uint4*>(wrow + (s + u) * 32);
#pragma unroll
        for (int f = 0; f < TF; ++f) xv[u][f].load(x, xoff[f] + (size_t)(s + u) * 32);
      } else {
        wv[u] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int f = 0; f < TF; ++f) xv[u][f].zero();
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bf16x8_t wf = __builtin_bit_cast(bf16x8_t, wv[u]);
#pragma unroll
      for (int f = 0; f < TF; ++f) {
        if constexpr (XF32) {
          const float v[8] = {xv[u][f].a.x, xv[u][f].a.y, xv[u][f].a.z, xv[u][f].a.w,
                              xv[u][f].b.x, xv[u][f].b.y, xv[u][f].b.z, xv[u][f].b.w};
          uint16_t t[8][3];
#pragma unroll
          for (int i = 0; i < 8; ++i) bf16_terms(v[i], t[i]);
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            uint4 p;
            p.x = t[0][q] | (uint32_t)t[1][q] << 16;
            p.y = t[2][q] | (uint32_t)t[3][q] << 16;
            p.z = t[4][q] | (uint32_t)t[5][q] << 16;
            p.w = t[6][q] | (uint32_t)t[7][q] << 16;
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8_t, p), acc[f], 0, 0, 0);
          }
        } else {
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8_t, xv[u][f].q), acc[f], 0, 0, 0);
        }
      }
    }
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
  for (int i = threadIdx.x; i < TF * 256; i += 64 * kFewWaves) {
    const int r = i & 15, tk = (i >> 4) & 15, f = i >> 8;
    const int t = 16 * f + tk;
    if (t >= T) continue;
    if (pair) {
      const int n = blockIdx.x * 8 + r;
      if (r < 8 && n < e.N) epi_one(e, t, n, total(f, r, tk), total(f, r + 8, tk));
    } else {
      const int n = blockIdx.x * 16 + r;
      if (n < e.N) epi_one(e, t, n, total(f, r, tk), 0.0f);
    }
  }
}

// ---- tiled product ------------------------------------------------------------------------

constexpr int kTM = 128, kTN = 128, kBK = 64;  // rows of A, rows of B, K-step
constexpr int kWM = 2, kWN = 2;                // waves
constexpr int kThreads = 64 * kWM * kWN;
constexpr int kFM = kTM / kWM / 32, kFN = kTN / kWN / 32;  // 32 x 32 fragments per wave
constexpr int kRows = kThreads / 8;                        // tile rows per pass of 16-byte loads
constexpr int kLA = kTM / kRows, kLB = kTN / kRows;
constexpr int kLds = std::max(2 * (kTM + kTN) * kBK * 2, kTM * kTN * 4);  // two buffers; then the fp32 tile

// 128-byte LDS rows of 64 bf16; 16-byte chunk c of row r sits at c ^ (r & 7), so that the 8 rows a fragment read
// takes at one chunk lie in 8 different places.
__device__ __forceinline__ int lds_at(int row, int chunk) { return row * kBK + ((chunk ^ (row & 7)) * 8); }

// Workgroup number to work item: each of the 8 dies (workgroup b runs on die b % 8) gets one contiguous range of
// items, so that neighbouring tiles share its L2.
__device__ __forceinline__ int die_item(int b, int total) {
  const int per = total >> 3, rem = total & 7, x = b & 7;
  return x * per + min(x, rem) + (b >> 3);
}

// Four columns n ... of a part's row, those below N.
__device__ __forceinline__ void put_part(float* out, int n, int N, int vec, const float (&z)[4]) {
  if (vec) {
    if (n < N) *reinterpret_cast<float4*>(out) = make_float4(z[0], z[1], z[2], z[3]);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < N) out[r] = z[r];
  }
}

// PAIR: SwiGLU, whose tiles hold kTN / 2 gate rows of W and the same up rows.
template <bool PAIR>
__global__ __launch_bounds__(kThreads, 2) void product_kernel(Group g) {
  constexpr int kStage = (kTM + kTN) * kBK;  // bf16 values of one buffer
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
  auto lds_a = [&](int buf) { return reinterpret_cast<uint16_t*>(lds) + buf * kStage; };
  auto lds_b = [&](int buf) { return reinterpret_cast<uint16_t*>(lds) + buf * kStage + kTM * kBK; };
  const int which = (int)blockIdx.x >= g.blocks0;
  const Prob& p = g.p[which];
  const int b = which ? blockIdx.x - g.blocks0 : blockIdx.x;
  const int total = which ? gridDim.x - g.blocks0 : g.blocks0;
  constexpr int cols = PAIR ? kTN / 2 : kTN;  // output columns per tile
  const int tm = (p.M + kTM - 1) / kTM, tn = (p.epi.N + cols - 1) / cols;
  const int item = die_item(b, total);
  const int part = item / (tm * tn);
  // tiles in bands of 8 row tiles, walked column by column
  const int tile = item - part * tm * tn;
  const int band = tile / (8 * tn), in_band = tile - band * 8 * tn;
  const int band_rows = min(8, tm - band * 8);
  const int mt = band * 8 + in_band % band_rows, nt = in_band / band_rows;
  const int m0 = mt * kTM, n0 = nt * cols;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / kWN, wn = wave % kWN;
  const int r0 = tid >> 3, ch = tid & 7;
  // offsets from the tile's first row; rows past the end read the last one and are not stored
  uint32_t oa[kLA], ob[kLB];
#pragma unroll
  for (int i = 0; i < kLA; ++i) oa[i] = (uint32_t)(min(m0 + r0 + kRows * i, p.M - 1) - m0) * p.lda + ch * 8;
#pragma unroll
  for (int i = 0; i < kLB; ++i) {
    const int r = r0 + kRows * i;
    constexpr int kW = kTN / kWN, kH = kW / 2;  // PAIR: each wave's rows are kH gate rows, then the kH up rows
    const int n = PAIR ? (r / kW) * kH + r % kH : r;
    const uint32_t up = PAIR && (r % kW) >= kH ? p.epi.N : 0;
    ob[i] = (min(n0 + n, p.epi.N - 1) - n0 + up) * (uint32_t)p.ldb + ch * 8;
  }
  const int seg_steps = (p.K + kBK - 1) / kBK;
  const int steps = seg_steps * p.nseg;
  const int lo = (int)((int64_t)steps * part / p.split), hi = (int)((int64_t)steps * (part + 1) / p.split);

  struct Stage {
    uint4 a[kLA], b[kLB];
  };
  auto load = [&](Stage& st, int step) {
    const int seg = step / seg_steps, k0 = (step - seg * seg_steps) * kBK;
    const uint16_t* A = p.A + ((p.sa >> (2 * seg)) & 3) * p.a_plane + (size_t)m0 * p.lda + k0;
    const uint16_t* B = p.B + ((p.sb >> (2 * seg)) & 3) * p.b_plane + (size_t)n0 * p.ldb + k0;
    if (k0 + kBK <= p.K) {
#pragma unroll
      for (int i = 0; i < kLA; ++i) st.a[i] = *reinterpret_cast<const uint4*>(A + oa[i]);
#pragma unroll
      for (int i = 0; i < kLB; ++i) st.b[i] = *reinterpret_cast<const uint4*>(B + ob[i]);
    } else {
      const bool in = k0 + ch * 8 < p.K;
#pragma unroll
      for (int i = 0; i < kLA; ++i) st.a[i] = in ? *reinterpret_cast<const uint4*>(A + oa[i]) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kLB; ++i) st.b[i] = in ? *reinterpret_cast<const uint4*>(B + ob[i]) : make_uint4(0, 0, 0, 0);
    }
  };
  auto store = [&](const Stage& st, int buf) {
#pragma unroll
    for (int i = 0; i < kLA; ++i) *reinterpret_cast<uint4*>(&lds_a(buf)[lds_at(r0 + kRows * i, ch)]) = st.a[i];
#pragma unroll
    for (int i = 0; i < kLB; ++i) *reinterpret_cast<uint4*>(&lds_b(buf)[lds_at(r0 + kRows * i, ch)]) = st.b[i];
  };
  f32x16_t acc[kFM][kFN];
#pragma unroll
  for (int i = 0; i < kFM; ++i)
#pragma unroll
    for (int j = 0; j < kFN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  const int fr = lane & 31, fh = lane >> 5;
  auto mma = [&](int buf) {
#pragma unroll
    for (int kk = 0; kk < kBK / 16; ++kk) {
      bf16x8_t af[kFM], bf[kFN];
#pragma unroll
      for (int i = 0; i < kFM; ++i)
        af[i] = *reinterpret_cast<const bf16x8_t*>(&lds_a(buf)[lds_at((kTM / kWM) * wm + 32 * i + fr, 2 * kk + fh)]);
#pragma unroll
      for (int j = 0; j < kFN; ++j)
        bf[j] = *reinterpret_cast<const bf16x8_t*>(&lds_b(buf)[lds_at((kTN / kWN) * wn + 32 * j + fr, 2 * kk + fh)]);
#pragma unroll
      for (int i = 0; i < kFM; ++i)
#pragma unroll
        for (int j = 0; j < kFN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
    }
  };

  // step s in LDS while step s + 1 waits in registers for the other buffer; loads past the part's end repeat its last
  if (lo < hi) {
    Stage st;
    load(st, lo);
    store(st, 0);
    load(st, min(lo + 1, hi - 1));
    __syncthreads();
    int buf = 0;
    for (int s = lo; s < hi; ++s, buf ^= 1) {
      store(st, buf ^ 1);
      load(st, min(s + 2, hi - 1));
      mma(buf);
      __syncthreads();
    }
  }

  // The fp32 tile goes through LDS so that a wave's loads and stores of the epilogue run along rows.  A lane holds
  // row lane & 31 of A and rows 8 (v / 4) + 4 (lane / 32) + v % 4 of B: 16-byte pieces, piece c of row m at
  // c ^ (m & 31), so that the 32 rows written at one piece lie in 32 different places.
  float* tile_c = reinterpret_cast<float*>(lds);
  constexpr int kPieces = kTN / 4;
#pragma unroll
  for (int i = 0; i < kFM; ++i)
#pragma unroll
    for (int j = 0; j < kFN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int m = (kTM / kWM) * wm + 32 * i + fr, c = (kTN / kWN / 4) * wn + 8 * j + 2 * q + fh;
        *reinterpret_cast<float4*>(tile_c + (m * kPieces + (c ^ (m & 31))) * 4) =
            make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
      }
  __syncthreads();
  constexpr int kOutPieces = cols / 4;
  const bool split = p.split > 1;
#pragma unroll 2
  for (int i = tid; i < kTM * kOutPieces; i += kThreads) {
    const int r = i / kOutPieces, o = i % kOutPieces;
    const int m = m0 + r, n = n0 + 4 * o;
    if (m >= p.M || n >= p.epi.N) continue;
    constexpr int kH = kTN / kWN / 8;  // pieces of a wave's gate rows
    const int c = PAIR ? (o / kH) * 2 * kH + o % kH : o;
    float z[4], zu[4];
    const float4 q = *reinterpret_cast<const float4*>(tile_c + (r * kPieces + (c ^ (r & 31))) * 4);
    z[0] = q.x; z[1] = q.y; z[2] = q.z; z[3] = q.w;
    if constexpr (PAIR) {
      const float4 u = *reinterpret_cast<const float4*>(tile_c + (r * kPieces + ((c + kH) ^ (r & 31))) * 4);
      zu[0] = u.x; zu[1] = u.y; zu[2] = u.z; zu[3] = u.w;
    }
    if (split) {
      float* out = p.partial + ((size_t)part * p.M + m) * p.ldp + n;
      put_part(out, n, p.epi.N, p.epi.vec, z);
      if constexpr (PAIR) put_part(out + p.epi.N, n, p.epi.N, p.epi.vec, zu);
    } else {
      epi_four(p.epi, m, n, z, zu);
    }
  }
}

// Adds the parts of split products in part order and applies their epilogue; the workgroups after those add the
// column sums' parts.  Four columns per thread.
__global__ __launch_bounds__(256) void join_kernel(Join jn) {
  int b = blockIdx.x;
  if (b < jn.n0 + jn.n1) {
    const Prob& p = jn.p[b >= jn.n0];
    if (b >= jn.n0) b -= jn.n0;
    const int quads = (p.epi.N + 3) >> 2;
    const int64_t i = (int64_t)b * 256 + threadIdx.x;
    if (i >= (int64_t)p.M * quads) return;
    const int m = (int)(i / quads), n = (int)(i - (int64_t)m * quads) * 4;
    const bool pair = p.epi.act == MOE_ACT_SWIGLU;
    float z[4] = {0.f, 0.f, 0.f, 0.f}, zu[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < p.split; ++s) {
      const float* in = p.partial + ((size_t)s * p.M + m) * p.ldp + n;
      if (p.epi.vec) {
        const float4 q = *reinterpret_cast<const float4*>(in);
        z[0] += q.x; z[1] += q.y; z[2] += q.z; z[3] += q.w;
        if (pair) {
          const float4 u = *reinterpret_cast<const float4*>(in + p.epi.N);
          zu[0] += u.x; zu[1] += u.y; zu[2] += u.z; zu[3] += u.w;
        }
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < p.epi.N) {
            z[r] += in[r];
            if (pair) zu[r] += in[p.epi.N + r];
          }
      }
    }
    epi_four(p.epi, m, n, z, zu);
    return;
  }
  const int c = (b - jn.n0 - jn.n1) * 256 + threadIdx.x;
  if (c >= jn.db_n) return;
  float v = 0.0f;
  for (int r = 0; r < jn.db_rows; ++r) v += jn.db_part[(size_t)r * jn.db_n + c];
  jn.db[c] = v;
}

__global__ __launch_bounds__(256) void terms_kernel(const float* __restrict__ x, int64_t n4, uint16_t* __restrict__ planes,
                                                    int64_t plane, int terms) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
    const float4 q = reinterpret_cast<const float4*>(x)[i];
    const float v[4] = {q.x, q.y, q.z, q.w};
    uint16_t t[4][3];
#pragma unroll
    for (int j = 0; j < 4; ++j) bf16_terms(v[j], t[j]);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < terms)
        reinterpret_cast<uint2*>(planes + k * plane)[i] =
            make_uint2(t[0][k] | (uint32_t)t[1][k] << 16, t[2][k] | (uint32_t)t[3][k] << 16);
  }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct LinearPlan {
  bool few;
  int terms, split;
  size_t planes, partial, bytes;  // offsets and size of the workspace
  int R, ldp;
};
LinearPlan linear_plan(int T, int K, int N, int act, moe_dtype x_t, moe_dtype y_t) {
  LinearPlan p{};
  p.R = act == MOE_ACT_SWIGLU ? 2 * N : N;
  p.ldp = (p.R + 3) / 4 * 4;
  p.few = T <= kFewT;
  if (p.few) return p;
  p.terms = x_t == MOE_BF16 ? 1 : y_t == MOE_F32 ? 3 : 1;
  p.split = prob_split(prob_tiles(T, N, act == MOE_ACT_SWIGLU), ceil_div(K, kBK) * p.terms);
  size_t o = 0;
  p.planes = o;
  if (x_t == MOE_F32) o = up256(o + (size_t)p.terms * T * K * 2);
  p.partial = o;
  if (p.split > 1) o = up256(o + (size_t)p.split * T * p.ldp * 4);
  p.bytes = o;
  return p;
}

bool epi_vec(const Epi& e) {
  auto ok = [](const void* q, int bf16) { return reinterpret_cast<uintptr_t>(q) % (bf16 ? 8 : 16) == 0; };
  return e.N % 4 == 0 && ok(e.y, e.y_bf16) && ok(e.pre, e.y_bf16) && ok(e.res, e.res_bf16) && ok(e.bias, 0);
}

}  // namespace

int64_t prob_tiles(int M, int N, bool swiglu) { return ceil_div(M, kTM) * ceil_div(N, swiglu ? kTN / 2 : kTN); }

int prob_split(int64_t tiles, int64_t steps) {
  const int64_t want = 512 / std::max<int64_t>(tiles, 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, steps / 4, 16}));
}

moe_status launch_products(int kid, Group& g, int count, const float* db_part, int db_rows, int db_n, float* db,
                           hipStream_t s, const char* what) {
  int64_t blocks[2] = {0, 0};
  Join j{};
  for (int i = 0; i < count; ++i) {
    Prob& p = g.p[i];
    p.epi.vec = epi_vec(p.epi);
    blocks[i] = prob_tiles(p.M, p.epi.N, p.epi.act == MOE_ACT_SWIGLU) * p.split;
    j.p[i] = p;
    if (p.split > 1) (i ? j.n1 : j.n0) = (int)ceil_div((int64_t)p.M * ((p.epi.N + 3) / 4), 256);
  }
  if (blocks[0] + blocks[1] > 0x7FFFFFFF) return fail(MOE_EUNSUPPORTED, std::string(what) + ": too many tiles");
  g.blocks0 = (int)blocks[0];
  if (count > 0) {
    const dim3 grid((unsigned)(blocks[0] + blocks[1]));
    if (g.p[0].epi.act == MOE_ACT_SWIGLU) launch_k(kid, product_kernel<true>, grid, dim3(kThreads), 0, s, g);
    else launch_k(kid, product_kernel<false>, grid, dim3(kThreads), 0, s, g);
    if (moe_status st = check_launch(what)) return st;
  }
  j.db_part = db_part;
  j.db = db;
  j.db_rows = db_rows;
  j.db_n = db ? db_n : 0;
  const int64_t jb = (int64_t)j.n0 + j.n1 + ceil_div(j.db_n, 256);
  if (jb > 0) {
    join_kernel<<<dim3((unsigned)jb), 256, 0, s>>>(j);
    return check_launch(what);
  }
  return MOE_OK;
}

moe_status launch_terms(const float* x, int64_t n, uint16_t* planes, int64_t plane, int terms, hipStream_t s) {
  const int64_t n4 = n / 4;
  terms_kernel<<<dim3((unsigned)std::min<int64_t>(2048, ceil_div(n4, 256))), 256, 0, s>>>(x, n4, planes, plane, terms);
  return check_launch("linear");
}

size_t linear_ws_bytes(int T, int K, int N, int act, moe_dtype x_t, moe_dtype y_t) {
  return linear_plan(T, K, N, act, x_t, y_t).bytes;
}

moe_status launch_linear(const void* x, moe_dtype x_t, const uint16_t* w, const float* bias, int act,
                         const void* residual, moe_dtype r_t, int T, int K, int N, void* y, moe_dtype y_t, void* pre,
                         void* ws, hipStream_t s) {
  const LinearPlan pl = linear_plan(T, K, N, act, x_t, y_t);
  Epi e{bias, residual, y, pre, N, pl.R, act, r_t == MOE_BF16, y_t == MOE_BF16, 0};
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
  Group g{};
  Prob& p = g.p[0];
  p.A = reinterpret_cast<const uint16_t*>(x);
  if (x_t == MOE_F32) {
    uint16_t* planes = reinterpret_cast<uint16_t*>(base + pl.planes);
    p.a_plane = (int64_t)T * K;
    if (moe_status st = launch_terms(reinterpret_cast<const float*>(x), (int64_t)T * K, planes, p.a_plane, pl.terms, s))
      return st;
    p.A = planes;
  }
  p.B = w;
  p.lda = p.ldb = K;
  p.M = T;
  p.R = pl.R;
  p.K = K;
  p.nseg = pl.terms;
  p.sa = 0 | 1u << 2 | 2u << 4;
  p.sb = 0;
  p.split = pl.split;
  p.partial = reinterpret_cast<float*>(base + pl.partial);
  p.ldp = pl.ldp;
  p.epi = e;
  return launch_products(MOE_KERNEL_LINEAR, g, 1, nullptr, 0, 0, nullptr, s, "linear");
}

}  // namespace moe
