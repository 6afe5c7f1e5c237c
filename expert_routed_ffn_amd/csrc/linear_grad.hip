// linear_grad.hip -- gradient of the dense product y = act(x W^T + b) + residual:
//   dz = dy act'(pre)   (SwiGLU: dz_gate = dy z_up silu'(z_gate), dz_up = dy silu(z_gate))
//   dx = dz W     dW = dz^T x     db = sum_t dz_t     (the residual's gradient is dy itself)
//
// Two launches and, where a reduction was cut, a third:
//   1. prep: dz is computed once from dy and the kept pre-activations and written as bf16 term planes [T][R]; fp32 x
//      becomes term planes too, and each workgroup adds its rows of dz in fp32 for db.  Left out where dy is dz as the
//      products take it (bf16, no activation) and db is not wanted.
//   2. products: both in one launch of the tiled kernel, which reads dz, W and x in place in either direction; db's
//      parts are added in workgroups behind the tiles.
//   3. join: parts of cut reductions, in a fixed order.
// Precision goes by the output's type.  An fp32 dx or dW is computed from operands held exactly: dz, and x where it
// is fp32, enter as three bf16 terms, and products of terms below 2^-24 of the whole are left out.  A bf16 dx or dW
// takes dz as two terms, which leave at most 2^-17 of each value (2^-9 of the half step that rounding the result costs),
// and x, where it is fp32, as two, so that the result carries its own rounding and no other that shows.  (One term is off
// by up to 2^-8 of each value: the error of a chunk's dx was 2.34e-3 of its norm then, against 1.66e-3.  8,192 x 512
// SwiGLU: 91 us with one term, 145 with two; the router's gradient 93 and 117.)
#include <algorithm>

#include "linear_dev.hpp"

namespace moe {
namespace {

// Of dy per workgroup: 32 threads of 8 columns by 8 rows at a time, up to 64 rows; fewer where that leaves less than 512
// workgroups (8,192 x 512 SwiGLU in one plane: 11.5 us with 32 rows, half as long again with 64, 14.6 in the two planes of
// a bf16 result; 333 x 201: 5.1 us with 8, five times that with 64).
constexpr int kPrepCols = 256;
int prep_rows(int T, int N) {
  int rows = 64;
  while (rows > 8 && ceil_div(T, rows) * ceil_div(N, kPrepCols) < 512) rows /= 2;
  return rows;
}

struct Prep {
  const void *dy, *pre;
  uint16_t* dz;            // planes [T][ldz], or null
  int64_t dz_plane;
  float* db_part;          // [row tiles][R], or null
  int T, N, R, ldz, terms, rows;
  int act;
  int blocks, tiles_n;
  const float* x;          // fp32 activations to `x_terms` planes, or null
  uint16_t* xt;
  int64_t x_plane, x4;     // plane and number of values / 4
  int x_terms;
};

// Columns i ... i + 8 of a row; without FULL, those past `left` as zeros.
template <bool BF16, bool FULL>
__device__ __forceinline__ void load8(const void* p, size_t i, int left, float (&v)[8]) {
  if constexpr (!FULL) {
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = r < left ? load_any(p, BF16, i + r) : 0.0f;
  } else if constexpr (BF16) {
    const u32x4_at2_t q = *reinterpret_cast<const u32x4_at2_t*>(reinterpret_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      v[2 * r] = __uint_as_float(w[r] << 16);
      v[2 * r + 1] = __uint_as_float(w[r] & 0xFFFF0000u);
    }
  } else {
    float a[4], b[4];
    load4(p, 0, i, a);
    load4(p, 0, i + 4, b);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      v[r] = a[r];
      v[4 + r] = b[r];
    }
  }
}

// Those 8 values as terms at element `at` of each plane.
template <bool FULL>
__device__ __forceinline__ void write8(uint16_t* dst, int64_t plane, int terms, size_t at, int left, const float (&v)[8]) {
  uint16_t t[8][3];
#pragma unroll
  for (int i = 0; i < 8; ++i) bf16_terms(v[i], t[i]);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (k >= terms) continue;
    uint16_t* o = dst + k * plane + at;
    if constexpr (FULL) {
      *reinterpret_cast<u32x4_at2_t*>(o) =
          u32x4_at2_t{t[0][k] | (uint32_t)t[1][k] << 16, t[2][k] | (uint32_t)t[3][k] << 16,
                      t[4][k] | (uint32_t)t[5][k] << 16, t[6][k] | (uint32_t)t[7][k] << 16};
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < left) o[i] = t[i][k];
    }
  }
}

// What dz is made of: dy alone, dy and one pre-activation, or dy and a SwiGLU pair.
enum PrepKind { kPlain, kSlope, kPair };

// One row's 8 columns from n on; of rows shorter than that (not FULL) the `left` that are there.  Everything that decides
// which loads there are is known to the compiler, so that a thread's loads are issued together (decided at run time, each
// was waited for before the next).
template <int KIND, bool BF16, bool FULL>
__device__ __forceinline__ void prep_row(const Prep& p, int t, int n, int left, float (&sa)[8], float (&su)[8]) {
  float g[8], z[8], zu[8], a[8], u[8];
  load8<BF16, FULL>(p.dy, (size_t)t * p.N + n, left, g);
  if constexpr (KIND != kPlain) load8<BF16, FULL>(p.pre, (size_t)t * p.R + n, left, z);
  if constexpr (KIND == kPair) load8<BF16, FULL>(p.pre, (size_t)t * p.R + p.N + n, left, zu);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (KIND == kPair) {
      const float h = sigmoid(z[j]);
      a[j] = g[j] * (zu[j] * (h * __builtin_fmaf(z[j], 1.0f - h, 1.0f)));  // (dy times up may pass fp32's range)
      u[j] = g[j] * (z[j] * h);
    } else if constexpr (KIND == kSlope) {
      a[j] = g[j] * act_slope(p.act, z[j]);
    } else {
      a[j] = g[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {  // (what is not there adds zero)
    sa[j] += a[j];
    if constexpr (KIND == kPair) su[j] += u[j];
  }
  if (!p.dz) return;
  const size_t at = (size_t)t * p.ldz + n;
  write8<FULL>(p.dz, p.dz_plane, p.terms, at, left, a);
  if constexpr (KIND == kPair) write8<FULL>(p.dz, p.dz_plane, p.terms, at + p.N, left, u);
  if (n + 8 >= p.N)  // the last columns' thread also fills the row's padding
    for (int c = p.R; c < p.ldz; ++c)
      for (int k = 0; k < p.terms; ++k) p.dz[k * p.dz_plane + (size_t)t * p.ldz + c] = 0;
}

template <int KIND, bool BF16>
__device__ void prep_dz(const Prep& p, int b, float (&sums)[2][8][kPrepCols]) {
  constexpr bool PAIR = KIND == kPair;
  const int tid = threadIdx.x;
  const int tt = b / p.tiles_n, n0 = (b % p.tiles_n) * kPrepCols;
  // The last columns of rows whose length is no multiple of 8 are the row's last 8: those before its own a thread
  // computes as its neighbour does, writes the same values and leaves out of the sums.  (A path of its own for them took
  // 7.2 us against 5.9 on 333 x 201, as the wave goes through both.)
  const int ry = tid >> 5, own = n0 + (tid & 31) * 8, n = p.N < 8 ? own : min(own, p.N - 8);
  const int t_first = tt * p.rows + ry, t_end = min(p.T, (tt + 1) * p.rows);
  float sa[8], su[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sa[j] = su[j] = 0.0f;
  if (own < p.N) {
    for (int t = t_first; t < t_end; t += 8) {
      if (p.N >= 8) prep_row<KIND, BF16, true>(p, t, n, 8, sa, su);
      else prep_row<KIND, BF16, false>(p, t, n, p.N, sa, su);
    }
  }
  if (!p.db_part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (n + j >= own && n + j < n0 + kPrepCols) {
      sums[0][ry][n - n0 + j] = sa[j];
      if (PAIR) sums[1][ry][n - n0 + j] = su[j];
    }
  }
  __syncthreads();
#pragma unroll
  for (int half = 0; half < (PAIR ? 2 : 1); ++half) {
    float v = sums[half][0][tid];
#pragma unroll
    for (int r = 1; r < 8; ++r) v += sums[half][r][tid];
    if (n0 + tid < p.N) p.db_part[(size_t)tt * p.R + half * p.N + n0 + tid] = v;
  }
}

template <int KIND, bool BF16>
__global__ __launch_bounds__(256) void linear_prep_kernel(Prep p) {
  __shared__ float sums[2][8][kPrepCols];
  if ((int)blockIdx.x < p.blocks) {
    prep_dz<KIND, BF16>(p, blockIdx.x, sums);
    return;
  }
  const int64_t step = (int64_t)(gridDim.x - p.blocks) * 256;
  for (int64_t i = (int64_t)(blockIdx.x - p.blocks) * 256 + threadIdx.x; i < p.x4; i += step) {
    if (p.x_terms == 2) write_terms<2>(p.x, i, p.xt, p.x_plane);
    else write_terms<3>(p.x, i, p.xt, p.x_plane);
  }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Which terms of the two operands meet: (a, b) pairs whose size reaches 2^-24 of the whole with three terms each,
// 2^-16 with two.
int segments(int ta, int tb, uint32_t& sa, uint32_t& sb) {
  const int most = std::max(ta, tb) - 1;
  int n = 0;
  sa = sb = 0;
  for (int sum = 0; sum <= most; ++sum)
    for (int a = 0; a <= sum && a < ta; ++a)
      if (sum - a < tb) {
        sa |= (uint32_t)a << (2 * n);
        sb |= (uint32_t)(sum - a) << (2 * n);
        ++n;
      }
  return n;
}

struct GradPlan {
  int R, ldr;              // product columns, and those rounded up to 8
  bool dx, dw, db, direct; // direct: dy is dz as the products take it
  int dx_terms, dw_terms, terms, x_terms;
  int segs_dx, segs_dw;
  uint32_t dx_sa, dx_sb, dw_sa, dw_sb;
  Plan plan;               // dW first where both are there
  int split_dx, split_dw, tiles_t;
  size_t dz, xt, part_dx, part_dw, db_part, bytes;
};

GradPlan grad_plan(int T, int K, int N, int act, moe_dtype dy_t, moe_dtype x_t, moe_dtype dx_t, moe_dtype dw_t,
                   int need) {
  GradPlan p{};
  p.R = act == MOE_ACT_SWIGLU ? 2 * N : N;
  p.ldr = (int)(ceil_div(p.R, 8) * 8);
  p.tiles_t = (int)ceil_div(T, prep_rows(T, N));
  p.dx = need & MOE_NEED_DX;
  p.dw = need & MOE_NEED_DW;
  p.db = need & MOE_NEED_DB;
  const bool one = act == MOE_ACT_NONE && dy_t == MOE_BF16;  // dz is dy: one term holds it
  p.dx_terms = one ? 1 : dx_t == MOE_BF16 ? 2 : 3;
  p.dw_terms = one ? 1 : dw_t == MOE_BF16 ? 2 : 3;
  p.terms = std::max(p.dx ? p.dx_terms : 1, p.dw ? p.dw_terms : 1);
  p.x_terms = x_t == MOE_BF16 ? 1 : dw_t == MOE_F32 ? 3 : 2;
  // (the products load 16 bytes of a row at a time)
  p.direct = one && p.R % 8 == 0;
  p.segs_dx = segments(p.dx_terms, 1, p.dx_sa, p.dx_sb);
  p.segs_dw = segments(p.dw_terms, p.x_terms, p.dw_sa, p.dw_sb);
  Shape s[2];
  int count = 0;
  if (p.dw) s[count++] = Shape{p.R, K, T, p.segs_dw};
  if (p.dx) s[count++] = Shape{T, K, p.R, p.segs_dx};
  if (count) p.plan = plan_products(s, count);
  p.split_dw = p.dw ? p.plan.split[0] : 1;
  p.split_dx = p.dx ? p.plan.split[count - 1] : 1;
  size_t o = 0;
  auto take = [&](bool want, size_t bytes) {
    const size_t at = o;
    if (want) o = up256(o + bytes);
    return at;
  };
  // dz's place is kept where dy could be taken directly, too: whether it can depends on its address as well
  p.dz = take(p.dx || p.dw, (size_t)p.terms * T * p.ldr * 2);
  p.xt = take(p.dw && x_t == MOE_F32, (size_t)p.x_terms * T * K * 2);
  p.part_dx = take(p.dx && p.split_dx > 1, (size_t)p.split_dx * T * K * 4);
  p.part_dw = take(p.dw && p.split_dw > 1, (size_t)p.split_dw * p.R * K * 4);
  p.db_part = take(p.db, (size_t)p.tiles_t * p.R * 4);
  p.bytes = o;
  return p;
}

__global__ __launch_bounds__(256) void zero_kernel(uint16_t* dw, int64_t n, float* db, int64_t m) {
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  for (int64_t i = i0; i < n; i += step) dw[i] = 0;
  for (int64_t i = i0; i < m; i += step) db[i] = 0.0f;
}

}  // namespace

size_t linear_backward_ws_bytes(int T, int K, int N, int act, moe_dtype dy_t, moe_dtype x_t, moe_dtype dx_t,
                                moe_dtype dw_t, int need) {
  return grad_plan(T, K, N, act, dy_t, x_t, dx_t, dw_t, need).bytes;
}

void linear_backward_form(int T, int K, int N, int act, moe_dtype dy_t, moe_dtype x_t, moe_dtype dx_t, moe_dtype dw_t,
                          int need, int32_t form[4]) {
  const GradPlan p = grad_plan(T, K, N, act, dy_t, x_t, dx_t, dw_t, need);
  form[0] = p.dx || p.dw ? tile_side(p.plan) : 0;
  form[1] = p.dw ? p.split_dw : 0;
  form[2] = p.dx ? p.split_dx : 0;
  form[3] = p.terms;
}

moe_status launch_linear_backward(const void* dy, moe_dtype dy_t, const void* pre, const void* x, moe_dtype x_t,
                                  const uint16_t* w, int act, int T, int K, int N, void* dx, moe_dtype dx_t, void* dw,
                                  moe_dtype dw_t, float* db, void* ws, hipStream_t s) {
  const int need = (dx ? MOE_NEED_DX : 0) | (dw ? MOE_NEED_DW : 0) | (db ? MOE_NEED_DB : 0);
  const GradPlan pl = grad_plan(T, K, N, act, dy_t, x_t, dx_t, dw_t, need);
  if (T == 0) {  // no rows: the sums over them are zero
    const int64_t n = dw ? (int64_t)pl.R * K * (dw_t == MOE_F32 ? 2 : 1) : 0, m = db ? pl.R : 0;
    if (n + m == 0) return MOE_OK;
    zero_kernel<<<dim3((unsigned)std::min<int64_t>(1024, ceil_div(std::max(n, m), 256))), 256, 0, s>>>(
        reinterpret_cast<uint16_t*>(dw), n, db, m);
    return check_launch("linear_backward");
  }
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  auto u16 = [&](size_t o) { return reinterpret_cast<uint16_t*>(base + o); };
  auto f32 = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
  const bool direct = pl.direct && reinterpret_cast<uintptr_t>(dy) % 16 == 0;
  Prep p{};
  p.dy = dy;
  p.pre = pre;
  p.T = T;
  p.N = N;
  p.R = pl.R;
  p.act = act;
  p.ldz = pl.ldr;
  p.terms = pl.terms;
  p.rows = prep_rows(T, N);
  p.dz_plane = (int64_t)T * pl.ldr;
  if ((pl.dx || pl.dw) && !direct) p.dz = u16(pl.dz);
  if (pl.db) p.db_part = f32(pl.db_part);
  p.tiles_n = (int)ceil_div(N, kPrepCols);
  const int64_t blocks = p.dz || p.db_part ? (int64_t)p.tiles_n * pl.tiles_t : 0;
  int64_t x_blocks = 0;
  if (pl.dw && x_t == MOE_F32) {
    p.x = reinterpret_cast<const float*>(x);
    p.xt = u16(pl.xt);
    p.x_plane = (int64_t)T * K;
    p.x4 = p.x_plane / 4;
    p.x_terms = pl.x_terms;
    x_blocks = std::min<int64_t>(2048, ceil_div(p.x4, 256));
  }
  if (blocks > 0x7FFF0000) return fail(MOE_EUNSUPPORTED, "moe_linear_backward: too many tiles");
  p.blocks = (int)blocks;
  if (blocks + x_blocks > 0) {
    const dim3 grid((unsigned)(blocks + x_blocks));
    auto go = [&](auto kernel) { kernel<<<grid, 256, 0, s>>>(p); };
    const bool bf16 = dy_t == MOE_BF16;
    if (act == MOE_ACT_SWIGLU) bf16 ? go(linear_prep_kernel<kPair, true>) : go(linear_prep_kernel<kPair, false>);
    else if (act == MOE_ACT_NONE) bf16 ? go(linear_prep_kernel<kPlain, true>) : go(linear_prep_kernel<kPlain, false>);
    else bf16 ? go(linear_prep_kernel<kSlope, true>) : go(linear_prep_kernel<kSlope, false>);
    if (moe_status st = check_launch("linear_backward")) return st;
  }

  const uint16_t* dz = direct ? reinterpret_cast<const uint16_t*>(dy) : p.dz;
  Prob g[2];
  int count = 0;
  auto product = [&](const uint16_t* B, int64_t b_plane, int M, int red, int nseg, uint32_t sa, uint32_t sb, int split,
                     float* partial, void* out, moe_dtype out_t) {
    Prob q{};
    q.A = dz;
    q.a_plane = p.dz_plane;
    q.lda = pl.ldr;
    q.B = B;
    q.b_plane = b_plane;
    q.ldb = K;
    q.M = M;
    q.R = K;
    q.K = red;
    q.nseg = nseg;
    q.sa = sa;
    q.sb = sb;
    q.split = split;
    q.partial = partial;
    q.ldp = K;
    q.epi = Epi{nullptr, nullptr, out, nullptr, K, K, MOE_ACT_NONE, 0, out_t == MOE_BF16};
    g[count++] = q;
  };
  if (pl.dw)
    product(p.x ? p.xt : reinterpret_cast<const uint16_t*>(x), p.x_plane, pl.R, T, pl.segs_dw, pl.dw_sa, pl.dw_sb,
            pl.split_dw, f32(pl.part_dw), dw, dw_t);
  if (pl.dx) product(w, 0, T, pl.R, pl.segs_dx, pl.dx_sa, pl.dx_sb, pl.split_dx, f32(pl.part_dx), dx, dx_t);
  if (count == 0 && !db) return MOE_OK;
  return launch_products(MOE_KERNEL_LINEAR_BACKWARD, pl.plan, g, count, true, pl.dw, DbSum{p.db_part, db, pl.tiles_t, pl.R},
                         s, "linear_backward");
}

}  // namespace moe
