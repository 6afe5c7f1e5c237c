// linear_grad.hip -- gradient of the dense product y = act(x W^T + b) + residual:
//   dz = dy act'(pre)   (SwiGLU: dz_gate = dy z_up silu'(z_gate), dz_up = dy silu(z_gate))
//   dx = dz W     dW = dz^T x     db = sum_t dz_t     (the residual's gradient is dy itself)
//
// Two launches and, where a reduction was cut or db is wanted, a third:
//   1. prep: dz is computed once from dy and the kept pre-activations, and written as bf16 term planes both as
//      [T][R] (dx's first operand) and, through LDS, as [R][T] (dW's); x and W are written transposed, so that both
//      products read their operands with the reduction contiguous.  The tiles add their columns of dz in fp32 for db.
//      What the reductions pad to a multiple of 64 is written as zeros.
//   2. product: both products in one launch of the tiled kernel, so the tiles of one fill what the other leaves idle.
//   3. join: parts of cut reductions, and db's parts, in a fixed order.
// Precision goes by the output's type.  An fp32 dx or dW is computed from operands held exactly: dz, and x where it
// is fp32, enter as three bf16 terms, and products of terms below 2^-24 of the whole are left out.  A bf16 dx or dW
// takes dz rounded once to bf16 (relative error at most 2^-9 per element, which adds to the same size of error from
// rounding the result) and x, where it is fp32, as two terms, so that dz's stays the only such rounding.
#include <algorithm>

#include "linear_dev.hpp"

namespace moe {
namespace {

constexpr int kPT = 64;  // tile side

struct Transpose {  // src [rows][cols] (fp32 or bf16) -> terms planes [cols][ld] of bf16, rows padded with zeros to ld
  const void* src;
  uint16_t* dst;
  int64_t plane;
  int rows, cols, ld, terms, f32;
  int blocks, tiles_c;
};

struct Prep {
  const void *dy, *pre;
  uint16_t *dz, *dzt;      // row-major and transposed planes (null: not wanted)
  int64_t dz_plane, dzt_plane;
  float* db_part;          // [tiles over T][R] or null
  int T, N, R, ldz, ldt;
  int act, bf16;           // dy's and pre's type
  int dz_terms, dzt_terms;
  int vec;                 // N % 4 == 0 and dy, pre aligned for 4-element loads
  int blocks, tiles_n;
  Transpose tr[2];
};

__device__ __forceinline__ void load4_any(const void* p, int bf16, size_t i, int vec, int valid, float (&v)[4]) {
  if (vec && valid >= 4) {
    if (bf16) {
      const uint2 q = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + i);
      v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xFFFF0000u);
      v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xFFFF0000u);
    } else {
      const float4 q = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
      v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    }
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = r < valid ? load_any(p, bf16, i + r) : 0.0f;
}

// A 64 x 64 fp32 tile in LDS, element (row, col); 65 words a row keep column reads off one bank.
typedef float Tile[kPT][kPT + 1];

// Column `tid / 4`, rows 16 (tid % 4) ... + 16 of the tile to row `c` of the transposed planes.
__device__ __forceinline__ void write_column(const Tile& t, uint16_t* dst, int64_t plane, int terms, size_t row_at,
                                             int tid) {
  const int c = tid >> 2, r0 = (tid & 3) * 16;
  uint32_t out[3][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint16_t a[3], b[3];
    bf16_terms(t[r0 + 2 * i][c], a);
    bf16_terms(t[r0 + 2 * i + 1][c], b);
#pragma unroll
    for (int k = 0; k < 3; ++k) out[k][i] = a[k] | (uint32_t)b[k] << 16;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < terms) {
      uint4* o = reinterpret_cast<uint4*>(dst + k * plane + row_at + r0);
      o[0] = make_uint4(out[k][0], out[k][1], out[k][2], out[k][3]);
      o[1] = make_uint4(out[k][4], out[k][5], out[k][6], out[k][7]);
    }
}

__device__ __forceinline__ void write_row4(uint16_t* dst, int64_t plane, int terms, size_t at, int aligned, int valid,
                                           const float (&v)[4]) {
  uint16_t t[4][3];
#pragma unroll
  for (int i = 0; i < 4; ++i) bf16_terms(v[i], t[i]);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (k >= terms) continue;
    uint16_t* o = dst + k * plane + at;
    if (aligned && valid >= 4) {
      *reinterpret_cast<uint2*>(o) = make_uint2(t[0][k] | (uint32_t)t[1][k] << 16, t[2][k] | (uint32_t)t[3][k] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < valid) o[i] = t[i][k];
    }
  }
}

__device__ void prep_dz(const Prep& p, int b, Tile& ta, Tile& tb) {
  const int tid = threadIdx.x;
  const int nt = b % p.tiles_n, tt = b / p.tiles_n;
  const int t0 = tt * kPT, n0 = nt * kPT;
  const bool pair = p.act == MOE_ACT_SWIGLU;
  const int c4 = (tid & 15) * 4, n = n0 + c4;
  const int valid = max(0, min(4, p.N - n));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (tid >> 4) + 16 * i, t = t0 + r;
    float a[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
    if (t < p.T && valid) {
      float g[4];
      load4_any(p.dy, p.bf16, (size_t)t * p.N + n, p.vec, valid, g);
      if (pair) {
        float zg[4], zu[4];
        load4_any(p.pre, p.bf16, (size_t)t * p.R + n, p.vec, valid, zg);
        load4_any(p.pre, p.bf16, (size_t)t * p.R + p.N + n, p.vec, valid, zu);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float h = sigmoid(zg[j]);
          a[j] = g[j] * zu[j] * (h * __builtin_fmaf(zg[j], 1.0f - h, 1.0f));
          u[j] = g[j] * (zg[j] * h);
        }
      } else if (p.act == MOE_ACT_NONE) {
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = g[j];
      } else {
        float z[4];
        load4_any(p.pre, p.bf16, (size_t)t * p.N + n, p.vec, valid, z);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = g[j] * act_slope(p.act, z[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j >= valid) a[j] = u[j] = 0.0f;
      if (p.dz) {
        const size_t at = (size_t)t * p.ldz + n;
        write_row4(p.dz, p.dz_plane, p.dz_terms, at, 1, valid, a);
        if (pair) write_row4(p.dz, p.dz_plane, p.dz_terms, at + p.N, p.N % 4 == 0, valid, u);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ta[r][c4 + j] = a[j];
      if (pair) tb[r][c4 + j] = u[j];
    }
  }
  if (p.dz && nt == p.tiles_n - 1 && p.ldz > p.R) {  // the padding columns of these rows
    const int w = p.ldz - p.R;
    for (int i = tid; i < kPT * w; i += 256) {
      const int t = t0 + i / w;
      if (t < p.T)
        for (int k = 0; k < p.dz_terms; ++k) p.dz[k * p.dz_plane + (size_t)t * p.ldz + p.R + i % w] = 0;
    }
  }
  __syncthreads();
  const int col = n0 + (tid >> 2);
  if (p.dzt && col < p.N) {
    write_column(ta, p.dzt, p.dzt_plane, p.dzt_terms, (size_t)col * p.ldt + t0, tid);
    if (pair) write_column(tb, p.dzt, p.dzt_plane, p.dzt_terms, (size_t)(p.N + col) * p.ldt + t0, tid);
  }
  if (p.db_part && tid < 2 * kPT) {
    const int c = tid & (kPT - 1), half = tid / kPT;
    if (n0 + c < p.N && (half == 0 || pair)) {
      float v = 0.0f;
      for (int r = 0; r < kPT; ++r) v += half ? tb[r][c] : ta[r][c];
      p.db_part[(size_t)tt * p.R + half * p.N + n0 + c] = v;
    }
  }
}

__device__ void prep_transpose(const Transpose& p, int b, Tile& tile) {
  const int tid = threadIdx.x;
  const int c0 = (b % p.tiles_c) * kPT, r0 = (b / p.tiles_c) * kPT;
  const int c4 = (tid & 15) * 4;
  const int valid = max(0, min(4, p.cols - c0 - c4));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (tid >> 4) + 16 * i;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (r0 + r < p.rows && valid) load4_any(p.src, !p.f32, (size_t)(r0 + r) * p.cols + c0 + c4, 1, valid, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) tile[r][c4 + j] = v[j];
  }
  __syncthreads();
  const int c = c0 + (tid >> 2);
  if (c < p.cols) write_column(tile, p.dst, p.plane, p.terms, (size_t)c * p.ld + r0, tid);
}

__global__ __launch_bounds__(256) void linear_prep_kernel(Prep p) {
  __shared__ Tile ta, tb;
  int b = blockIdx.x;
  if (b < p.blocks) {
    prep_dz(p, b, ta, tb);
    return;
  }
  b -= p.blocks;
  if (b < p.tr[0].blocks) prep_transpose(p.tr[0], b, ta);
  else prep_transpose(p.tr[1], b - p.tr[0].blocks, ta);
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
  int R, ldr, ldt;         // product columns; reductions of dx and dW padded to 64
  bool dx, dw, db, direct; // direct: dy itself is dx's first operand
  int dx_terms, dw_terms, x_terms;
  int segs_dx, segs_dw;
  uint32_t dx_sa, dx_sb, dw_sa, dw_sb;
  int split_dx, split_dw, tiles_t;
  size_t dz, dzt, wt, xt, part_dx, part_dw, db_part, bytes;
};

GradPlan grad_plan(int T, int K, int N, int act, moe_dtype dy_t, moe_dtype x_t, moe_dtype dx_t, moe_dtype dw_t,
                   int need) {
  GradPlan p{};
  p.R = act == MOE_ACT_SWIGLU ? 2 * N : N;
  p.ldr = (int)(ceil_div(p.R, 64) * 64);
  p.ldt = (int)(ceil_div(T, 64) * 64);
  p.tiles_t = (int)ceil_div(T, kPT);
  p.dx = need & MOE_NEED_DX;
  p.dw = need & MOE_NEED_DW;
  p.db = need & MOE_NEED_DB;
  const bool one = act == MOE_ACT_NONE && dy_t == MOE_BF16;  // dz is dy: one term holds it
  p.dx_terms = one || dx_t == MOE_BF16 ? 1 : 3;
  p.dw_terms = one || dw_t == MOE_BF16 ? 1 : 3;
  p.x_terms = x_t == MOE_BF16 ? 1 : dw_t == MOE_F32 ? 3 : one ? 1 : 2;
  p.direct = p.dx && one && p.R % 8 == 0;
  p.segs_dx = segments(p.dx_terms, 1, p.dx_sa, p.dx_sb);
  p.segs_dw = segments(p.dw_terms, p.x_terms, p.dw_sa, p.dw_sb);
  const int64_t tiles = (p.dx ? prob_tiles(T, K, false) : 0) + (p.dw ? prob_tiles(p.R, K, false) : 0);
  p.split_dx = p.dx ? prob_split(tiles, p.ldr / 64 * p.segs_dx) : 1;
  p.split_dw = p.dw ? prob_split(tiles, p.ldt / 64 * p.segs_dw) : 1;
  size_t o = 0;
  auto take = [&](bool want, size_t bytes) {
    const size_t at = o;
    if (want) o = up256(o + bytes);
    return at;
  };
  p.dz = take(p.dx && !p.direct, (size_t)p.dx_terms * T * p.ldr * 2);
  p.wt = take(p.dx, (size_t)K * p.ldr * 2);
  p.dzt = take(p.dw, (size_t)p.dw_terms * p.R * p.ldt * 2);
  p.xt = take(p.dw, (size_t)p.x_terms * K * p.ldt * 2);
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
  Prep p{};
  p.dy = dy;
  p.pre = pre;
  p.T = T;
  p.N = N;
  p.R = pl.R;
  p.act = act;
  p.bf16 = dy_t == MOE_BF16;
  p.ldz = pl.ldr;
  p.ldt = pl.ldt;
  p.dz_terms = pl.dx_terms;
  p.dzt_terms = pl.dw_terms;
  p.dz_plane = (int64_t)T * pl.ldr;
  p.dzt_plane = (int64_t)pl.R * pl.ldt;
  if (pl.dx && !pl.direct) p.dz = u16(pl.dz);
  if (pl.dw) p.dzt = u16(pl.dzt);
  if (pl.db) p.db_part = f32(pl.db_part);
  const uintptr_t al = p.bf16 ? 8 : 16;
  p.vec = N % 4 == 0 && reinterpret_cast<uintptr_t>(dy) % al == 0 && reinterpret_cast<uintptr_t>(pre) % al == 0;
  p.tiles_n = (int)ceil_div(N, kPT);
  const bool any = p.dz || p.dzt || p.db_part;
  const int64_t blocks = any ? (int64_t)p.tiles_n * pl.tiles_t : 0;
  int64_t more[2] = {0, 0};
  auto transpose = [&](int i, const void* src, int rows, int cols, bool f, uint16_t* dst, int ld, int terms) {
    Transpose& t = p.tr[i];
    t = Transpose{src, dst, (int64_t)cols * ld, rows, cols, ld, terms, f, 0, (int)ceil_div(cols, kPT)};
    more[i] = (int64_t)t.tiles_c * (ld / kPT);
  };
  if (pl.dx) transpose(0, w, pl.R, K, false, u16(pl.wt), pl.ldr, 1);
  if (pl.dw) transpose(1, x, T, K, x_t == MOE_F32, u16(pl.xt), pl.ldt, pl.x_terms);
  if (blocks + more[0] + more[1] > 0x7FFFFFFF) return fail(MOE_EUNSUPPORTED, "moe_linear_backward: too many tiles");
  p.blocks = (int)blocks;
  p.tr[0].blocks = (int)more[0];
  p.tr[1].blocks = (int)more[1];
  linear_prep_kernel<<<dim3((unsigned)(blocks + more[0] + more[1])), 256, 0, s>>>(p);
  if (moe_status st = check_launch("linear_backward")) return st;

  Group g{};
  int count = 0;
  auto product = [&](const uint16_t* A, int64_t a_plane, int lda, const uint16_t* B, int64_t b_plane, int ldb, int M,
                     int red, int nseg, uint32_t sa, uint32_t sb, int split, float* partial, void* out, moe_dtype out_t) {
    Prob& q = g.p[count++];
    q.A = A;
    q.a_plane = a_plane;
    q.lda = lda;
    q.B = B;
    q.b_plane = b_plane;
    q.ldb = ldb;
    q.M = M;
    q.R = K;
    q.K = red;
    q.nseg = nseg;
    q.sa = sa;
    q.sb = sb;
    q.split = split;
    q.partial = partial;
    q.ldp = K;
    q.epi = Epi{nullptr, nullptr, out, nullptr, K, K, MOE_ACT_NONE, 0, out_t == MOE_BF16, 0};
  };
  if (pl.dx)
    product(pl.direct ? reinterpret_cast<const uint16_t*>(dy) : p.dz, p.dz_plane, pl.direct ? pl.R : pl.ldr, u16(pl.wt),
            0, pl.ldr, T, pl.direct ? pl.R : pl.ldr, pl.segs_dx, pl.dx_sa, pl.dx_sb, pl.split_dx, f32(pl.part_dx), dx,
            dx_t);
  if (pl.dw)
    product(p.dzt, p.dzt_plane, pl.ldt, u16(pl.xt), (int64_t)K * pl.ldt, pl.ldt, pl.R, pl.ldt, pl.segs_dw, pl.dw_sa,
            pl.dw_sb, pl.split_dw, f32(pl.part_dw), dw, dw_t);
  return launch_products(MOE_KERNEL_LINEAR_BACKWARD, g, count, p.db_part, pl.tiles_t, pl.R, db, s, "linear_backward");
}

}  // namespace moe
