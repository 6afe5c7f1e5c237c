// linear_q8.hip -- dense product of 8-bit integers with a scale per token and per weight row:
//   z = (sum_c qx[c] qw[c]) sx sw + b,  y = act(z) + residual,  SwiGLU: y = silu(z_gate) z_up + residual.
//
// The integer sums are exact in 32 bits (at most 16,384 * 128 * 128 = 2^28); one conversion, two products with the scales
// and the epilogue's sums round in fp32.  fp32 and bf16 activations are coded on the way in (quantize_dev.hpp): in the
// product's own launch for a few tokens, else by a launch of quantize_rows before it.
//
// Up to 64 tokens: q8_few_kernel, weights straight from memory into matrix operands.  More: the loop of product_dev.hpp on
// v_mfma_i32_16x16x64_i8, which does twice bf16's products in the same time from the same number of bytes.
#include "product_dev.hpp"
#include "quantize_dev.hpp"

namespace moe {
namespace {

// A sum times both scales, the one of smaller magnitude first: the sum's magnitude is at least 1 (or it is 0), so nothing is
// lost below a normal scale's range, and nothing passes its top that the result would not.
__device__ __forceinline__ float scaled(int sum, float a, float b) {
  const bool first = fabsf(a) < fabsf(b);
  return (float)sum * (first ? a : b) * (first ? b : a);
}

struct Scales {
  const float *x, *w;  // [T], [R]
};

// ---- up to 64 tokens --------------------------------------------------------------------

constexpr int kFewT = 64, kFewWaves = 8, kFewThreads = 64 * kFewWaves;
constexpr int kOwnGroups = 4;                             // groups of 8 values a thread codes itself
constexpr int kOwnValues = kFewThreads * kOwnGroups * 8;  // 16,384 of all tokens

// Grid: one workgroup per 16 rows of W (8 gate and 8 up rows for SwiGLU), 8 waves.  v_mfma_i32_16x16x64_i8 takes the 16
// rows as its first operand and 16 tokens as its second; TF such token fragments share each weight fragment.  Wave w works
// through its eighth of the K-steps with the loads of four steps in flight; the eight sums of an element are added through
// LDS.  XT: the activations are codes (0), bf16 (1) or fp32 (2); in the last two every workgroup codes all of them into LDS
// while its first weights are on their way (each value by one thread, rows' maxima by LDS atomics, whose order does not
// matter).  Rows of W past R and tokens past T read the last valid one and are not stored.
//
// One token of 2,048 -> 512 SwiGLU: 4.0 us, three of 512 -> 2,048 3.8, where the weights' 2.1 and 1.0 MB are 0.4 and 0.2 us
// of memory: what counts is the launch, one round trip to memory, the codes' two barriers and the join of the waves.  Of weights
// that come from HBM, one token of 8,192 -> 8,192 takes 17.3 us (67 MB at 3.9 TB/s; in bf16 28.0), of 4,096 -> 4,096 7.8 (2.1 TB/s;
// bf16 9.0).  64 tokens of 8,192 -> 8,192 take 42.9 from codes: each workgroup reads all of x, four times its weights' bytes.
template <int XT, int TF>
__global__ __launch_bounds__(kFewThreads) void q8_few_kernel(const void* __restrict__ x, const int8_t* __restrict__ w,
                                                             Scales sc, int T, int K, Epi e) {
  constexpr int U = 4;
  constexpr int kPad = 16;  // bytes between rows in LDS, so that 16 tokens' pieces fall on different banks
  __shared__ __attribute__((aligned(16))) int red[kFewWaves][TF][64][4];
  __shared__ __attribute__((aligned(16))) int8_t codes[XT ? kOwnValues + 16 * TF * kPad : 16];
  __shared__ uint32_t amax[16 * TF];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const bool pair = e.act == MOE_ACT_SWIGLU;
  const int fr = lane & 15, fq = lane >> 4;
  int row;
  if (pair) {
    row = min((int)blockIdx.x * 8 + (fr & 7), e.N - 1) + (fr >= 8 ? e.N : 0);
  } else {
    row = min((int)blockIdx.x * 16 + fr, e.N - 1);
  }
  const int8_t* wrow = w + (size_t)row * K;
  const int steps = (K + 63) / 64;
  const int s0 = steps * wave / kFewWaves, s1 = steps * (wave + 1) / kFewWaves;
  // a K-step past the wave's last, or a half of it past K, counts as zeros
  auto load_w = [&](uint4 (&q)[U], int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u) * 64 + fq * 16;
      const bool in = s + u < s1 && k < K;
      q[u] = *reinterpret_cast<const uint4*>(wrow + (in ? k : 0));
      if (!in) q[u] = make_uint4(0, 0, 0, 0);
    }
  };
  uint4 wq[U];
  load_w(wq, s0);

  // The results this thread will finish, with what their epilogue reads.
  constexpr int kElems = (TF * 256 + kFewThreads - 1) / kFewThreads;
  struct {
    int t, n, r;  // t < 0: none
    float sx, sw, su;
    EpiIn in;
  } el[kElems];
#pragma unroll
  for (int i = 0; i < kElems; ++i) {
    const int at = i * kFewThreads + threadIdx.x;
    el[i].r = at & 15;
    el[i].n = blockIdx.x * (pair ? 8 : 16) + el[i].r;
    const bool has = at < TF * 256 && at >> 4 < T && el[i].n < e.N && !(pair && el[i].r >= 8);
    el[i].t = has ? at >> 4 : -1;
    if (has) {
      el[i].in = epi_in(e, el[i].t, el[i].n);
      el[i].sw = sc.w[el[i].n];
      el[i].su = pair ? sc.w[e.N + el[i].n] : 0.0f;
      if constexpr (XT == 0) el[i].sx = sc.x[el[i].t];
    }
  }

  if constexpr (XT != 0) {
    Eight<XT == 2> v[kOwnGroups];
    const int total = T * K;
#pragma unroll
    for (int i = 0; i < kOwnGroups; ++i) v[i].load(x, min((i * kFewThreads + (int)threadIdx.x) * 8, total - 8));
    if (threadIdx.x < 16 * TF) amax[threadIdx.x] = 0;
    __syncthreads();
    int at[kOwnGroups], of[kOwnGroups];  // where each group lies, and its row
#pragma unroll
    for (int i = 0; i < kOwnGroups; ++i) {
      at[i] = (i * kFewThreads + threadIdx.x) * 8;
      of[i] = at[i] / K;
      // K is a multiple of 32, so four neighbouring groups are of one row
      uint32_t m = at[i] < total ? amax_bits(v[i]) : 0;
      m = max(m, dpp_u32<0xB1, 0xF>(m));  // quad_perm 1 0 3 2
      m = max(m, dpp_u32<0x4E, 0xF>(m));  // quad_perm 2 3 0 1
      if (at[i] < total && (threadIdx.x & 3) == 0) atomicMax(&amax[of[i]], m);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOwnGroups; ++i) {
      if (at[i] >= total) break;
      const uint32_t m = amax[of[i]];
      const RowScale r = row_scale(m);
      float f[8];
      v[i].get(f);
      *reinterpret_cast<uint2*>(codes + at[i] + of[i] * kPad) = finite_bits(m) ? codes8(f, r) : make_uint2(0, 0);
    }
    __syncthreads();
  }

  i32x4_t acc[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) acc[f] = i32x4_t{0, 0, 0, 0};
  size_t xoff[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) xoff[f] = (size_t)min(16 * f + fr, T - 1) * (XT ? K + kPad : K);
  const int8_t* xs = XT ? codes : reinterpret_cast<const int8_t*>(x);
  for (int s = s0; s < s1; s += U) {
    uint4 xq[U][TF];
#pragma unroll
    for (int u = 0; u < U; ++u) {  // (what does not count meets weights of zero)
      const int k = (s + u) * 64 + fq * 16;
#pragma unroll
      for (int f = 0; f < TF; ++f) xq[u][f] = *reinterpret_cast<const uint4*>(xs + xoff[f] + (k < K ? k : 0));
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int f = 0; f < TF; ++f)
        acc[f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, wq[u]),
                                                       __builtin_bit_cast(i32x4_t, xq[u][f]), acc[f], 0, 0, 0);
    if (s + U < s1) load_w(wq, s + U);
  }
  // lane: token 16 f + (lane & 15), rows 4 (lane >> 4) + r
#pragma unroll
  for (int f = 0; f < TF; ++f) *reinterpret_cast<i32x4_t*>(red[wave][f][lane]) = acc[f];
  __syncthreads();
  auto sum_of = [&](int f, int r, int tk) {  // row r of the workgroup's 16, token tk of fragment f
    const int l = 16 * (r >> 2) + tk;
    int v = 0;
#pragma unroll
    for (int i = 0; i < kFewWaves; ++i) v += red[i][f][l][r & 3];
    return v;
  };
#pragma unroll
  for (int i = 0; i < kElems; ++i) {
    if (el[i].t < 0) continue;
    const int f = el[i].t >> 4, tk = el[i].t & 15;
    const float sx = XT ? row_scale(amax[el[i].t]).s : el[i].sx;
    epi_one(e, el[i].t, el[i].n, scaled(sum_of(f, el[i].r, tk), sx, el[i].sw),
            pair ? scaled(sum_of(f, el[i].r + 8, tk), sx, el[i].su) : 0.0f, el[i].in);
  }
}

// ---- more tokens ---------------------------------------------------------------------------

// Sums to products: four columns' scales stay in registers, a row's comes from where `row` finds it.
template <bool PAIR>
struct ColumnScales {
  float s[4], u[4];
  __device__ __forceinline__ void load(const float* w, int n, int N) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s[r] = w[min(n + r, N - 1)];
      u[r] = PAIR ? w[N + min(n + r, N - 1)] : 0.0f;
    }
  }
};

// 8,192 x 4,096 x 4,096 without an epilogue takes 123 us (2.23 POP/s; a library product of 8,192^3 has 2.0), with SiLU,
// residual and a bf16 result 144: the epilogue of one workgroup per CU is overlapped by nothing.  8,192 x 2,048 -> 512 SwiGLU on
// 128 x 128 tiles 23.4 us (1.47 POP/s; two workgroups a CU, one round of them).
template <typename T, bool PAIR>
__global__ __launch_bounds__(T::kThreads, 2) void q8_product_kernel(Prob p, Scales sc) {
  constexpr int TM = T::TM, TN = T::TN, WM = T::WM, WN = T::WN, kFM = T::kFM, kFN = T::kFN, kThreads = T::kThreads;
  constexpr int cols = PAIR ? TN / 2 : TN;  // output columns per tile
  constexpr int kTile = TM * TN * 4 / T::kPasses;  // bytes of sums in LDS at once; the rows' scales lie behind them
  __shared__ __attribute__((aligned(16))) uint8_t lds[std::max(T::kBuffers, kTile + TM * 4)];
  const int tm = (p.M + TM - 1) / TM, tn = (p.epi.N + cols - 1) / cols;
  const int item = die_item(blockIdx.x, gridDim.x);
  const int part = uniform(item / (tm * tn));
  // tiles in bands of 8 row tiles, walked column by column
  const int tile = item - part * tm * tn;
  const int band = tile / (8 * tn), in_band = tile - band * 8 * tn;
  const int band_rows = min(8, tm - band * 8);
  const int m0 = uniform((band * 8 + in_band % band_rows) * TM), n0 = uniform(in_band / band_rows * cols);
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int kg = wave / (WM * WN), wm = T::KG == 1 ? wave / WN : wave / WN % WM, wn = wave % WN;
  const int steps = (p.K + kBK - 1) / kBK;
  const int lo = uniform((int)((int64_t)steps * part / p.split)), hi = uniform((int)((int64_t)steps * (part + 1) / p.split));
  const float row_s = tid < TM ? sc.x[min(m0 + tid, p.M - 1)] : 0.0f;
  i32x4_t acc[kFM][kFN];
  // rows past the end read the last one and are not stored
  product_loop<T, false, false, 0, KindI8>(
      p, m0, n0, lo, hi, [&](int r) { return min(m0 + r, p.M - 1) - m0; },
      [&](int r) {  // SwiGLU: each wave's gate rows before its up rows
        constexpr int kW = TN / WN, kH = kW / 2;
        const int n = PAIR ? (r / kW) * kH + r % kH : r;
        return min(n0 + n, p.epi.N - 1) - n0 + (PAIR && r % kW >= kH ? p.epi.N : 0);
      },
      lds, acc);

  // Through LDS, so that the epilogue's loads and stores run along rows: 16-byte pieces, piece c of row m at c ^ (m % 16).
  int* tile_c = reinterpret_cast<int*>(lds);
  float* rows_s = reinterpret_cast<float*>(lds + kTile);
  constexpr int kPieces = TN / 4, kPassRows = TM / T::kPasses, kOutPieces = cols / 4;
  const int r16 = lane & 15, q = lane >> 4;
#pragma unroll
  for (int pass = 0; pass < T::kPasses; ++pass) {
    hand_over();
    if (pass == 0 && tid < TM) rows_s[tid] = row_s;
    auto put = [&](auto add) {
#pragma unroll
      for (int i = 0; i < kFM; ++i)
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
          const int m = (T::kPasses == 1 ? (TM / WM) * wm : 0) + 16 * i + r16, c = (TN / WN / 4) * wn + 4 * j + q;
          i32x4_t* at = reinterpret_cast<i32x4_t*>(tile_c + (m * kPieces + (c ^ (m & 15))) * 4);
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
    // a thread keeps to four columns and walks down the rows
    static_assert(kThreads % kOutPieces == 0, "columns per thread");
    const int o = tid % kOutPieces, n = n0 + 4 * o;
    constexpr int kH = TN / WN / 8;  // PAIR: pieces of a wave's gate rows
    const int c = PAIR ? (o / kH) * 2 * kH + o % kH : o;
    constexpr int kStep = kThreads / kOutPieces;
    const int r0 = tid / kOutPieces, m = m0 + pass * kPassRows + r0;
    const int rows = n < p.epi.N ? min(kPassRows - r0, p.M - m) : 0;  // counted from r0 on, in steps of kStep
    auto piece = [&](int r, int at) { return *reinterpret_cast<const i32x4_t*>(tile_c + (r * kPieces + (at ^ (r & 15))) * 4); };
    if (p.split > 1) {
      int* out = reinterpret_cast<int*>(p.partial) + ((size_t)part * p.M + m) * p.ldp + n;
      for (int d = 0; d < rows; d += kStep) {  // (ldp holds whole groups of four behind each half's last column)
        *reinterpret_cast<i32x4_t*>(out) = piece(r0 + d, c);
        if constexpr (PAIR) *reinterpret_cast<i32x4_t*>(out + p.ldp / 2) = piece(r0 + d, c + kH);
        out += (size_t)kStep * p.ldp;
      }
    } else {
      ColumnScales<PAIR> cs;
      if (rows > 0) cs.load(sc.w, n, p.epi.N);
      epi_rows<PAIR, kStep>(p.epi, m, n, rows, [&](int d, float (&z)[4], float (&zu)[4]) {
        const float s = rows_s[pass * kPassRows + r0 + d];
        const i32x4_t v = piece(r0 + d, c);
#pragma unroll
        for (int r = 0; r < 4; ++r) z[r] = scaled(v[r], s, cs.s[r]);
        if constexpr (PAIR) {
          const i32x4_t u = piece(r0 + d, c + kH);
#pragma unroll
          for (int r = 0; r < 4; ++r) zu[r] = scaled(u[r], s, cs.u[r]);
        }
      });
    }
  }
}

// Adds the parts of a cut reduction (integers: exact in any order) and applies scales and epilogue, four columns a thread.
template <bool PAIR>
__global__ __launch_bounds__(256) void q8_join_kernel(Prob p, Scales sc) {
  const int quads = (p.epi.N + 3) >> 2;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.M * quads) return;
  const int m = (int)(i / quads), n = (int)(i - (int64_t)m * quads) * 4;
  i32x4_t v = {0, 0, 0, 0}, u = {0, 0, 0, 0};
  const size_t step = (size_t)p.M * p.ldp;
  const int* in = reinterpret_cast<const int*>(p.partial) + (size_t)m * p.ldp + n;
#pragma unroll 4
  for (int s = 0; s < p.split; ++s) {
    v += *reinterpret_cast<const i32x4_t*>(in + s * step);
    if constexpr (PAIR) u += *reinterpret_cast<const i32x4_t*>(in + s * step + p.ldp / 2);
  }
  const float s = sc.x[m];
  ColumnScales<PAIR> cs;
  cs.load(sc.w, n, p.epi.N);
  epi_rows<PAIR, 1>(p.epi, m, n, 1, [&](int, float (&z)[4], float (&zu)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      z[r] = scaled(v[r], s, cs.s[r]);
      zu[r] = PAIR ? scaled(u[r], s, cs.u[r]) : 0.0f;
    }
  });
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Q8Plan {
  bool few, own;  // own: the product's launch codes the activations
  bool codes;     // a launch before it does
  Plan plan;
  int R, ldp;
  size_t code, scale, partial, bytes;  // offsets and size of the workspace
};
Q8Plan q8_plan(int T, int K, int N, int act, moe_dtype x_t) {
  Q8Plan p{};
  const bool pair = act == MOE_ACT_SWIGLU;
  p.R = pair ? 2 * N : N;
  p.ldp = (N + 3) / 4 * 4 * (pair ? 2 : 1);
  p.few = T <= kFewT;
  // In a graph: 16 tokens of 1,024 bf16 values for 1,024 columns 6.9 us either way, 32 of 512 7.0 against 7.4 (fp32: 5.8,
  // 7.2), one of 2,048 4.2 against 5.9; of twice as many values 16 x 2,048 9.7 against 7.7.
  p.own = x_t != MOE_I8 && p.few && T * K <= kOwnValues;
  p.codes = x_t != MOE_I8 && !p.own;
  size_t o = 0;
  p.code = o;
  if (p.codes) o = up256(o + (size_t)T * K);
  p.scale = o;
  if (p.codes) o = up256(o + (size_t)T * 4);
  p.partial = o;
  if (!p.few) {
    const Shape shape{T, p.R, K / 2, 1, false, 1};  // two values a word
    p.plan = plan_products(&shape, 1);
    if (p.plan.split[0] > 1) o = up256(o + (size_t)p.plan.split[0] * T * p.ldp * 4);
  }
  p.bytes = o;
  return p;
}

}  // namespace

size_t linear_q8_ws_bytes(int T, int K, int N, int act, moe_dtype x_t) { return q8_plan(T, K, N, act, x_t).bytes; }

void linear_q8_form(int T, int K, int N, int act, moe_dtype x_t, int32_t form[3]) {
  const Q8Plan p = q8_plan(T, K, N, act, x_t);
  form[0] = p.few ? 0 : tile_side(p.plan);
  form[1] = p.few ? 1 : p.plan.split[0];
  form[2] = p.codes;
}

moe_status launch_linear_q8(const void* x, moe_dtype x_t, const float* x_scale, const int8_t* w, const float* w_scale,
                            const float* bias, int act, const void* residual, moe_dtype r_t, int T, int K, int N, void* y,
                            moe_dtype y_t, void* ws, hipStream_t s) {
  const Q8Plan pl = q8_plan(T, K, N, act, x_t);
  const bool pair = act == MOE_ACT_SWIGLU;
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  Epi e{bias, residual, y, nullptr, N, pl.R, act, r_t == MOE_BF16, y_t == MOE_BF16};
  Scales sc{x_scale, w_scale};
  if (pl.codes) {
    int8_t* codes = reinterpret_cast<int8_t*>(base + pl.code);
    float* scale = reinterpret_cast<float*>(base + pl.scale);
    if (moe_status st = launch_quantize_rows(x, x_t, T, K, codes, scale, s)) return st;
    x = codes;
    sc.x = scale;
  }
  if (pl.few) {
    const dim3 grid((unsigned)ceil_div(N, pair ? 8 : 16));
    auto go = [&](auto kernel) { launch_k(MOE_KERNEL_LINEAR_Q8, kernel, grid, dim3(kFewThreads), 0, s, x, w, sc, T, K, e); };
    auto tokens = [&](auto xt) {
      constexpr int X = decltype(xt)::value;
      if (T <= 16) go(q8_few_kernel<X, 1>);
      else if (T <= 32) go(q8_few_kernel<X, 2>);
      else go(q8_few_kernel<X, 4>);
    };
    if (!pl.own) tokens(std::integral_constant<int, 0>{});
    else if (x_t == MOE_BF16) tokens(std::integral_constant<int, 1>{});
    else tokens(std::integral_constant<int, 2>{});
    return check_launch("linear_q8");
  }
  Prob p{};
  p.A = reinterpret_cast<const uint16_t*>(x);
  p.B = reinterpret_cast<const uint16_t*>(w);
  p.lda = p.ldb = p.K = K / 2;
  p.M = T;
  p.R = pl.R;
  p.nseg = 1;
  p.split = pl.plan.split[0];
  p.partial = reinterpret_cast<float*>(base + pl.partial);
  p.ldp = pl.ldp;
  p.epi = e;
  const int side = tile_side(pl.plan);
  const int64_t blocks = ceil_div(T, side) * ceil_div(N, pair ? side / 2 : side) * p.split;
  const dim3 grid((unsigned)blocks);
  auto go = [&](auto tile) {
    using Tl = decltype(tile);
    auto run = [&](auto kernel) { launch_k(MOE_KERNEL_LINEAR_Q8, kernel, grid, dim3((unsigned)Tl::kThreads), 0, s, p, sc); };
    pair ? run(q8_product_kernel<Tl, true>) : run(q8_product_kernel<Tl, false>);
  };
  if (pl.plan.shape == 0) go(Tiny{});
  else if (pl.plan.shape == 1) go(Small{});
  else go(Large{});
  if (moe_status st = check_launch("linear_q8")) return st;
  if (p.split > 1) {
    const dim3 joins((unsigned)ceil_div((int64_t)T * ((N + 3) / 4), 256));
    pair ? q8_join_kernel<true><<<joins, 256, 0, s>>>(p, sc) : q8_join_kernel<false><<<joins, 256, 0, s>>>(p, sc);
    return check_launch("linear_q8");
  }
  return MOE_OK;
}

}  // namespace moe
