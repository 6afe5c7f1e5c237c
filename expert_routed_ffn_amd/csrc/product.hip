// product.hip -- the tiled bf16 product behind the dense product and its gradient:
//   C[m][n] = sum_k A(m, k) B(n, k),  fp32 sums,  then the epilogue of linear_dev.hpp
// Either operand lies with k contiguous ([m][k]) or with its own index contiguous ([k][m]): the forward product reads
// x and W as they are, dx = dz W and dW = dz^T x read W, dz and x in the second form, so no operand is transposed in
// memory.
//
// v_mfma_f32_16x16x32_bf16 with B's rows first, so a lane holds four consecutive columns of C.  16 x 16 fragments
// measured 10% faster than 32 x 32 ones in the same kernel (36.5 against 40.5 us on 8192 x 2048 x 1024, 224 against
// 241 us on 8192 x 4096 x 4096).  Tiles go from memory straight to LDS (16 bytes a lane, two buffers of 64 k), and
// the step's loop is turned so that neither the loads nor the LDS reads are waited for with the matrix units idle:
// fragments of one 32-k half are read while the other half is multiplied, and the barrier that hands over the buffers
// stands before the last half's products.
//
// LDS places: 64 banks of 4 bytes serve 16 lanes of a 16-byte read at once.  [m][k] tiles are rows of 128 bytes whose
// 16-byte piece c lies at c ^ (row / 2 % 8): the 16 rows that such a group reads at one piece fall on 16 different
// places (with row % 8 they fell on 8, and half of all LDS cycles were conflicts).  [k][m] tiles are read with
// ds_read_b64_tr_b16, where 16 lanes take 4 k of 16 columns and each receives its column's 4 values; the 32-byte
// stretch s of row k lies at s ^ (k % 4 + 4 (k / 8 % 2)), which spreads the 8 rows that 32 lanes touch over 256 bytes.
//
// Three tile shapes, chosen by plan_products.  256 x 256 (8 waves, 128 KB of LDS, one workgroup per CU) reads half as
// much per product as 128 x 128 (4 waves, two workgroups per CU), but needs enough tiles to fill 256 CUs evenly.  64 x 64
// tiles are for products of few tiles, whose time is the latency of their loads: five buffers keep four steps' loads
// under way, and two groups of four waves take half of each step's k (one group: 10 to 15% slower).  (Rings of 3 or 4
// buffers of 32 k under the large tiles measured no better than two of 64.)
//
// fp32 A of the forward product (Direct): 64 x 64 tiles whose A stays fp32 up to the fragments, which are split into bf16
// terms there, each value once per workgroup.  W's tile then meets all terms in one pass, and no launch writes term
// planes: 777 x 1056 x 1001 in three terms 27.8 -> 14.4 us, 8192 x 2048 x 512 91 -> 67.  It takes three buffers (72 KB, two
// workgroups per CU; 8192 x 2048 x 512 with four: 79).  Reading the next step's fragments ahead of the products cost 5%.
#include "product_dev.hpp"

namespace moe {
namespace {

// Four columns n ... of a part's row, those below N.
__device__ __forceinline__ void put_part(float* out, int n, int N, const float (&z)[4]) {
  if (n + 4 <= N) {
    store4(out, 0, 0, z);
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (n + r < N) out[r] = z[r];
  }
}

// One tile of one part of a product's reduction.  AK, BK: the operand is [k][index].  PAIR: SwiGLU, whose tiles hold
// TN / 2 gate rows of W and the same up rows, each wave's gate rows before its up rows.  TERMS: A is fp32 and enters as so
// many bf16 terms, split here; 0: A is bf16.
template <typename T, bool AK, bool BK, bool PAIR, int TERMS = 0>
__device__ __forceinline__ void product_tile(const Prob& p, int b, int total, uint8_t* lds) {
  constexpr int TM = T::TM, TN = T::TN, WM = T::WM, WN = T::WN, kFM = T::kFM, kFN = T::kFN, kThreads = T::kThreads;
  constexpr int cols = PAIR ? TN / 2 : TN;  // output columns per tile
  const int tm = (p.M + TM - 1) / TM, tn = (p.epi.N + cols - 1) / cols;
  const int item = die_item(b, total);
  const int part = uniform(item / (tm * tn));
  // tiles in bands of 8 row tiles, walked column by column
  const int tile = item - part * tm * tn;
  const int band = tile / (8 * tn), in_band = tile - band * 8 * tn;
  const int band_rows = min(8, tm - band * 8);
  const int m0 = uniform((band * 8 + in_band % band_rows) * TM), n0 = uniform(in_band / band_rows * cols);

  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int kg = wave / (WM * WN), wm = T::KG == 1 ? wave / WN : wave / WN % WM, wn = wave % WN;
  const int seg_steps = (p.K + kBK - 1) / kBK, steps = seg_steps * p.nseg;
  const int lo = uniform((int)((int64_t)steps * part / p.split)), hi = uniform((int)((int64_t)steps * (part + 1) / p.split));
  f32x4_t acc[kFM][kFN];
  // rows past the end read the last one and are not stored
  product_loop<T, AK, BK, TERMS, KindBf16>(
      p, m0, n0, lo, hi, [&](int r) { return min(m0 + r, p.M - 1) - m0; },
      [&](int r) {
        constexpr int kW = TN / WN, kH = kW / 2;
        const int n = PAIR ? (r / kW) * kH + r % kH : r;
        return min(n0 + n, p.epi.N - 1) - n0 + (PAIR && r % kW >= kH ? p.epi.N : 0);
      },
      lds, acc);

  // The fp32 tile goes through LDS so that a wave's loads and stores of the epilogue run along rows.  A lane holds
  // row lane % 16 of A and four rows 4 (lane / 16) of B: 16-byte pieces, piece c of row m at c ^ (m % 16), so that the
  // lanes that write together lie in 16 different places.
  float* tile_c = reinterpret_cast<float*>(lds);
  constexpr int kPieces = TN / 4, kPassRows = TM / T::kPasses, kOutPieces = cols / 4;
  const int r16 = lane & 15, q = lane >> 4;
  const bool split = p.split > 1;
#pragma unroll
  for (int pass = 0; pass < T::kPasses; ++pass) {
    hand_over();  // the loads and reads of the loop, or the reads of the pass before, are done
    auto put = [&](auto add) {
#pragma unroll
      for (int i = 0; i < kFM; ++i)
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
          const int m = (T::kPasses == 1 ? (TM / WM) * wm : 0) + 16 * i + r16, c = (TN / WN / 4) * wn + 4 * j + q;
          f32x4_t* at = reinterpret_cast<f32x4_t*>(tile_c + (m * kPieces + (c ^ (m & 15))) * 4);
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
    auto piece = [&](int r, int at, float (&z)[4]) {
      const float4 v = *reinterpret_cast<const float4*>(tile_c + (r * kPieces + (at ^ (r & 15))) * 4);
      z[0] = v.x; z[1] = v.y; z[2] = v.z; z[3] = v.w;
    };
    auto value = [&](int d, float (&z)[4], float (&zu)[4]) {  // row r0 + d
      piece(r0 + d, c, z);
      if constexpr (PAIR) piece(r0 + d, c + kH, zu);
    };
    if (split) {
      float* out = p.partial + ((size_t)part * p.M + m) * p.ldp + n;
      for (int d = 0; d < rows; d += kStep) {
        float z[4], zu[4];
        value(d, z, zu);
        put_part(out, n, p.epi.N, z);
        if constexpr (PAIR) put_part(out + p.epi.N, n, p.epi.N, zu);
        out += (size_t)kStep * p.ldp;
      }
    } else {
      epi_rows<PAIR, kStep>(p.epi, m, n, rows, value);
    }
  }
}

// The forward product.
template <typename T, bool PAIR, int TERMS>
__global__ __launch_bounds__(T::kThreads, 2) void linear_product_kernel(Prob p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[T::kLds];
  product_tile<T, false, false, PAIR, TERMS>(p, blockIdx.x, gridDim.x, lds);
}

// db from its parts: 64 columns a workgroup; four waves take every fourth part, and their sums are added in wave order.
__device__ __forceinline__ void add_db(const DbSum& d, int group, float* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = group * 64 + lane;
  if (wave < 4) {
    float v = 0.0f;
    if (c < d.n) {
#pragma unroll 8
      for (int r = wave; r < d.rows; r += 4) v += d.part[(size_t)r * d.n + c];
    }
    lds[64 * wave + lane] = v;
  }
  __syncthreads();
  if (wave == 0 && c < d.n) d.db[c] = lds[lane] + lds[64 + lane] + lds[128 + lane] + lds[192 + lane];
}

// The gradient's two products in one grid, so that the tiles of one fill what the other leaves idle: first dW (the
// longer reduction as a rule), then dx, then db's column groups.
template <typename T>
__global__ __launch_bounds__(T::kThreads, 2) void grad_products_kernel(Prob dw, Prob dx, int dw_blocks, int dx_blocks,
                                                                       DbSum db) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[T::kLds];
  const int b = blockIdx.x;
  if (b < dw_blocks) product_tile<T, true, true, false>(dw, b, dw_blocks, lds);
  else if (b < dw_blocks + dx_blocks) product_tile<T, false, true, false>(dx, b - dw_blocks, dx_blocks, lds);
  else add_db(db, b - dw_blocks - dx_blocks, reinterpret_cast<float*>(lds));
}

// Adds the parts of split products in part order and applies their epilogue; without any, adds db's.  Four columns per
// thread.
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
    const size_t step = (size_t)p.M * p.ldp;
    const float* in = p.partial + (size_t)m * p.ldp + n;
    if (n + 4 <= p.epi.N) {
#pragma unroll 4
      for (int s = 0; s < p.split; ++s) {
        float q[4];
        load4(in + s * step, 0, 0, q);
#pragma unroll
        for (int r = 0; r < 4; ++r) z[r] += q[r];
        if (pair) {
          load4(in + s * step, 0, p.epi.N, q);
#pragma unroll
          for (int r = 0; r < 4; ++r) zu[r] += q[r];
        }
      }
    } else {
      for (int s = 0; s < p.split; ++s) {
#pragma unroll
        for (int r = 0; r < 3; ++r)
          if (n + r < p.epi.N) {
            z[r] += in[s * step + r];
            if (pair) zu[r] += in[s * step + p.epi.N + r];
          }
      }
    }
    const auto value = [&](int, float (&a)[4], float (&u)[4]) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        a[r] = z[r];
        u[r] = zu[r];
      }
    };
    pair ? epi_rows<true, 1>(p.epi, m, n, 1, value) : epi_rows<false, 1>(p.epi, m, n, 1, value);
    return;
  }
  __shared__ float lds[256];
  add_db(jn.db, b, lds);
}

int64_t tiles_of(const Shape& s, int side) { return ceil_div(s.M, side) * ceil_div(s.R, side); }
int64_t steps_of(const Shape& s, int shape) { return ceil_div(s.K, kBK) * (shape == kDirect ? 1 : s.nseg); }

// Time of a launch in microseconds, from measurements of the tile shapes over 1 to 192 K-steps and 16 to 4,096 tiles:
// a workgroup costs a start and an epilogue besides its K-steps, less of each while it has a CU to itself, and a cut
// reduction costs a second launch and its parts' way through memory.
//   500 x 2048 x 1024: 64 x 64 tiles 12.1 us, 128 x 128 22.1;  65 x 4096 x 4096: 64 x 64 17.4 us, in four parts 14.6
//   fp32 A, two terms: 2048 x 512 x 512 7.9 us, x 4096 x 512 32.0; 4096 x 512 x 512 10.8 us, x 4096 x 512 49.8
//   fp32 A, three terms: 65 x 4096 x 4096 37.3 us, in two parts 24.7, as term planes 45.8;  2048 x 2048 x 512 21.6, as
//   planes 34.1, in two parts 26.2
//   8192 x 2048 x 1024: 128 x 128 tiles 37.5 us, 256 x 256 (half the CUs idle) 54, in two parts 41 + 15 for the join
//   8192 x 1024 x 2048: 43.8 against 38.8;  8192 x 4096 x 4096: 261 against 224
//   1024 x 8192 x 2048 in parts: one 117, two 57, four 47 us
struct Rates {
  int slots, side;              // workgroups at once, tile side
  double start, step;           // with all slots taken
  double start_alone, step_alone;  // up to half of them
};
constexpr Rates kRates[3] = {{512, 64, 2.2, 0.37, 1.9, 0.205}, {512, 128, 3.5, 0.99, 2.7, 0.58}, {256, 256, 13.0, 1.50, 10.5, 1.19}};
constexpr Rates kDirectRates[2] = {{512, 64, 2.7, 0.69, 2.5, 0.42}, {512, 64, 2.7, 0.92, 2.5, 0.52}};  // two terms, three

double cost_of(int shape, const Shape* s, const int* split, int count) {
  const Rates& r = shape == kDirect ? kDirectRates[s[0].nseg > 2] : kRates[shape];
  int64_t blocks = 0;
  double parts = 0;  // bytes of fp32 sums
  for (int i = 0; i < count; ++i) {
    blocks += tiles_of(s[i], r.side) * split[i];
    if (split[i] > 1) parts += 4.0 * split[i] * s[i].M * s[i].R;
  }
  const bool alone = blocks <= r.slots / 2;
  double sum = 0, longest = 0;
  for (int i = 0; i < count; ++i) {
    const int64_t steps = ceil_div(steps_of(s[i], shape), split[i]);
    const double d = alone ? r.start_alone + r.step_alone * steps : r.start + r.step * steps;
    const int64_t n = tiles_of(s[i], r.side) * split[i];
    sum += d * (count == 1 ? (double)(ceil_div(n, r.slots) * r.slots) : (double)n);
    longest = std::max(longest, d);
  }
  // 2 us of launch; parts are read again at about 5 TB/s, by a launch of 4 us (1024 x 8192 x 2048 in four parts: 8 us)
  return 2.0 + std::max(sum / r.slots, longest) + (parts > 0 ? 4.0 + parts / 5.0e6 : 0.0);
}

}  // namespace

// The tile shape and the parts of one or two products launched together: the cheapest of a few cuts by cost_of.
Plan plan_products(const Shape* s, int count) {
  Plan best{};
  double least = 0;
  for (int shape = 0; shape < (s[0].f32 ? 4 : 3); ++shape)
    for (int share = 1 << 20; share >= 8; share = share > 128 ? 128 : share / 2) {  // K-steps of a part, about
      Plan p{};
      p.shape = shape;
      for (int i = 0; i < count; ++i)
        p.split[i] = (int)std::max<int64_t>(1, std::min<int64_t>(16, (steps_of(s[i], shape) + share / 2) / share));
      double c;
      if (s[0].f32 && shape != kDirect) {  // a launch of its own writes the term planes
        Shape turn = s[0];
        turn.M = (int)ceil_div(s[0].M, s[0].turns);
        c = s[0].turns * (cost_of(shape, &turn, p.split, 1) + 4.0 + (4.0 + 2.0 * turn.nseg) * turn.M * turn.K / 5.0e6);
      } else {
        c = cost_of(shape, s, p.split, count);
      }
      if (least == 0 || c < least) {
        least = c;
        best = p;
      }
    }
  return best;
}

int tile_side(const Plan& plan) { return plan.shape == kDirect ? Direct::TM : kRates[plan.shape].side; }

moe_status launch_products(int kid, const Plan& plan, Prob* p, int count, bool grad, bool first_is_dw, const DbSum& db,
                           hipStream_t s, const char* what) {
  const int side = tile_side(plan);
  const int64_t db_blocks = db.db ? ceil_div(db.n, 64) : 0;
  int64_t blocks[2] = {0, 0};
  Join j{};
  for (int i = 0; i < count; ++i) {
    blocks[i] = tiles_of(Shape{p[i].M, p[i].R, p[i].K, p[i].nseg}, side) * p[i].split;
    // (SwiGLU tiles hold half as many output columns, of which there are half as many as rows of W)
    if (p[i].epi.act == MOE_ACT_SWIGLU) blocks[i] = ceil_div(p[i].M, side) * ceil_div(p[i].epi.N, side / 2) * p[i].split;
    j.p[i] = p[i];
    if (p[i].split > 1) (i ? j.n1 : j.n0) = (int)ceil_div((int64_t)p[i].M * ((p[i].epi.N + 3) / 4), 256);
  }
  const int64_t total = blocks[0] + blocks[1] + db_blocks;
  if (total > 0x7FFFFFFF) return fail(MOE_EUNSUPPORTED, std::string(what) + ": too many tiles");
  if (count == 0) {
    j.db = db;
    join_kernel<<<dim3((unsigned)db_blocks), 256, 0, s>>>(j);
    return check_launch(what);
  }
  const dim3 grid((unsigned)total);
  const bool pair = p[0].epi.act == MOE_ACT_SWIGLU;
  auto go = [&](auto tile) {
    using T = decltype(tile);
    const dim3 threads((unsigned)T::kThreads);
    auto forward = [&](auto kernel) { launch_k(kid, kernel, grid, threads, 0, s, p[0]); };
    if constexpr (std::is_same_v<T, Direct>) {
      if (p[0].terms == 2) pair ? forward(linear_product_kernel<T, true, 2>) : forward(linear_product_kernel<T, false, 2>);
      else pair ? forward(linear_product_kernel<T, true, 3>) : forward(linear_product_kernel<T, false, 3>);
    } else if (grad) {
      launch_k(kid, grad_products_kernel<T>, grid, threads, 0, s, p[0], p[count - 1], first_is_dw ? (int)blocks[0] : 0,
               first_is_dw ? (int)blocks[1] : (int)blocks[0], db);
    } else {
      pair ? forward(linear_product_kernel<T, true, 0>) : forward(linear_product_kernel<T, false, 0>);
    }
  };
  if (plan.shape == 0) go(Tiny{});
  else if (plan.shape == 1) go(Small{});
  else if (plan.shape == 2) go(Large{});
  else go(Direct{});
  if (moe_status st = check_launch(what)) return st;
  if (j.n0 + j.n1 > 0) {
    join_kernel<<<dim3((unsigned)(j.n0 + j.n1)), 256, 0, s>>>(j);
    return check_launch(what);
  }
  return MOE_OK;
}

}  // namespace moe
