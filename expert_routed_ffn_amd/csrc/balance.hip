// balance.hip -- the router's balance loss with its per-expert counts, and the gradient that reaches the logits.
//
// Token t takes part when the mask keeps it and its logits row holds anything above -inf; n such tokens.  With
// p_te = softmax over all E experts and c_e = number of (t, j) with ids[t][j] = e over the tokens that take part,
//   loss[0] = E / (n^2 k) * sum_e c_e * sum_t p_te      (1 when the experts are called evenly)
//   loss[1] = 1 / n * sum_t lse_t^2                     lse_t = log sum_e exp l_te
// The counts are constants of the gradient:
//   dl_te = d0 E / (n^2 k) * p_te (c_e - sum_f p_tf c_f) + d1 2 / n * lse_t p_te
// and the gate weights w = softmax over the k selected logits add, at e = ids[t][j], w_tj (dw_tj - sum_i w_ti dw_ti).
//
// Both kernels take one wave per row and hold the row in registers (E <= 1024: at most 16 values a lane), so each
// logit is read once per kernel; the loss has to be complete before its gradient can start.  A lane owns the same
// columns in every row of its wave, so the column sums of p stay in registers too and reach memory once per
// workgroup.  No atomics on floats: counts are integer LDS atomics, sums go through fixed-order partials, and two
// calls on the same inputs give the same bits.
#include "wave_dev.hpp"

namespace moe {
namespace {

// e^t for t <= 0 from the hardware's 2^h: the part of t log2(e) that h = fl(t log2 e) rounds off is put back to first
// order, 2^(h + l) = 2^h (1 + l ln 2 + O(l^2)) with |l| below 2^-17.  Without it the relative error grows with |t|
// (1e-6 at t = -20).  t is kept at -126 or above, whose exponential is 0 in fp32; fmaxf takes a NaN there too.
__device__ __forceinline__ float exp_neg(float t) {
  t = fmaxf(t, -126.0f);
  const float h = t * 1.44269502f;  // log2(e) = 1.44269502162933349609375 + 1.92596299e-8
  const float l = __builtin_fmaf(t, 1.92596299e-8f, __builtin_fmaf(t, 1.44269502f, -h));
  const float r = __builtin_amdgcn_exp2f(h);
  return __builtin_fmaf(r, l * 0.693147181f, r);
}

// Which columns a lane owns: with VEC (E % 4 == 0, 16-byte aligned rows) value i is column 256 (i / 4) + 4 lane +
// i % 4, loaded as 16-byte pieces; otherwise column 64 i + lane.
template <bool VEC>
__device__ __forceinline__ int col_of(int lane, int i) {
  return VEC ? 256 * (i >> 2) + 4 * lane + (i & 3) : 64 * i + lane;
}

// A row of logits to registers.  The loads stand under no condition, as a conditional one is waited for where its branch
// ends, which made each of a wave's loads a round trip of its own: columns past E read column 0 and are set to -inf by
// mask_row when the row is worked on.
template <int N, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, float (&v)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const int c = col_of<true>(lane, i);
      const float4 q = *reinterpret_cast<const float4*>(row + (c < E ? c : 0));
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = col_of<false>(lane, i);
      v[i] = row[c < E ? c : 0];
    }
  }
}
template <int N, bool VEC>
__device__ __forceinline__ void mask_row(int E, int lane, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (col_of<VEC>(lane, i) >= E) v[i] = kNegInf;
}

// v becomes exp(v - max) (0 where v = -inf).  Returns false when every value is -inf.  `inv` = 1 / sum of those
// exponentials, `lse` = log of the sum of the original exponentials; both NaN when a value is NaN or +inf.
template <int N>
__device__ __forceinline__ bool row_softmax(float (&v)[N], float& inv, float& lse) {
  float m = kNegInf;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    odd |= v[i] != v[i];
    m = fmaxf(m, v[i]);
  }
  m = wave_max(m);
  const bool bad = __ballot(odd) != 0 || m == -kNegInf;
  if (m == kNegInf && !bad) return false;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = exp_neg(v[i] - m);
    s += v[i];
  }
  s = wave_sum(s);
  if (bad) s = __builtin_nanf("");
  inv = 1.0f / s;
  lse = m + logf(s);
  return true;
}

// ---- the loss --------------------------------------------------------------------

constexpr int kLossWaves = 8;  // per workgroup
constexpr int kLossParts = 256;  // workgroups at most

struct LossParts {  // workspace
  double* cp;       // [column groups] sum of c_e P_e
  float* p;         // [parts][E] column sums of p
  int32_t* c;       // [parts][E] counts
  float* z;         // [parts] sum of lse^2
  int32_t* n;       // [parts] tokens that take part
  uint32_t* done;   // [1] column groups that are finished
};
constexpr int kJoinCols = 64, kJoinGroups = kMaxE / kJoinCols;

__host__ __device__ inline size_t loss_parts_bytes(int parts, int E) {
  return 8 * kJoinGroups + (size_t)parts * (8 * (size_t)E + 8) + 4;
}
__host__ __device__ inline LossParts loss_parts(void* ws, int parts, int E) {
  LossParts w;
  w.cp = reinterpret_cast<double*>(ws);
  w.p = reinterpret_cast<float*>(w.cp + kJoinGroups);
  w.c = reinterpret_cast<int32_t*>(w.p + (size_t)parts * E);
  w.z = reinterpret_cast<float*>(w.c + (size_t)parts * E);
  w.n = reinterpret_cast<int32_t*>(w.z + parts);
  w.done = reinterpret_cast<uint32_t*>(w.n + parts);
  return w;
}

// The losses from the whole sums, by one thread.
__device__ __forceinline__ void write_loss(double cp, double z, int n, int E, int k, float* loss, int32_t* counts) {
  const double dn = n;
  loss[0] = n ? (float)(cp * E / (dn * dn * k)) : 0.0f;
  loss[1] = n ? (float)(z / dn) : 0.0f;
  counts[E] = n;
}
template <typename V>
__device__ __forceinline__ V lanes_sum(V v) {  // (of types that wave_all does not take)
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Grid: `parts` workgroups of 8 waves; wave g of all takes rows g, g + waves, ..., U at a time: their loads are issued
// together, the next U rows' before the present ones are worked on.  With one workgroup the loss is written here;
// otherwise the workgroup's sums go to the workspace and balance_join_kernel adds them.
template <int N, bool VEC>
__global__ __launch_bounds__(64 * kLossWaves) void balance_rows_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int T, int E,
    int k, float* __restrict__ lse_out, float* __restrict__ loss, int32_t* __restrict__ counts, LossParts parts) {
  constexpr int U = N <= 8 ? 2 : 1;
  __shared__ float s_p[kLossWaves][64 * N];
  __shared__ int s_c[64 * N];
  __shared__ float s_z[kLossWaves];
  __shared__ int s_n[kLossWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < E; e += 64 * kLossWaves) s_c[e] = 0;
  __syncthreads();

  float psum[N];
#pragma unroll
  for (int i = 0; i < N; ++i) psum[i] = 0.0f;
  float zsum = 0.0f;
  int n = 0;
  const int step = gridDim.x * kLossWaves;
  int t = blockIdx.x * kLossWaves + wave;
  float next[U][N];
  int next_id[U], next_keep[U];
  auto fetch = [&](int r) {
#pragma unroll
    for (int u = 0; u < U; ++u, r += step) {
      const int row = min(r, T - 1);  // (past the end: the last row again, not worked on)
      load_row<N, VEC>(logits + (size_t)row * E, E, lane, next[u]);
      next_id[u] = ids[(size_t)row * k + min(lane, k - 1)];
      next_keep[u] = mask ? mask[row] : 1;
    }
  };
  if (T > 0) fetch(t);
  for (; t < T; t += U * step) {
    float v[U][N];
    int id[U], keep[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[u][i] = next[u][i];
      mask_row<N, VEC>(E, lane, v[u]);
      id[u] = lane < k ? next_id[u] : -1;
      keep[u] = next_keep[u];
    }
    if (t + U * step < T) fetch(t + U * step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u * step >= T) continue;
      float inv, lse = kNegInf;
      if (keep[u] && row_softmax<N>(v[u], inv, lse)) {
#pragma unroll
        for (int i = 0; i < N; ++i) psum[i] = __builtin_fmaf(v[u][i], inv, psum[i]);
        zsum = __builtin_fmaf(lse, lse, zsum);
        ++n;
        if ((unsigned)id[u] < (unsigned)E) atomicAdd(&s_c[id[u]], 1);
      } else {
        lse = kNegInf;
      }
      if (lane == 0) lse_out[t + u * step] = lse;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = col_of<VEC>(lane, i);
    if (c < E) s_p[wave][c] = psum[i];
  }
  if (lane == 0) {
    s_z[wave] = zsum;
    s_n[wave] = n;
  }
  __syncthreads();

  const bool alone = gridDim.x == 1;
  for (int e = tid; e < E; e += 64 * kLossWaves) {
    float p = s_p[0][e];
#pragma unroll
    for (int w = 1; w < kLossWaves; ++w) p += s_p[w][e];
    if (alone) {
      s_p[0][e] = p;
      counts[e] = s_c[e];
    } else {
      parts.p[(size_t)blockIdx.x * E + e] = p;
      parts.c[(size_t)blockIdx.x * E + e] = s_c[e];
    }
  }
  if (alone) __syncthreads();
  if (wave == 0) {
    float z = 0.0f;
    int nt = 0;
#pragma unroll
    for (int w = 0; w < kLossWaves; ++w) {
      z += s_z[w];
      nt += s_n[w];
    }
    if (alone) {
      double cp = 0.0;
      for (int e = lane; e < E; e += 64) cp += (double)s_p[0][e] * s_c[e];
      cp = lanes_sum(cp);
      if (lane == 0) write_loss(cp, z, nt, E, k, loss, counts);
    } else if (lane == 0) {
      parts.z[blockIdx.x] = z;
      parts.n[blockIdx.x] = nt;
      if (blockIdx.x == 0) *parts.done = 0;
    }
  }
}

// One workgroup of 16 waves per 64 columns: wave g adds parts g, g + 16, ... of its columns, the waves' shares are added
// in wave order.  The workgroup that finishes last (a counter that the launch before set to 0) adds the column groups'
// products, in one order whoever that is, and writes the losses.  All of it is latency: the parts' other sums are read
// by every workgroup's first wave at the start, beside its columns, and the products by one lane each at once.
__global__ __launch_bounds__(1024) void balance_join_kernel(LossParts parts, int nparts, int E, int k,
                                                            float* __restrict__ loss, int32_t* __restrict__ counts) {
  __shared__ float s_p[16][kJoinCols];
  __shared__ int s_c[16][kJoinCols];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.x * kJoinCols + lane;
  float p = 0.0f, zi[kLossParts / 64];
  int c = 0, ni[kLossParts / 64];
  if (wave == 0) {
#pragma unroll
    for (int i = 0; i < kLossParts / 64; ++i) {
      const int r = 64 * i + lane;
      zi[i] = r < nparts ? parts.z[r] : 0.0f;
      ni[i] = r < nparts ? parts.n[r] : 0;
    }
  }
  if (e < E) {
#pragma unroll 16
    for (int r = wave; r < nparts; r += 16) {
      p += parts.p[(size_t)r * E + e];
      c += parts.c[(size_t)r * E + e];
    }
  }
  s_p[wave][lane] = p;
  s_c[wave][lane] = c;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) {
    p += s_p[w][lane];
    c += s_c[w][lane];
  }
  if (e < E) counts[e] = c;
  double cp = lanes_sum((double)p * c);
  if (gridDim.x > 1) {
    uint32_t before = 0;
    if (lane == 0) {
      __hip_atomic_store(parts.cp + blockIdx.x, cp, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      before = __hip_atomic_fetch_add(parts.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(before) != gridDim.x - 1) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    cp = lane < (int)gridDim.x ? __hip_atomic_load(parts.cp + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
    cp = lanes_sum(cp);
  }
  double z = 0.0;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kLossParts / 64; ++i) {
    z += zi[i];
    n += ni[i];
  }
  z = lanes_sum(z);
  n = lanes_sum(n);
  if (lane == 0) write_loss(cp, z, n, E, k, loss, counts);
}

// Workgroups of balance_rows_kernel.  One takes all rows up to 64, which saves the second launch.
constexpr int kLossAloneRows = 64;
int loss_grid(int T) {
  if (T <= kLossAloneRows) return 1;
  return (int)std::min<int64_t>(kLossParts, ceil_div(T, kLossWaves));
}

// ---- the gradient ------------------------------------------------------------------

constexpr int kGradWaves = 4;

// One wave per row, U rows at a time, their loads issued together.  The gate part of a row has at most k entries:
// lanes 0..k-1 hold the selected experts, an expert named twice gets the sum of its entries on its first lane (in
// ascending j), and the wave's own LDS row carries them from those lanes to the lanes that own the columns.
template <int N, bool VEC>
__global__ __launch_bounds__(64 * kGradWaves) void route_backward_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ w,
    const float* __restrict__ dw, const float* __restrict__ lse_in, const int32_t* __restrict__ counts,
    const float* __restrict__ dloss, int T, int E, int k, float* __restrict__ dlogits) {
  constexpr int U = N <= 8 ? 2 : 1;
  __shared__ __attribute__((aligned(16))) float s_gate[kGradWaves][64 * N];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* gate = s_gate[wave];
  const bool has_gate = w != nullptr, has_loss = lse_in != nullptr;
  const int step = gridDim.x * kGradWaves;
  // ahead of the rows' loads, which would otherwise all have to land before the first row is worked on
  float cnt[N];
  float a = 0.0f, z2 = 0.0f;
  if (has_loss) {
#pragma unroll
    for (int i = 0; i < N; i += VEC ? 4 : 1) {
      const int c = col_of<VEC>(lane, i);
      if constexpr (VEC) {
        const int4 q = *reinterpret_cast<const int4*>(counts + (c < E ? c : 0));  // (of columns past E: times 0)
        cnt[i] = (float)q.x; cnt[i + 1] = (float)q.y; cnt[i + 2] = (float)q.z; cnt[i + 3] = (float)q.w;
      } else {
        cnt[i] = (float)counts[c < E ? c : 0];
      }
    }
    const float n = (float)counts[E];
    if (n > 0.0f) {
      a = dloss[0] * (float)E / (n * n * (float)k);
      z2 = 2.0f * dloss[1] / n;
    }
  }
  for (int t0 = blockIdx.x * kGradWaves + wave; t0 < T; t0 += U * step) {
    float v[U][N], wj[U], dwj[U], lse[U];
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t t = min(t0 + u * step, T - 1);  // (past the end: the last row again, not worked on)
      id[u] = -1;
      wj[u] = dwj[u] = lse[u] = 0.0f;
      if (has_loss) {
        load_row<N, VEC>(logits + t * E, E, lane, v[u]);
        lse[u] = lse_in[t];
      }
      if (has_gate) {
        const size_t at = t * k + min(lane, k - 1);
        id[u] = ids[at];
        wj[u] = w[at];
        dwj[u] = dw[at];
      }
    }
    if (t0 < step) {  // the wave's first rows
#pragma unroll
      for (int i = 0; i < N; ++i) gate[col_of<VEC>(lane, i)] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * step;
      if (t >= T) continue;
      const bool takes = !has_loss || !(lse[u] == kNegInf);  // the forward pass wrote -inf for rows that take no part
      float inv = 0.0f, own_lse = 0.0f;
      if (has_loss) mask_row<N, VEC>(E, lane, v[u]);
      if (has_loss && takes && row_softmax<N>(v[u], inv, own_lse)) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          v[u][i] *= inv;
          s = __builtin_fmaf(v[u][i], cnt[i], s);
        }
        s = wave_sum(s);
        const float z = z2 * lse[u];
#pragma unroll
        for (int i = 0; i < N; ++i) v[u][i] *= __builtin_fmaf(a, cnt[i] - s, z);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[u][i] = 0.0f;
      }
      if (has_gate && takes) {
        const float dot = wave_sum(lane < k ? wj[u] * dwj[u] : 0.0f);
        const float g = wj[u] * (dwj[u] - dot);
        float sum = g;
        bool first = lane < k && (unsigned)id[u] < (unsigned)E;
        // an expert named twice: the lanes that find another's mark at their place
        __builtin_amdgcn_wave_barrier();
        if (first) gate[id[u]] = __int_as_float(lane + 1);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const bool twice = first && __float_as_int(gate[id[u]]) != lane + 1;
        if (__ballot(twice) != 0) {
          sum = 0.0f;
          for (int i = 0; i < k; ++i) {
            const int idi = __builtin_amdgcn_readlane(id[u], i);
            const float gi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), i));
            if (idi == id[u]) {
              sum += gi;
              if (i < lane) first = false;
            }
          }
        }
        __builtin_amdgcn_wave_barrier();
        if (first) gate[id[u]] = sum;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if constexpr (VEC) {
#pragma unroll
          for (int i = 0; i < N; i += 4) {
            const float4 q = *reinterpret_cast<const float4*>(gate + col_of<true>(lane, i));
            v[u][i] += q.x; v[u][i + 1] += q.y; v[u][i + 2] += q.z; v[u][i + 3] += q.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) v[u][i] += gate[col_of<false>(lane, i)];
        }
        __builtin_amdgcn_wave_barrier();
        if (first) gate[id[u]] = 0.0f;  // clean for the wave's next row
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      float* out = dlogits + (size_t)t * E;
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const int c = col_of<true>(lane, i);
          if (c < E) *reinterpret_cast<float4*>(out + c) = make_float4(v[u][i], v[u][i + 1], v[u][i + 2], v[u][i + 3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = col_of<false>(lane, i);
          if (c < E) out[c] = v[u][i];
        }
      }
    }
  }
}

constexpr int kGradGrid = 1024;  // workgroups at most: four per CU, which are there at once

}  // namespace

size_t balance_loss_ws_bytes(int T, int E) {
  const int parts = loss_grid(T);
  return parts == 1 ? 0 : loss_parts_bytes(parts, E);
}

moe_status launch_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int T, int E, int k,
                               float* loss, int32_t* counts, float* lse, void* ws, hipStream_t s) {
  const int parts = loss_grid(T);
  const LossParts w = parts == 1 ? LossParts{} : loss_parts(ws, parts, E);
  const bool vec = E % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
  auto go = [&](auto kernel) {
    launch_k(MOE_KERNEL_BALANCE, kernel, dim3((unsigned)parts), dim3(64 * kLossWaves), 0, s, logits, ids, mask, T, E, k,
             lse, loss, counts, w);
  };
  if (E <= 256) vec ? go(balance_rows_kernel<4, true>) : go(balance_rows_kernel<4, false>);
  else if (E <= 512) vec ? go(balance_rows_kernel<8, true>) : go(balance_rows_kernel<8, false>);
  else vec ? go(balance_rows_kernel<16, true>) : go(balance_rows_kernel<16, false>);
  if (moe_status st = check_launch("balance_loss")) return st;
  if (parts == 1) return MOE_OK;
  balance_join_kernel<<<dim3((unsigned)ceil_div(E, kJoinCols)), 1024, 0, s>>>(w, parts, E, k, loss, counts);
  return check_launch("balance_loss");
}

moe_status launch_route_backward(const float* logits, const int32_t* ids, const float* w, const float* dw,
                                 const float* lse, const int32_t* counts, const float* dloss, int T, int E, int k,
                                 float* dlogits, hipStream_t s) {
  const bool vec = E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits) | reinterpret_cast<uintptr_t>(counts)) % 16 == 0;
  const unsigned grid = (unsigned)std::min<int64_t>(kGradGrid, ceil_div(T, kGradWaves));
  auto go = [&](auto kernel) {
    launch_k(MOE_KERNEL_ROUTE_BACKWARD, kernel, dim3(grid), dim3(64 * kGradWaves), 0, s, logits, ids, w, dw, lse, counts,
             dloss, T, E, k, dlogits);
  };
  if (E <= 256) vec ? go(route_backward_kernel<4, true>) : go(route_backward_kernel<4, false>);
  else if (E <= 512) vec ? go(route_backward_kernel<8, true>) : go(route_backward_kernel<8, false>);
  else vec ? go(route_backward_kernel<16, true>) : go(route_backward_kernel<16, false>);
  return check_launch("route_backward");
}

}  // namespace moe
