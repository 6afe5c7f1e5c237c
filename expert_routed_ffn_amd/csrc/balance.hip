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
#include "internal.hpp"

namespace moe {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();

// e^t for t <= 0 from the hardware's 2^h: the part of t * log2(e) that h = fl(t * log2 e) rounds off is put back to
// first order, 2^(h + l) = 2^h (1 + l ln 2 + O(l^2)) with |l| below 2^-17.  Without it the relative error grows
// with |t| (1e-6 at t = -20).  Below -120 the result is 0 in fp32 terms; a NaN fails the comparison and stays one.
__device__ __forceinline__ float exp_neg(float t) {
  const float h = t * 1.44269502f;  // log2(e) = 1.44269502162933349609375 + 1.92596299e-8
  const float l = __builtin_fmaf(t, 1.44269502f, -h) + t * 1.92596299e-8f;
  const float r = __builtin_amdgcn_exp2f(h);
  return t < -120.0f ? 0.0f : __builtin_fmaf(r, l * 0.693147181f, r);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}

// Which columns a lane owns: with VEC (E % 4 == 0, 16-byte aligned rows) value i is column 256 (i / 4) + 4 lane +
// i % 4, loaded as 16-byte pieces; otherwise column 64 i + lane.
template <bool VEC>
__device__ __forceinline__ int col_of(int lane, int i) {
  return VEC ? 256 * (i >> 2) + 4 * lane + (i & 3) : 64 * i + lane;
}

// A row of logits in registers; columns past E read as -inf.
template <int N, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, float (&v)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const int c = col_of<true>(lane, i);
      const float4 q = c < E ? *reinterpret_cast<const float4*>(row + c) : make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = col_of<false>(lane, i);
      v[i] = c < E ? row[c] : kNegInf;
    }
  }
}

// v becomes exp(v - max) (0 where v = -inf).  Returns false when every value is -inf.  `inv` = 1 / sum of those
// exponentials, `lse` = log of the sum of the original exponentials.
template <int N>
__device__ __forceinline__ bool row_softmax(float (&v)[N], float& inv, float& lse) {
  float m = kNegInf;
  bool any = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    any |= !(v[i] == kNegInf);  // a NaN counts: it has to show in the results
    m = fmaxf(m, v[i]);
  }
  if (__ballot(any) == 0) return false;
  m = wave_max(m);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = v[i] == kNegInf ? 0.0f : exp_neg(v[i] - m);
    s += v[i];
  }
  s = wave_sum(s);
  inv = 1.0f / s;
  lse = m + logf(s);
  return true;
}

// ---- the loss --------------------------------------------------------------------

constexpr int kLossWaves = 8;  // per workgroup

struct LossParts {  // workspace: per workgroup
  float* p;         // [parts][E] column sums of p
  int32_t* c;       // [parts][E] counts
  float* z;         // [parts] sum of lse^2
  int32_t* n;       // [parts] tokens that take part
};

__host__ __device__ inline size_t loss_parts_bytes(int parts, int E) { return (size_t)parts * (8 * (size_t)E + 8); }
__host__ __device__ inline LossParts loss_parts(void* ws, int parts, int E) {
  LossParts w;
  w.p = reinterpret_cast<float*>(ws);
  w.c = reinterpret_cast<int32_t*>(w.p + (size_t)parts * E);
  w.z = reinterpret_cast<float*>(w.c + (size_t)parts * E);
  w.n = reinterpret_cast<int32_t*>(w.z + parts);
  return w;
}

// loss from the whole sums; called by the first wave of one workgroup with this lane's share of sum_e c_e P_e.
__device__ __forceinline__ void write_loss(double cp, double z, int n, int E, int k, int lane, float* loss,
                                           int32_t* counts) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) cp += __shfl_xor(cp, off, 64);
  if (lane) return;
  const double dn = n;
  loss[0] = n ? (float)(cp * E / (dn * dn * k)) : 0.0f;
  loss[1] = n ? (float)(z / dn) : 0.0f;
  counts[E] = n;
}

// Grid: `parts` workgroups of 8 waves; wave g of all takes rows g, g + waves, ...; the next row is loaded while the
// present one is worked on.  With one workgroup the loss is written here; otherwise the workgroup's sums go to the
// workspace and balance_join_kernel adds them.
template <int N, bool VEC>
__global__ __launch_bounds__(64 * kLossWaves) void balance_rows_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int T, int E,
    int k, float* __restrict__ lse_out, float* __restrict__ loss, int32_t* __restrict__ counts, LossParts parts) {
  __shared__ float s_p[kLossWaves][kMaxE];
  __shared__ int s_c[kMaxE];
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
  float next[N];
  int next_id = -1, next_keep = 0;
  auto fetch = [&](int r) {
    load_row<N, VEC>(logits + (size_t)r * E, E, lane, next);
    next_id = lane < k ? ids[(size_t)r * k + lane] : -1;
    next_keep = mask ? mask[r] : 1;
  };
  if (t < T) fetch(t);
  for (; t < T; t += step) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = next[i];
    const int id = next_id, keep = next_keep;
    if (t + step < T) fetch(t + step);
    float inv, lse = kNegInf;
    if (keep && row_softmax<N>(v, inv, lse)) {
#pragma unroll
      for (int i = 0; i < N; ++i) psum[i] = __builtin_fmaf(v[i], inv, psum[i]);
      zsum = __builtin_fmaf(lse, lse, zsum);
      ++n;
      if ((unsigned)id < (unsigned)E) atomicAdd(&s_c[id], 1);
    } else {
      lse = kNegInf;
    }
    if (lane == 0) lse_out[t] = lse;
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
      write_loss(cp, z, nt, E, k, lane, loss, counts);
    } else if (lane == 0) {
      parts.z[blockIdx.x] = z;
      parts.n[blockIdx.x] = nt;
    }
  }
}

// One workgroup of 1024 threads: thread (g, e) adds the parts g, g + G, ... of column e (G = 1024 / columns rounded
// to 64), then the G shares of each column and the products with the counts are added in a fixed order.
__global__ __launch_bounds__(1024) void balance_join_kernel(LossParts parts, int nparts, int E, int k,
                                                            float* __restrict__ loss, int32_t* __restrict__ counts) {
  __shared__ float s_p[1024];
  __shared__ int s_c[1024];
  __shared__ double s_cp[16];
  __shared__ float s_z[16];
  __shared__ int s_n[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cols = (E + 63) & ~63, G = 1024 / cols;
  const int g = tid / cols, e = tid - g * cols;
  float p = 0.0f;
  int c = 0;
  if (g < G && e < E) {
#pragma unroll 8
    for (int r = g; r < nparts; r += G) {
      p += parts.p[(size_t)r * E + e];
      c += parts.c[(size_t)r * E + e];
    }
  }
  s_p[tid] = p;
  s_c[tid] = c;
  float z = 0.0f;
  int n = 0;
  for (int r = tid; r < nparts; r += 1024) {
    z += parts.z[r];
    n += parts.n[r];
  }
  z = wave_sum(z);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off, 64);
  __syncthreads();
  double cp = 0.0;
  if (tid < E) {  // then g = 0 and e = tid
    for (int h = 1; h < G; ++h) {
      p += s_p[h * cols + e];
      c += s_c[h * cols + e];
    }
    counts[e] = c;
    cp = (double)p * c;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) cp += __shfl_xor(cp, off, 64);
  if (lane == 0) {
    s_cp[wave] = cp;
    s_z[wave] = z;
    s_n[wave] = n;
  }
  __syncthreads();
  if (wave == 0) {
    double zt = 0.0;
    int nt = 0;
    for (int w = 0; w < 16; ++w) {
      zt += s_z[w];
      nt += s_n[w];
    }
    write_loss(lane < 16 ? s_cp[lane] : 0.0, zt, nt, E, k, lane, loss, counts);
  }
}

// Workgroups of balance_rows_kernel.  One takes all rows up to 64 (8 per wave), which saves the second launch.
constexpr int kLossAloneRows = 64, kLossParts = 128;
int loss_grid(int T) {
  if (T <= kLossAloneRows) return 1;
  return (int)std::min<int64_t>(kLossParts, ceil_div(T, kLossWaves));
}

// ---- the gradient ------------------------------------------------------------------

constexpr int kGradWaves = 4;

// Grid-stride over rows, one wave per row.  The gate part of a row has at most k entries: lanes 0..k-1 hold the
// selected experts, an expert named twice gets the sum of its entries on its first lane (in ascending j), and the
// wave's own LDS row carries them from those lanes to the lanes that own the columns.
template <int N, bool VEC>
__global__ __launch_bounds__(64 * kGradWaves) void route_backward_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ w,
    const float* __restrict__ dw, const float* __restrict__ lse_in, const int32_t* __restrict__ counts,
    const float* __restrict__ dloss, int T, int E, int k, float* __restrict__ dlogits) {
  __shared__ __attribute__((aligned(16))) float s_gate[kGradWaves][kMaxE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* gate = s_gate[wave];
  const bool has_gate = w != nullptr, has_loss = lse_in != nullptr;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = col_of<VEC>(lane, i);
    if (c < E) gate[c] = 0.0f;
  }
  float cnt[N];
  float a = 0.0f, z2 = 0.0f;
  if (has_loss) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = col_of<VEC>(lane, i);
      cnt[i] = c < E ? (float)counts[c] : 0.0f;
    }
    const float n = (float)counts[E];
    if (n > 0.0f) {
      a = dloss[0] * (float)E / (n * n * (float)k);
      z2 = 2.0f * dloss[1] / n;
    }
  }
  const int step = gridDim.x * kGradWaves;
  int t = blockIdx.x * kGradWaves + wave;
  float next[N];
  int next_id = -1;
  float next_w = 0.0f, next_dw = 0.0f, next_lse = 0.0f;
  auto fetch = [&](int r) {
    if (has_loss) {
      load_row<N, VEC>(logits + (size_t)r * E, E, lane, next);
      next_lse = lse_in[r];
    }
    if (has_gate && lane < k) {
      next_id = ids[(size_t)r * k + lane];
      next_w = w[(size_t)r * k + lane];
      next_dw = dw[(size_t)r * k + lane];
    }
  };
  if (t < T) fetch(t);
  for (; t < T; t += step) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = has_loss ? next[i] : 0.0f;
    const int id = next_id;
    const float wj = next_w, dwj = next_dw, lse = next_lse;
    if (t + step < T) fetch(t + step);
    const bool takes = !has_loss || !(lse == kNegInf);  // the forward pass wrote -inf for rows that take no part
    float inv = 0.0f, own_lse = 0.0f;
    if (has_loss && takes && row_softmax<N>(v, inv, own_lse)) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] *= inv;
        s = __builtin_fmaf(v[i], cnt[i], s);
      }
      s = wave_sum(s);
      const float z = z2 * lse;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= __builtin_fmaf(a, cnt[i] - s, z);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.0f;
    }
    bool first = false;
    if (has_gate && takes) {
      const float dot = wave_sum(lane < k ? wj * dwj : 0.0f);
      const float g = wj * (dwj - dot);
      float sum = 0.0f;
      first = lane < k && (unsigned)id < (unsigned)E;
      for (int i = 0; i < k; ++i) {
        const int idi = __builtin_amdgcn_readlane(id, i);
        const float gi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), i));
        if (idi == id) {
          sum += gi;
          if (i < lane) first = false;
        }
      }
      __builtin_amdgcn_wave_barrier();
      if (first) gate[id] = sum;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const int c = col_of<true>(lane, i);
          if (c < E) {
            const float4 q = *reinterpret_cast<const float4*>(gate + c);
            v[i] += q.x; v[i + 1] += q.y; v[i + 2] += q.z; v[i + 3] += q.w;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = col_of<false>(lane, i);
          if (c < E) v[i] += gate[c];
        }
      }
      __builtin_amdgcn_wave_barrier();
      if (first) gate[id] = 0.0f;  // clean for the wave's next row
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    float* out = dlogits + (size_t)t * E;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const int c = col_of<true>(lane, i);
        if (c < E) *reinterpret_cast<float4*>(out + c) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = col_of<false>(lane, i);
        if (c < E) out[c] = v[i];
      }
    }
  }
}

constexpr int kGradGrid = 512;  // workgroups at most: two per CU

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
  balance_join_kernel<<<1, 1024, 0, s>>>(w, parts, E, k, loss, counts);
  return check_launch("balance_loss");
}

moe_status launch_route_backward(const float* logits, const int32_t* ids, const float* w, const float* dw,
                                 const float* lse, const int32_t* counts, const float* dloss, int T, int E, int k,
                                 float* dlogits, hipStream_t s) {
  const bool vec = E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits)) % 16 == 0;
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
