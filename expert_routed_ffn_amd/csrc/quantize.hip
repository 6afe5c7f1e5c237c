// quantize.hip -- rows to 8-bit codes and one scale each (arithmetic in quantize_dev.hpp).
//
// Memory-bound: each row is read once and held in registers between its maximum and its codes.  Up to 4,096 columns a
// wave takes a row (4 rows a workgroup, no barrier), beyond that a workgroup of 256 threads does.  8,192 rows of 2,048 bf16
// values take 10.1 us and of 4,096 18.5, 5.0 and 5.4 TB/s, where a 1 GiB copy has 5.1; 1,001 rows of 4,096 fp32 values 5.1
// (4 at the copy's rate).
#include "quantize_dev.hpp"

namespace moe {
namespace {

// N: groups of 8 values a lane holds; WAVES waves share a row.
template <bool F32, int N, int WAVES>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* __restrict__ x, int T, int K,
                                                            int8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int kRows = 4 / WAVES, kLanes = 64 * WAVES;
  const int64_t row = (int64_t)blockIdx.x * kRows + (WAVES == 1 ? threadIdx.x >> 6 : 0);
  if (row >= T) return;
  const int lane = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const size_t at = (size_t)row * K;
  Eight<F32> v[N];
  // (groups past the row's end read its last one again, which changes no maximum)
#pragma unroll
  for (int i = 0; i < N; ++i) v[i].load(x, at + min((i * kLanes + lane) * 8, K - 8));
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, amax_bits(v[i]));
  m = wave_max_u32(m);
  if constexpr (WAVES > 1) {
    __shared__ uint32_t parts[WAVES];
    if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WAVES; ++i) m = max(m, parts[i]);
  }
  const RowScale r = row_scale(m);
  if (lane == 0) scale[row] = r.s;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * kLanes + lane) * 8;
    if (c >= K) break;
    float f[8];
    v[i].get(f);
    *reinterpret_cast<uint2*>(q + at + c) = finite_bits(m) ? codes8(f, r) : make_uint2(0, 0);
  }
}

}  // namespace

moe_status launch_quantize_rows(const void* x, moe_dtype x_t, int T, int K, int8_t* q, float* scale, hipStream_t s) {
  const bool f = x_t == MOE_F32;
  auto go = [&](auto kernel, int rows) {
    launch_k(MOE_KERNEL_QUANTIZE, kernel, dim3((unsigned)ceil_div(T, rows)), dim3(256), 0, s, x, T, K, q, scale);
  };
  if (K <= 512) f ? go(quantize_rows_kernel<true, 1, 1>, 4) : go(quantize_rows_kernel<false, 1, 1>, 4);
  else if (K <= 1024) f ? go(quantize_rows_kernel<true, 2, 1>, 4) : go(quantize_rows_kernel<false, 2, 1>, 4);
  else if (K <= 2048) f ? go(quantize_rows_kernel<true, 4, 1>, 4) : go(quantize_rows_kernel<false, 4, 1>, 4);
  else if (K <= 4096) f ? go(quantize_rows_kernel<true, 8, 1>, 4) : go(quantize_rows_kernel<false, 8, 1>, 4);
  else if (K <= 8192) f ? go(quantize_rows_kernel<true, 4, 4>, 1) : go(quantize_rows_kernel<false, 4, 4>, 1);
  else f ? go(quantize_rows_kernel<true, 8, 4>, 1) : go(quantize_rows_kernel<false, 8, 4>, 1);
  return check_launch("quantize_rows");
}

}  // namespace moe
