// product_dev.hpp -- the main loop of a tiled matrix product, for the kernels that put their own epilogue behind it:
// tile shapes, loaders of operands into LDS, readers of fragments, and product_loop.  What each part does and measured is
// told where it was built, at the head of product.hip.
//
// Memory is handled in 16-bit words whatever the values are: bf16 and fp16 are one word each, two 8-bit integers share
// one, so that a step of kBK words holds 64 or 128 values of the reduction and every place in LDS is the same.
#pragma once

#include <algorithm>
#include <type_traits>

#include "linear_dev.hpp"

namespace moe {
namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
constexpr int kBK = 64;

template <int TM_, int TN_, int WM_, int WN_, int BUFFERS = 2, int KG_ = 1, int A_BYTES = 2>
struct Tile {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, kRing = BUFFERS;
  static constexpr int KG = KG_;  // groups of WM x WN waves: with two, each multiplies one 32-k half of every step
  static constexpr int kThreads = 64 * WM * WN * KG;
  static constexpr int kFM = TM / WM / 16, kFN = TN / WN / 16;  // 16 x 16 fragments per wave
  static constexpr int kStageA = TM * kBK * A_BYTES / 2;        // 16-bit words of A's part of a buffer
  static constexpr int kStage = kStageA + TN * kBK;             // and of all of it
  static constexpr int kBuffers = kRing * kStage * 2;           // bytes
  // the fp32 tile passes through the same LDS, in one piece or by rows of waves
  static constexpr int kPasses = TM * TN * 4 <= 64 * 1024 ? 1 : WM;
  static constexpr int kLds = std::max(kBuffers, TM * TN * 4 / kPasses);
};
using Tiny = Tile<64, 64, 2, 2, 5, 2>;
using Direct = Tile<64, 64, 4, 1, 3, 2, 4>;  // A is fp32
using Small = Tile<128, 128, 2, 2>;
using Large = Tile<256, 256, 2, 4>;
static_assert(std::max({Tiny::kLds, Direct::kLds, Small::kLds}) <= 80 * 1024 && Large::kLds <= 160 * 1024, "LDS of a CU");

// Workgroup number to work item: each of the 8 dies (workgroup b runs on die b % 8) gets one contiguous range of
// items, so that neighbouring tiles share its L2.
__device__ __forceinline__ int die_item(int b, int total) {
  const int per = total >> 3, rem = total & 7, x = b & 7;
  return x * per + min(x, rem) + (b >> 3);
}

__device__ __forceinline__ void to_lds16(const void* g, uint16_t* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)g,
                                   (__attribute__((address_space(3))) uint32_t*)l, 16, 0, 0);
}

// A value that is the same in every lane, kept in a scalar register (integer divisions leave theirs in vector ones).
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Four values of a column by ds_read_b64_tr_b16.  The compiler takes a read it knows nothing about to wait for every
// load into LDS that is under way; `p` being restrict tells it that this one does not (hand_over below orders the two).
// Without it the gradient's products waited for each step's loads right after issuing them.
__device__ __forceinline__ s16x4_t read_tr(const uint16_t* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)p);
}

// (restrict for the same reason: with it 65 x 4096 x 4096 took 37 us, without 55)
__device__ __forceinline__ f32x4_t read_f32(const float* __restrict__ p) { return *reinterpret_cast<const f32x4_t*>(p); }

// Loader and reader of one operand's tile: ROWS indices (m or n) by 64 k.  `w64` is the wave's first thread.
template <int ROWS, int THREADS, bool KROWS>
struct Operand;

template <int ROWS, int THREADS>
struct Operand<ROWS, THREADS, false> {  // [m][k]
  static constexpr int kPer = THREADS / 8, kLoads = ROWS / kPer;
  uint32_t off[kLoads];  // from the tile's first row
  int chunk;             // which 16 bytes of a row this thread brings
  // `row(i)` is the source row, relative to the tile's first, of tile row i
  template <typename Row>
  __device__ __forceinline__ void init(int ld, int, Row row) {
    const int r = threadIdx.x >> 3;
    chunk = (threadIdx.x & 7) ^ ((r >> 1) & 7);  // kPer is a multiple of 16: the same for each load
#pragma unroll
    for (int i = 0; i < kLoads; ++i) off[i] = (uint32_t)row(r + kPer * i) * ld + chunk * 8;
  }
  __device__ __forceinline__ const uint16_t* at(const uint16_t* p, size_t first, int k0, int ld) const {
    return p + first * ld + k0;
  }
  __device__ __forceinline__ void load(const uint16_t* p, int, uint16_t* lds, int w64) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) to_lds16(p + off[i], lds + (i * THREADS + w64) * 8);
  }
  // the last step of a reduction that is no multiple of 64: `left` k are there, the others become zeros
  __device__ __forceinline__ void load_tail(const uint16_t* p, int, int left, uint16_t* lds) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint4 v = chunk * 8 < left ? *reinterpret_cast<const uint4*>(p + off[i]) : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(lds + (i * THREADS + threadIdx.x) * 8) = v;
    }
  }
  // a last step whose fragments are masked when they are read: what is not there takes the first values again
  __device__ __forceinline__ void load_short(const uint16_t* p, int, int left, uint16_t* lds, int w64) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) to_lds16(p + off[i] - (chunk * 8 < left ? 0 : chunk * 8), lds + (i * THREADS + w64) * 8);
  }
  template <int F>
  __device__ __forceinline__ void read(const uint16_t* lds, int base, int kk, bf16x8_t (&f)[F]) const {
    const int r16 = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const int row = base + 16 * i + r16;
      f[i] = *reinterpret_cast<const bf16x8_t*>(lds + row * kBK + (((4 * kk + q) ^ ((row >> 1) & 7)) * 8));
    }
  }
};

template <int ROWS, int THREADS>
struct Operand<ROWS, THREADS, true> {  // [k][m]
  static constexpr int kSlots = ROWS / 8, kPer = THREADS / kSlots, kLoads = kBK / kPer;  // 16-byte pieces of a row; k per load
  static_assert(kPer % 16 == 0, "the turn repeats");
  uint32_t off;
  // what row k's stretches are turned by; of 64 columns two rows fill 256 bytes, so every other k turns
  static __device__ __forceinline__ int turn(int k_mod4, int k8) {
    return ROWS >= 128 ? k_mod4 | k8 << 2 : k_mod4 >> 1 | k8 << 1;
  }
  template <typename Row>
  __device__ __forceinline__ void init(int ld, int cols, Row) {
    const int k = threadIdx.x / kSlots, s = threadIdx.x % kSlots;
    const int c = s ^ (turn(k & 3, (k >> 3) & 1) << 1);  // kPer is a multiple of 16: the same for each load
    // `cols` columns are there from the tile's first on (a multiple of 8); further ones repeat the last and are not stored
    off = (uint32_t)k * ld + min(c * 8, cols - 8);
  }
  __device__ __forceinline__ const uint16_t* at(const uint16_t* p, size_t first, int k0, int ld) const {
    return p + (size_t)k0 * ld + first;
  }
  __device__ __forceinline__ void load(const uint16_t* p, int ld, uint16_t* lds, int w64) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) to_lds16(p + off + (uint32_t)i * kPer * ld, lds + (i * THREADS + w64) * 8);
  }
  __device__ __forceinline__ void load_tail(const uint16_t* p, int ld, int left, uint16_t* lds) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool in = i * kPer + (int)threadIdx.x / kSlots < left;
      const uint4 v = in ? *reinterpret_cast<const uint4*>(p + off + (uint32_t)i * kPer * ld) : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(lds + (i * THREADS + threadIdx.x) * 8) = v;
    }
  }
  __device__ __forceinline__ void load_short(const uint16_t* p, int ld, int left, uint16_t* lds, int w64) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int k = i * kPer + (int)threadIdx.x / kSlots;
      to_lds16(p + off + (uint32_t)i * kPer * ld - (k < left ? 0u : (uint32_t)k * ld), lds + (i * THREADS + w64) * 8);
    }
  }
  template <int F>
  __device__ __forceinline__ void read(const uint16_t* lds, int base, int kk, bf16x8_t (&f)[F]) const {
    const int l16 = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;
    const int g = turn(l16 >> 2, q & 1);
    // lane l16 of a group of 16 reads 4 columns (l16 % 4) of k = 8 q + l16 / 4 (then 4 further) and gets column l16
    const uint16_t* p = lds + (32 * kk + 8 * q + (l16 >> 2)) * ROWS + (l16 & 3) * 4;
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const uint16_t* s = p + (((base >> 4) + i) ^ g) * 16;
      const s16x4_t a = read_tr(s);
      const s16x4_t b = read_tr(s + 4 * ROWS);
      f[i] = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// [m][k] of fp32 values, split into TERMS bf16 terms as they are read (fragments of one row group: its terms in order).
template <int ROWS, int THREADS, int TERMS>
struct OperandF32 {
  static constexpr int kPer = THREADS / 16, kLoads = ROWS / kPer;
  uint32_t off[kLoads];
  int chunk;  // which 16 bytes of a row's 256 this thread brings; piece c of row m lies at c ^ (m % 16)
  template <typename Row>
  __device__ __forceinline__ void init(int ld, int, Row row) {
    const int r = threadIdx.x >> 4;
    chunk = (threadIdx.x & 15) ^ (r & 15);  // kPer is a multiple of 16: the same for each load
    static_assert(kPer % 16 == 0, "the turn repeats");
#pragma unroll
    for (int i = 0; i < kLoads; ++i) off[i] = (uint32_t)row(r + kPer * i) * ld + chunk * 4;
  }
  __device__ __forceinline__ const float* at(const float* p, size_t first, int k0, int ld) const {
    return p + first * ld + k0;
  }
  __device__ __forceinline__ void load(const float* p, int, uint16_t* lds, int w64) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) to_lds16(p + off[i], lds + (i * THREADS + w64) * 8);
  }
  __device__ __forceinline__ void load_short(const float* p, int, int left, uint16_t* lds, int w64) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) to_lds16(p + off[i] - (chunk * 4 < left ? 0 : chunk * 4), lds + (i * THREADS + w64) * 8);
  }
  template <int F>
  __device__ __forceinline__ void read(const uint16_t* lds, int base, int kk, bf16x8_t (&f)[F]) const {
    const int r16 = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;
#pragma unroll
    for (int i = 0; i < F / TERMS; ++i) {
      const float* row = reinterpret_cast<const float*>(lds) + (base + 16 * i + r16) * kBK;
      const int c = 8 * kk + 2 * q;
      const f32x4_t a = read_f32(row + (c ^ r16) * 4);
      const f32x4_t b = read_f32(row + ((c + 1) ^ r16) * 4);
      uint32_t t[4][TERMS];
      split_terms<TERMS>(a.x, a.y, t[0]);
      split_terms<TERMS>(a.z, a.w, t[1]);
      split_terms<TERMS>(b.x, b.y, t[2]);
      split_terms<TERMS>(b.z, b.w, t[3]);
#pragma unroll
      for (int k = 0; k < TERMS; ++k)
        f[i * TERMS + k] = __builtin_bit_cast(bf16x8_t, make_uint4(t[0][k], t[1][k], t[2][k], t[3][k]));
    }
  }
};

// Fragments with k = first + 8 (lane / 16) ... : values at `left` and past it become zeros.
template <int F>
__device__ __forceinline__ void mask_k(bf16x8_t (&f)[F], int first, int left) {
  const int k = first + 8 * ((threadIdx.x >> 4) & 3);
#pragma unroll
  for (int i = 0; i < F; ++i) {
    uint4 q = __builtin_bit_cast(uint4, f[i]);
    uint32_t* w = &q.x;
#pragma unroll
    for (int d = 0; d < 4; ++d) w[d] &= (k + 2 * d < left ? 0xFFFFu : 0u) | (k + 2 * d + 1 < left ? 0xFFFF0000u : 0u);
    f[i] = __builtin_bit_cast(bf16x8_t, q);
  }
}

// What the matrix units multiply: a fragment is 16 bytes of a row, a lane's accumulator four rows of B by one of A.
struct KindBf16 {
  typedef f32x4_t Acc;
  static __device__ __forceinline__ Acc mma(bf16x8_t b, bf16x8_t a, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
  }
};

typedef int i32x4_t __attribute__((ext_vector_type(4)));
struct KindI8 {  // a fragment holds 16 values of k; sums are exact
  typedef i32x4_t Acc;
  static __device__ __forceinline__ Acc mma(bf16x8_t b, bf16x8_t a, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, b), __builtin_bit_cast(i32x4_t, a), c, 0, 0, 0);
  }
};
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
struct KindF16 {
  typedef f32x4_t Acc;
  static __device__ __forceinline__ Acc mma(bf16x8_t b, bf16x8_t a, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, b), __builtin_bit_cast(f16x8_t, a), c, 0, 0, 0);
  }
};

// Hands the buffers over: this wave's loads into one have landed and its reads of the other are done, then everyone's.
__device__ __forceinline__ void hand_over() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Sums of steps lo ... hi - 1 (of ceil(K / kBK) for each of p.nseg segments) of the tile whose first rows are m0 and n0;
// row_a(r) and row_b(r) are the source rows, relative to m0 and n0, of tile row r.  AK, BK: the operand is [k][index].
// TERMS: A is fp32 and enters as so many bf16 terms, split here; 0: A is of KIND.
template <typename T, bool AK, bool BK, int TERMS, typename KIND, typename RowA, typename RowB>
__device__ __forceinline__ void product_loop(const Mats& p, int m0, int n0, int lo, int hi, RowA row_a, RowB row_b,
                                             uint8_t* lds, typename KIND::Acc (&acc)[T::kFM][T::kFN]) {
  constexpr int TM = T::TM, TN = T::TN, WM = T::WM, WN = T::WN, kFM = T::kFM, kFN = T::kFN, kThreads = T::kThreads;
  const int wave = uniform(threadIdx.x >> 6);
  const int kg = wave / (WM * WN), wm = T::KG == 1 ? wave / WN : wave / WN % WM, wn = wave % WN;
  using LoaderA = std::conditional_t<TERMS != 0, OperandF32<TM, kThreads, std::max(TERMS, 1)>, Operand<TM, kThreads, AK>>;
  using ValueA = std::conditional_t<TERMS != 0, float, uint16_t>;
  constexpr int kTerms = std::max(TERMS, 1);
  LoaderA A;
  Operand<TN, kThreads, BK> B;
  A.init(p.lda, p.lda - m0, row_a);
  B.init(p.ldb, p.ldb - n0, row_b);
  const int seg_steps = (p.K + kBK - 1) / kBK;
  uint16_t* const base = reinterpret_cast<uint16_t*>(lds);
  int seg = uniform(lo / seg_steps), kstep = lo - seg * seg_steps, next = lo;  // the step that is loaded next
  const int last = p.K - kBK;
  const ValueA* src_a;
  const uint16_t* src_b;
  auto place = [&] {
    src_a = A.at(reinterpret_cast<const ValueA*>(p.A) + ((p.sa >> (2 * seg)) & 3) * p.a_plane, m0, kstep * kBK, p.lda);
    src_b = B.at(p.B + ((p.sb >> (2 * seg)) & 3) * p.b_plane, n0, kstep * kBK, p.ldb);
  };
  place();
  const int64_t step_a = AK ? (int64_t)kBK * p.lda : kBK, step_b = BK ? (int64_t)kBK * p.ldb : kBK;
  auto load = [&](int buf) {
    uint16_t* la = base + buf * T::kStage;
    uint16_t* lb = la + T::kStageA;
    const int k0 = kstep * kBK;
    if (k0 <= last) {
      A.load(src_a, p.lda, la, 64 * wave);
      B.load(src_b, p.ldb, lb, 64 * wave);
    } else if constexpr (T::kRing > 2) {
      A.load_short(src_a, p.lda, p.K - k0, la, 64 * wave);
      B.load_short(src_b, p.ldb, p.K - k0, lb, 64 * wave);
    } else {
      A.load_tail(src_a, p.lda, p.K - k0, la);
      B.load_tail(src_b, p.ldb, p.K - k0, lb);
    }
    if (++next < hi) {  // (past the part's end the last step is loaded again, into a buffer that nobody reads)
      src_a += step_a;
      src_b += step_b;
      if (++kstep == seg_steps) {
        kstep = 0;
        ++seg;
        place();
      }
    }
  };

#pragma unroll
  for (int i = 0; i < kFM; ++i)
#pragma unroll
    for (int j = 0; j < kFN; ++j) acc[i][j] = typename KIND::Acc{};
  bf16x8_t af[2][kFM * kTerms], bf[2][kFN];
  auto read = [&](int buf, int kk, int w) {
    const uint16_t* la = base + buf * T::kStage;
    B.template read<kFN>(la + T::kStageA, (TN / WN) * wn, kk, bf[w]);
    A.template read<kFM * kTerms>(la, (TM / WM) * wm, kk, af[w]);
  };
  auto mma = [&](int w) {
#pragma unroll
    for (int i = 0; i < kFM; ++i)
#pragma unroll
      for (int t = 0; t < kTerms; ++t)
#pragma unroll
        for (int j = 0; j < kFN; ++j)
          acc[i][j] = KIND::mma(bf[w][j], af[w][i * kTerms + t], acc[i][j]);
  };
  constexpr int kReads = kFM * (AK ? 2 : 1) + kFN * (BK ? 2 : 1);
  auto mix = [&] {  // the reads of the next half spread between the products of this one
    constexpr int kPerRead = std::max(1, std::min(2, kFM * kFN / kReads));
#pragma unroll
    for (int x = 0; x < kReads; ++x) {
      __builtin_amdgcn_sched_group_barrier(0x008, kPerRead, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    if constexpr (kFM * kFN > kPerRead * kReads) __builtin_amdgcn_sched_group_barrier(0x008, kFM * kFN - kPerRead * kReads, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  if constexpr (T::kRing > 2) {
    // The time is the latency of the loads, so kRing - 1 steps of them are kept under way.  A step's own have
    // landed once no more are outstanding than the later steps issued.  The last step of a reduction that is no multiple
    // of 64 is no exception: it loads what it can and masks both operands' fragments.
    constexpr int kPer = decltype(A)::kLoads + decltype(B)::kLoads, kLeft = (T::kRing - 2) * kPer;
    static_assert(kLeft < 64, "vmcnt's bits");
    constexpr int kHalves = 2 / T::KG;  // of a step, per wave
    if (lo < hi) {
#pragma unroll
      for (int i = 0; i < T::kRing - 1; ++i) load(i);
      const int rem = p.K % kBK;
      int now = 0, free = T::kRing - 1;
      auto step = [&](auto masked) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0070 | (kLeft & 15) | (kLeft >> 4) << 14);  // vmcnt(kLeft) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        load(free);
#pragma unroll
        for (int w = 0; w < kHalves; ++w) read(now, T::KG == 2 ? kg : w, w);
        if constexpr (decltype(masked)::value) {
#pragma unroll
          for (int w = 0; w < kHalves; ++w) {
            mask_k(af[w], 32 * (T::KG == 2 ? kg : w), rem);
            mask_k(bf[w], 32 * (T::KG == 2 ? kg : w), rem);
          }
        }
#pragma unroll
        for (int w = 0; w < kHalves; ++w) mma(w);
        now = now + 1 == T::kRing ? 0 : now + 1;
        free = free + 1 == T::kRing ? 0 : free + 1;
      };
      int whole = seg_steps - 1 - lo % seg_steps;  // steps before the segment's last
      for (int s = lo; s < hi;) {
        const int until = rem ? min(hi, s + whole) : hi;
        for (; s < until; ++s) step(std::false_type{});
        if (s < hi) {
          step(std::true_type{});
          ++s;
          whole = seg_steps - 1;
        }
      }
    }
  } else if (lo < hi) {
    load(0);
    hand_over();
    load(1);
    read(0, 0, 0);
    int buf = 0;
    for (int s = lo; s < hi; ++s, buf ^= 1) {
      read(buf, 1, 1);
      mma(0);
      mix();
      hand_over();  // the other buffer holds step s + 1; nobody reads this one any more
      load(buf);
      __builtin_amdgcn_sched_barrier(0);
      read(buf ^ 1, 0, 0);
      mma(1);
      mix();
    }
  }
}

}  // namespace
}  // namespace moe
