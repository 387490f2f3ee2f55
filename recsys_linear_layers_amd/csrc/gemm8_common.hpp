// What the kernels of the 8-bit product share: the matrix instruction, loads
// into LDS, and stores of C.
#pragma once

#include "gemm8.hpp"
#include "quant8.hpp"

namespace ll {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 frag8(i32x4 lo, i32x4 hi) {
  return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// A block's sums: D[i][j] = sum over 128 k of W[i][k] X[j][k], from fragments of
// which lane l holds row l % 16 and 32 of the 128 k (any, as long as both
// operands take the same); lane l gets D[4 (l / 16) + r][l % 16].  W is LL_E4M3,
// X LL_E5M2 if E5M2.
//
// The 8-bit matrix instructions align the eight products of a group to the
// largest and drop what lies below 2^-13 of its power of two (measured: beside
// 448 * 448 a product of 8 is kept, one of 4 lost): up to 7 * 2^-13 of the
// group's largest product.  Of the result's norm, without C's rounding (512 x 512 x
// 4096): 1.4e-5 on normally distributed operands, 2.8e-5 where 0.4% of A's columns
// stand out by 20, 5.5e-5 where 1% do by 100, 7.3e-5 by 1000, 2.1e-5 with lognormal
// entries (sigma 2).  A 16-bit C is rounded to 2^-8 or 2^-11 of itself (1.6e-3 and
// 2e-4 of the norm) and takes them, unless the caller asks for full sums.  Those, and
// a C in fp32, are EXACT: the operands are widened to bf16, which holds every 8-bit
// value, and multiplied at half the rate, where the same sums are off by 8e-8.
template <bool E5M2, bool EXACT>
struct Block8;

template <bool E5M2>
struct Block8<E5M2, false> {
  typedef i32x8 W;
  typedef i32x8 X;
  static __device__ __forceinline__ W w(i32x8 v) { return v; }
  static __device__ __forceinline__ X x(i32x8 v) { return v; }
  // with no scale operands the instruction's own (per-32) scales are 1
  static __device__ __forceinline__ f32x4 product(const W& w, const X& x) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{0.f, 0.f, 0.f, 0.f}, 0, E5M2 ? 1 : 0, 0, 0, 0,
                                                            0);
  }
};

template <bool E5M2>
struct Block8<E5M2, true> {
  struct Wide {
    bf16x8 v[4];
  };
  typedef Wide W;
  typedef Wide X;
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  template <bool B5>
  static __device__ __forceinline__ bf16x2 pair(int word, bool high) {
    if constexpr (B5)
      return high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)word, 1.f, true)
                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)word, 1.f, false);
    else
      return high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)word, 1.f, true)
                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)word, 1.f, false);
  }
  template <bool B5>
  static __device__ __forceinline__ Wide widen(i32x8 v) {
    Wide o;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bf16x2 lo = pair<B5>(v[i], false), hi = pair<B5>(v[i], true);
      o.v[i >> 1][4 * (i & 1)] = lo[0];
      o.v[i >> 1][4 * (i & 1) + 1] = lo[1];
      o.v[i >> 1][4 * (i & 1) + 2] = hi[0];
      o.v[i >> 1][4 * (i & 1) + 3] = hi[1];
    }
    return o;
  }
  static __device__ __forceinline__ W w(i32x8 v) { return widen<false>(v); }
  static __device__ __forceinline__ X x(i32x8 v) { return widen<E5M2>(v); }
  static __device__ __forceinline__ f32x4 product(const W& w, const X& x) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 4; ++h) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[h], x.v[h], d, 0, 0, 0);
    return d;
  }
};

// Chunk c of A's row r sits at c ^ swz8_a(r), of B's at c ^ swz8_b(r).  A row's
// 128 bytes are half of the banks (which half goes by the row's parity), and a
// pass of a 16-byte LDS read serves 16 lanes, the 16 rows of a fragment at one
// chunk: the eight rows of each parity need eight different values.  A's rows
// follow one another; B's are four times four, 4 FN rows apart.
__device__ __forceinline__ int swz8_a(int r) { return ((r >> 1) & 1) | (((r >> 3) & 1) << 1) | (r & 4); }
template <int GF>
__device__ __forceinline__ int swz8_b(int r) {
  return ((r >> 1) & 1) | (((r / (8 * GF)) & 1) << 1) | (((r / (4 * GF)) & 1) << 2);
}

// dma16 for one word per lane: lane l's 4 bytes land at LDS byte address m0 + 4 l.
__device__ __forceinline__ void dma4(i32x4 rsrc, uint32_t lds_addr, uint32_t voff) {
  asm volatile("s_nop 4\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(rsrc), "{m0}"(lds_addr)
               : "memory");
}

// The first `left` (all, if as many) of CNT values to consecutive places, in
// 16-byte stores at whatever alignment; fewer go one by one.
template <int TYPE, int CNT, typename E>
__device__ __forceinline__ void store_piece8(E* dst, const float (&v)[CNT], int left) {
  if constexpr (TYPE == LL_F32) {
    if (left >= CNT) {
#pragma unroll
      for (int i = 0; i < CNT; i += 4) {
        const f32x4 q = {v[i], v[i + 1], v[i + 2], v[i + 3]};
        __builtin_memcpy(dst + i, &q, sizeof q);
      }
    } else {
#pragma unroll
      for (int i = 0; i < CNT; ++i)
        if (i < left) dst[i] = v[i];
    }
  } else {
    constexpr int VEC = CNT < 8 ? CNT : 8;
#pragma unroll
    for (int k = 0; k < CNT; k += VEC) {
      Chunk<TYPE, VEC> c;
#pragma unroll
      for (int i = 0; i < VEC; i += 2) c.put2(i, v[k + i], v[k + i + 1]);
      c.template store<true>(dst + k, left - k);
    }
  }
}

// CNT consecutive columns of row m of C from column n on, or of the partials.
template <int CNT>
__device__ __forceinline__ void store_c8(const Gemm8Args& p, int split, int m, int n, const float (&v)[CNT]) {
  if (m >= p.M || n >= p.N) return;
  const int left = p.N - n;
  const int64_t at = (int64_t)m * p.ldc + n;
  if (p.partial)
    store_piece8<LL_F32, CNT>(p.partial + ((int64_t)split * p.M + m) * p.N + n, v, left);
  else if (p.c_type == LL_F32)
    store_piece8<LL_F32, CNT>((float*)p.c + at, v, left);
  else if (p.c_type == LL_BF16)
    store_piece8<LL_BF16, CNT>((uint16_t*)p.c + at, v, left);
  else
    store_piece8<LL_F16, CNT>((uint16_t*)p.c + at, v, left);
}

}  // namespace ll
