// Device helpers of the cross entropy's row kernels.
#pragma once

#include <type_traits>

#include "kernels.hpp"
#include "ops_common.hpp"
#include "xent.hpp"

namespace ll {

constexpr float kNegInf = -__builtin_huge_valf();

// (m, s) joined with (m2, s2).  An empty or all -inf piece is (-inf, 0).
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float M = fmaxf(m, m2);
  s = (m == M ? s : s * __expf(m - M)) + (m2 == M ? s2 : s2 * __expf(m2 - M));
  m = M;
}

__device__ __forceinline__ bool has_target(const XentRows& r, int64_t t) { return t >= 0 && t < r.V && t != r.ignore; }

template <int TY>
__device__ __forceinline__ f32x4 mfma16(const Chunk<TY, 8>& a, const Chunk<TY, 8>& b, f32x4 c) {
  if constexpr (TY == LL_F16) {
    f16x8 u, v;
    __builtin_memcpy(&u, &a, 16);
    __builtin_memcpy(&v, &b, 16);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(u, v, c, 0, 0, 0);
  } else {
    bf16x8 u, v;
    __builtin_memcpy(&u, &a, 16);
    __builtin_memcpy(&v, &b, 16);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(u, v, c, 0, 0, 0);
  }
}

// A 16x16x32 operand whose inner index runs over two groups of four rows of an
// LDS image, each read transposed: lane l of 16 gives the address of row l / 4,
// columns 4 (l % 4) .. + 3 of its group and gets column l.
template <int TY>
__device__ __forceinline__ Chunk<TY, 8> frag_pair(const uint16_t LL_LDS* p, const uint16_t LL_LDS* q) {
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((i16x4 LL_LDS*)p);
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((i16x4 LL_LDS*)q);
  const i16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  Chunk<TY, 8> c;
  __builtin_memcpy(&c, &v, 16);
  return c;
}

}  // namespace ll
