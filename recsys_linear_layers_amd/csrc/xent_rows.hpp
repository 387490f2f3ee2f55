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

// scale = {S, 1 / S} by one workgroup of THREADS; red: THREADS / 64 floats.
template <int THREADS>
__device__ __forceinline__ void scale_block(const XentRows& r, float* red) {
  float m = 0.f;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < r.N; i += THREADS) {
    const float g = fabsf(r.dloss[i]);
    if (has_target(r, r.target[i]) && g < __builtin_huge_valf()) m = fmaxf(m, g);
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < THREADS / 64; ++w) m = fmaxf(m, red[w]);
    // largest |dloss| in [2^13, 2^14); the inverse stays a normal number
    int e = 0;
    if (m > 0.f) frexpf(m, &e);
    e = max(-100, min(100, 14 - e));
    r.scale[0] = ldexpf(1.f, e);
    r.scale[1] = ldexpf(1.f, -e);
  }
}

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
