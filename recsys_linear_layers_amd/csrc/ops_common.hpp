// Element types and small device helpers shared by the memory-bound operators
// (embedding, layer norm) and the cross entropy's row kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/linlayers.h"
#include "gemm_kernel.hpp"

namespace ll {

// One element type (an ll_dtype code) as stored; every computation is in fp32.
template <int TY>
struct Elem;
template <>
struct Elem<LL_BF16> {
  typedef uint16_t raw;
  static __device__ __forceinline__ float get(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }
  static __device__ __forceinline__ uint16_t put(float v) { return f32_to_bf16_bits(v); }
};
template <>
struct Elem<LL_F16> {
  typedef uint16_t raw;
  static __device__ __forceinline__ float get(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }
  static __device__ __forceinline__ uint16_t put(float v) { return f32_to_f16_bits(v); }
};
template <>
struct Elem<LL_F32> {
  typedef uint32_t raw;
  static __device__ __forceinline__ float get(uint32_t b) { return __builtin_bit_cast(float, b); }
  static __device__ __forceinline__ uint32_t put(float v) { return __builtin_bit_cast(uint32_t, v); }
};

// VEC consecutive elements, moved by one load or store whatever their
// alignment (a 16-byte access at any element is one instruction here).
template <int TY, int VEC>
struct Chunk {
  typedef typename Elem<TY>::raw raw;
  raw e[VEC];
  __device__ __forceinline__ float get(int i) const { return Elem<TY>::get(e[i]); }
  __device__ __forceinline__ void put(int i, float v) { e[i] = Elem<TY>::put(v); }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = 0;
  }
  // The n elements of a row from p on, as many as there are (the others 0).
  // TAIL false: all VEC are there.
  template <bool TAIL>
  __device__ __forceinline__ void load(const raw* p, int n) {
    if (!TAIL || n >= VEC) {
      __builtin_memcpy(this, p, sizeof(*this));
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = i < n ? p[i] : (raw)0;
    }
  }
  template <bool TAIL>
  __device__ __forceinline__ void store(raw* p, int n) const {
    if (!TAIL || n >= VEC) {
      __builtin_memcpy(p, this, sizeof(*this));
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < n) p[i] = e[i];
    }
  }
};

// Elements of a 16-byte access.
template <int TY>
constexpr int kWide = 16 / (int)sizeof(typename Elem<TY>::raw);

inline int dtype_size(int ty) { return ty == LL_F32 ? 4 : 2; }

// Sum over aligned groups of W lanes (a power of two up to 64); every lane gets it.
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int m = 1; m < W; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}

}  // namespace ll
