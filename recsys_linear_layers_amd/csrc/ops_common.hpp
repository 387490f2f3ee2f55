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
// alignment (a 16-byte access at any element is one instruction here).  Held
// as whole words: as an array of 16-bit elements each would take a register
// of its own once it lives across a loop step.
template <int TY, int VEC>
struct Chunk {
  typedef typename Elem<TY>::raw raw;
  static constexpr int PER = 4 / (int)sizeof(raw);  // elements per word
  static_assert(VEC % PER == 0, "whole words");
  uint32_t w[VEC / PER];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (TY == LL_F32) return Elem<TY>::get(w[i]);
    else if constexpr (TY == LL_BF16)
      return __builtin_bit_cast(float, i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    else return Elem<TY>::get((raw)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]));
  }
  __device__ __forceinline__ void put_raw(int i, raw v) {
    if constexpr (PER == 1) w[i] = v;
    else w[i >> 1] = i & 1 ? (w[i >> 1] & 0xFFFFu) | (uint32_t)v << 16 : (w[i >> 1] & 0xFFFF0000u) | v;
  }
  __device__ __forceinline__ raw get_raw(int i) const {
    if constexpr (PER == 1) return w[i];
    else return (raw)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]);
  }
  __device__ __forceinline__ void put(int i, float v) { put_raw(i, Elem<TY>::put(v)); }
  // Elements i and i + 1, i even, 16-bit types: one conversion and no merging of halves.
  __device__ __forceinline__ void put2(int i, float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    if constexpr (TY == LL_BF16) {
      typedef __bf16 h2 __attribute__((ext_vector_type(2)));
      w[i >> 1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, h2));
    } else {
      typedef _Float16 h2 __attribute__((ext_vector_type(2)));
      w[i >> 1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, h2));
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < VEC / PER; ++i) w[i] = 0;
  }
  // Forgets what the compiler has derived from the stored elements: their fp32
  // values are formed again where they are used next, instead of being held
  // in twice the registers until then.
  __device__ __forceinline__ void keep_packed() {
    if constexpr (PER > 1) {
#pragma unroll
      for (int i = 0; i < VEC / PER; ++i) asm volatile("" : "+v"(w[i]));
    }
  }
  // The n elements of a row from p on, as many as there are (the others 0).
  // TAIL false: all VEC are there.
  template <bool TAIL>
  __device__ __forceinline__ void load(const raw* p, int n) {
    if (!TAIL || n >= VEC) {
      __builtin_memcpy(this, p, sizeof(*this));
    } else {
      clear();
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < n) put_raw(i, p[i]);
    }
  }
  // NT: not read again soon (non-temporal).
  template <bool TAIL, bool NT = false>
  __device__ __forceinline__ void store(raw* p, int n) const {
    if (!TAIL || n >= VEC) {
      if constexpr (NT) {
        typedef uint32_t words __attribute__((ext_vector_type(VEC / PER)));
        typedef words unaligned_words __attribute__((aligned(sizeof(raw))));
        words v;
        __builtin_memcpy(&v, this, sizeof v);
        __builtin_nontemporal_store(v, (unaligned_words*)p);
      } else {
        __builtin_memcpy(p, this, sizeof(*this));
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < n) p[i] = get_raw(i);
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
