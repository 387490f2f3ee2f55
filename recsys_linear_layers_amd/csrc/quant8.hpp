// Quantisation in blocks of 128: the arithmetic of one block, and the arguments
// and launch of the kernel that quantises a matrix (quant8.hip).
#pragma once

#include "ops_common.hpp"

namespace ll {

constexpr int kBlock8 = 128;

template <int Q>
constexpr float kLargest8 = Q == LL_E4M3 ? 448.f : 57344.f;

// A block's scale and its reciprocal, from the largest magnitude as a bit
// pattern: compared as integers NaN > infinity > every finite value, so that
// neither is lost on the way (a maximum of floats drops NaN).  A scale of at
// least 2^-126 keeps its reciprocal finite and makes a block of zeros zeros.
struct Scale8 {
  float scale, inv;
};
// Both are correctly rounded without a division's ten instructions each: a
// quotient by a constant whose reciprocal is rounded, and a reciprocal from the
// hardware's estimate, each corrected once by its remainder (Markstein's theorem;
// for every fp32 amax, and every scale there is, the same bits as the divisions).
template <int Q>
__device__ __forceinline__ Scale8 scale8(uint32_t amax_bits) {
  const float amax = __builtin_bit_cast(float, amax_bits);
  constexpr float F = kLargest8<Q>, R = 1.f / F;
  const float q = amax * R;
  float s = fmaxf(fmaf(fmaf(-q, F, amax), R, q), 0x1p-126f);
  if (amax_bits >= 0x7F800000u) s = __builtin_bit_cast(float, 0x7FC00000u);
  const float y = __builtin_amdgcn_rcpf(s);
  return {s, fmaf(fmaf(-s, y, 1.f), y, y)};
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

// Largest over aligned groups of 16 or 32 lanes; every lane gets it.  Within 16
// the exchange is part of the maximum's own instruction: the neighbour, the other
// pair of four, the other four (mirrored), the other eight (mirrored).
template <int W>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  static_assert(W == 16 || W == 32, "lanes of a block");
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));
  if constexpr (W == 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
  return v;
}

// Four values, already divided by their scale, as four bytes (round to nearest
// even).  Their magnitude is at most F (1 + 2^-22), which rounds to F: nothing
// saturates, and the hardware's overflow rule does not matter.
template <int Q>
__device__ __forceinline__ uint32_t pack8(float a, float b, float c, float d) {
  if constexpr (Q == LL_E4M3)
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
  else
    return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(c, d, __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false), true);
}

// W words of bytes to any address; TAIL: only the first n bytes.  Non-temporal.
template <bool TAIL, int W>
__device__ __forceinline__ void store8(uint8_t* p, const uint32_t (&w)[W], int n) {
  if (!TAIL || n >= 4 * W) {
    typedef uint32_t words __attribute__((ext_vector_type(W)));
    typedef words unaligned_words __attribute__((aligned(1)));
    words v;
    __builtin_memcpy(&v, w, sizeof v);
    if constexpr (W == 1) __builtin_memcpy(p, w, sizeof w);
    else __builtin_nontemporal_store(v, (unaligned_words*)p);
  } else {
#pragma unroll
    for (int i = 0; i < 4 * W; ++i)
      if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

struct Quant8Args {
  const void* x;
  uint8_t* q;      // null: not wanted
  float* scale;
  uint8_t* qt;     // null: not wanted
  float* scale_t;
  int64_t ldx, ldq, ldqt;
  int64_t sn, sb, tn, tb;
  int32_t N, D;
  int32_t aligned;  // rows of x start at multiples of 16 bytes
};

hipError_t launch_quant8(const Quant8Args& a, int type, int q_type, int block, hipStream_t s);

}  // namespace ll
