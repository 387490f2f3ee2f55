// The hand-ordered 256x256 GEMM kind (gemm_sq4.hpp) as the logits of the
// vocabulary cross entropy: z = x w^T (both operands K-contiguous), of which
// only what the softmax needs leaves the tile.
//
// A wave holds 128 rows by 128 columns of z in its accumulators; 16 lanes
// share a row.  Row block by row block (16 rows): the maximum over the lane's
// eight columns and then over the 16 lanes, the exponentials, and their sum
// the same way.  So every 128 columns of a row give one pair (maximum, sum),
// and in fp32 z exists nowhere else.  With numerators, exp(z - maximum) leaves
// as fp16 through the staged image that a 16-bit C takes, whatever the
// operands' type: 11 bits, an eighth of the rounding that bf16 gradients take.
//
// Cost: one wave per SIMD, so nothing hides the epilogue's ~10 vector
// operations per element: 16384 x 32768 (32 tiles per CU) takes 370 us with D =
// 192, 590 with 512 and 930 with 1024 (statistics alone), so about 1.4 us per 64 of
// the inner dimension and 7 us per tile beside it; with numerators 5 us more.
#include "kernels.hpp"
#include "gemm_sq4.hpp"

namespace ll {

constexpr float kLog2e = 1.442695041f;

// z - base as exp2's argument is fma(z, log2 e, -base * log2 e), one instruction,
// but with the rounding of its addend, half a step of |base| log2 e: at 256 that
// is 2^-16, 1.1e-5 of the exponential.  Further out (an entry of the vocabulary
// masked by a huge negative value, a logit of 1e9) it would grow past 1 and the
// exponential become anything from 0 to infinity, so the difference is formed
// first there, for such rows alone (a row's bits depend on nothing but the row, and
// rows past the last hold anything), by a branch per 16 rows (statistics alone of
// 16384 x 32768 x 192: 368 us with it, 363 without; a branch per row 388).
constexpr float kFarBase = 256.f;

// The value 8, 4, 2 or 1 lanes further in each group of 16 (rotated).
template <int N>
__device__ __forceinline__ float ror16(float v) {
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xF, 0xF, false));
}
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, ror16<8>(v));
  v = fmaxf(v, ror16<4>(v));
  v = fmaxf(v, ror16<2>(v));
  return fmaxf(v, ror16<1>(v));
}
__device__ __forceinline__ float sum16(float v) {
  v += ror16<8>(v);
  v += ror16<4>(v);
  v += ror16<2>(v);
  return v + ror16<1>(v);
}

// Row block I: lane l holds rows 16 I + 4 (l / 16) + r, columns 16 J + l % 16.
template <bool F16, int EPI, int I>
__device__ __forceinline__ void softmax_rows(const GemmKArgs& p, const TileInfo& ti, int wm0, int wn0, int lane,
                                             int cols, char LL_LDS* img) {
  f32x4 v[8] = {sq4_acc<8 * I + 0>(), sq4_acc<8 * I + 1>(), sq4_acc<8 * I + 2>(), sq4_acc<8 * I + 3>(),
                sq4_acc<8 * I + 4>(), sq4_acc<8 * I + 5>(), sq4_acc<8 * I + 6>(), sq4_acc<8 * I + 7>()};
  const int c = lane & 15, row = 16 * I + 4 * (lane >> 4);
  if constexpr (EPI == kSoftmaxGradient) {
    const int64_t r0 = ti.m0 + wm0 + row;  // a multiple of 4: the arrays are read 16 bytes at a time
    const f32x4 lse = *(const f32x4*)(p.lse + r0), coef = *(const f32x4*)(p.coef + r0);
    const i32x4 col = *(const i32x4*)(p.column + r0);
    f32x4 base = lse;
    const float top = fmaxf(fmaxf(fabsf(lse[0]), fabsf(lse[1])), fmaxf(fabsf(lse[2]), fabsf(lse[3])));
    if (__any(top > kFarBase)) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool far = fabsf(lse[r]) > kFarBase;
#pragma unroll
        for (int J = 0; J < 8; ++J) v[J][r] -= far ? lse[r] : 0.f;
        base[r] = far ? 0.f : lse[r];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float l2 = base[r] * kLog2e;
      const int at = col[r] - p.col0 - ti.n0 - wn0 - c;  // 16 J where this lane holds the target
#pragma unroll
      for (int J = 0; J < 8; ++J) {
        float e = __builtin_amdgcn_exp2f(fmaf(v[J][r], kLog2e, -l2)) - (at == 16 * J ? 1.f : 0.f);
        e = col[r] >= 0 && 16 * J + c < cols ? e * coef[r] : 0.f;
        *(uint16_t LL_LDS*)(img + sq4_stage_off(row + r, 32 * J + 2 * c)) = to_c16<F16 ? 2 : 1>(e);
      }
    }
  } else {
    if (cols < 128) {  // the vocabulary ends in this block (uniform)
#pragma unroll
      for (int J = 0; J < 8; ++J)
        if (16 * J + c >= cols)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[J][r] = -__builtin_huge_valf();
    }
    float m[4], m2[4], s[4], top = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = max16(fmaxf(fmaxf(fmaxf(v[0][r], v[1][r]), fmaxf(v[2][r], v[3][r])),
                         fmaxf(fmaxf(v[4][r], v[5][r]), fmaxf(v[6][r], v[7][r]))));
      // all -inf: exp2(-inf) = 0 for every column
      m2[r] = m[r] == -__builtin_huge_valf() ? 0.f : m[r];
      top = fmaxf(top, fabsf(m2[r]));
    }
    if (__any(top > kFarBase)) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool far = fabsf(m2[r]) > kFarBase;
#pragma unroll
        for (int J = 0; J < 8; ++J) v[J][r] -= far ? m2[r] : 0.f;
        m2[r] = far ? 0.f : m2[r];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m2[r] *= kLog2e;
      float sum = 0.f;
#pragma unroll
      for (int J = 0; J < 8; ++J) {
        const float e = __builtin_amdgcn_exp2f(fmaf(v[J][r], kLog2e, -m2[r]));
        sum += e;
        if constexpr (EPI == kSoftmaxNumerators)
          *(uint16_t LL_LDS*)(img + sq4_stage_off(row + r, 32 * J + 2 * c)) =
              to_c16<2>(e * kNumeratorScale);
      }
      s[r] = sum16(sum);
    }
    // lanes c < 4 of each 16 store row `row + c`: 16 rows side by side
    const float ms = c == 0 ? m[0] : c == 1 ? m[1] : c == 2 ? m[2] : m[3];
    const float ss = c == 0 ? s[0] : c == 1 ? s[1] : c == 2 ? s[2] : s[3];
    if (c < 4)
      p.parts[(int64_t)(p.part0 + (ti.n0 + wn0) / 128) * p.part_ld + ti.m0 + wm0 + row + c] = float2{ms, ss};
  }
}

template <bool F16, int EPI>
__device__ void sq4_softmax(const GemmKArgs& p, const TileInfo& ti, int wm0, int wn0, int lane, char LL_LDS* img) {
  const int cols = p.N - ti.n0 - wn0;  // of the vocabulary from this block's first column on
  softmax_rows<F16, EPI, 0>(p, ti, wm0, wn0, lane, cols, img);
  softmax_rows<F16, EPI, 1>(p, ti, wm0, wn0, lane, cols, img);
  softmax_rows<F16, EPI, 2>(p, ti, wm0, wn0, lane, cols, img);
  softmax_rows<F16, EPI, 3>(p, ti, wm0, wn0, lane, cols, img);
  softmax_rows<F16, EPI, 4>(p, ti, wm0, wn0, lane, cols, img);
  softmax_rows<F16, EPI, 5>(p, ti, wm0, wn0, lane, cols, img);
  softmax_rows<F16, EPI, 6>(p, ti, wm0, wn0, lane, cols, img);
  softmax_rows<F16, EPI, 7>(p, ti, wm0, wn0, lane, cols, img);
  if constexpr (EPI != kSoftmaxStats) sq4_flush(p, ti, wm0, wn0, lane, img);
}

hipError_t launch_gemm_sq4_xent(int f16, int epi, const GemmKArgs& a, int grid, hipStream_t s) {
#define LL_XENT_CASE(F, E)                                                                                     \
  if (!!f16 == F && epi == E) {                                                                                \
    hipLaunchKernelGGL((gemm_sq4<F, E, true, false>), dim3(grid), dim3(Sq4::THREADS), 0, s, a);               \
    return hipGetLastError();                                                                                  \
  }
  LL_XENT_CASE(false, kSoftmaxStats)
  LL_XENT_CASE(false, kSoftmaxNumerators)
  LL_XENT_CASE(false, kSoftmaxGradient)
  LL_XENT_CASE(true, kSoftmaxStats)
  LL_XENT_CASE(true, kSoftmaxNumerators)
  LL_XENT_CASE(true, kSoftmaxGradient)
#undef LL_XENT_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_gemm_sq4_am_scaled_f16(const GemmKArgs& a, int grid, hipStream_t s) {
  hipLaunchKernelGGL((gemm_sq4<true, kScaleEpilogue, false, true>), dim3(grid), dim3(Sq4::THREADS), 0, s, a);
  return hipGetLastError();
}

}  // namespace ll
