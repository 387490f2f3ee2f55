// The product of 8-bit matrices with a scale per block of 128 along K:
// arguments, the choice of kernel, and launches (gemm8_tile.hpp, gemm8_few.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/linlayers.h"

namespace ll {

// n / d as (n * magic) >> shift, for n < 2^22 and d < 2^26: with 2^s the power of two
// from d on, shift = 22 + s and magic = 2^shift / d + e, 0 < e <= 1, the product
// is too large by n * e < 2^22 <= 2^shift / d, less than what would reach the next quotient.
struct Quotient8 {
  uint32_t magic, shift;
};

inline Quotient8 quotient8(uint32_t d) {
  uint32_t s = 0;
  while ((1u << s) < d) ++s;
  return {(uint32_t)(((uint64_t)1 << (22 + s)) / d + 1), 22 + s};
}

struct Gemm8Args {
  const uint8_t* a;
  const uint8_t* b;
  const float* sa;
  const float* sb;
  void* c;          // c_type, or null where partial is set
  float* partial;   // [splits][M][N], or null
  int64_t lda, ldb, ldc;
  int64_t sam, sab, sbn, sbb;  // strides of the scales: from row to row, from block to block
  int32_t M, N, K;
  int32_t c_type;
  int32_t blocks;   // of 128 along K
  int32_t splits, per_split;  // K is split into runs of per_split blocks
  int32_t tiles_m, tiles_n, total;
  int32_t cus;      // of the device
  Quotient8 by_group, by_last;  // a tile's group (8 rows of tiles), and its column in a last group of fewer rows
};

// By rows and columns of C that a workgroup forms.
enum Gemm8Kind {
  kG8Few16x16, kG8Few16x32, kG8Few32x16, kG8Few32x32, kG8Few64x16, kG8Few64x32,
  kG8Tile64x128, kG8Tile128x128, kG8Tile128x256, kG8Tile256x256,
  kG8Kinds
};

struct Gemm8Plan {
  int kind;  // -1: a forced kernel that cannot take the sizes
  int bm, bn;
  int tiles_m, tiles_n, splits, per_split;
  size_t partial_bytes;  // > 0: the kernel leaves its sums in the workspace, a second one joins and rounds them
};

// Whether blocks' sums have fp32's precision (Block8's EXACT).
inline bool gemm8_exact(const gemm8_desc& d) { return d.c_type == LL_F32 || (d.flags & LL_GEMM8_FULL_SUMS); }

// Sizes and strides alone decide (no device is asked).
Gemm8Plan gemm8_plan(const gemm8_desc& d);
const char* gemm8_kind_name(int kind);
// a_e5m2: A holds LL_E5M2; rows: B's scales are per row (b_block 1); exact: gemm8_exact.
// The tiles' exact kernels store fp32 alone: a 16-bit C goes by the partials.
hipError_t launch_gemm8(const Gemm8Args& a, int kind, bool a_e5m2, bool rows, bool exact, hipStream_t s);

hipError_t launch_gemm8_tile64x128(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s);
hipError_t launch_gemm8_tile64x128_exact(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s);
hipError_t launch_gemm8_tile128x128(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s);
hipError_t launch_gemm8_tile128x128_exact(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s);
hipError_t launch_gemm8_tile128x256(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s);
hipError_t launch_gemm8_tile128x256_exact(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s);
hipError_t launch_gemm8_tile256x256(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s);
hipError_t launch_gemm8_tile256x256_exact(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s);
hipError_t launch_gemm8_few(const Gemm8Args& a, int kind, bool a_e5m2, bool rows, bool exact, hipStream_t s);

}  // namespace ll
