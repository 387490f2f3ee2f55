// Row kernels of the vocabulary cross entropy: arguments and launches (xent.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ll {

struct XentRows {
  const void* x;           // [N][ldx]
  const void* w;           // [V][ldw], for the target's logit
  const int64_t* target;
  const float* dloss;      // null without gradients
  int64_t N, V, ldx, ldw, ignore;
  int32_t D, ldp;
  // workspace
  void* xp;                // [N][ldp] copy of x: zeros past D and in rows without a target
  float* zt;               // [N] the target's logit
  float* lse;              // [N], as coef and column up to whole tiles of rows
  float* coef;             // [N] upstream gradient times scale[0]; 0 without a target
  int32_t* column;         // [N] the target, -1 for none
  float* scale;            // fp16: {S, 1/S}; null otherwise
  // Per part of a row's logits: maximum m and sum s of exp(z - m), [np][part_ld];
  // parts from factor0 on then hold in place of m what turns their numerators
  // exp(z - m) * kNumeratorScale into gradients.
  float2* parts;
  int64_t part_ld;
  int32_t np, factor0;
  // outputs
  float* loss;
  float* lse_out;          // null: not wanted
};

// dst[i][0 .. ldp) = src[i][0 .. cols), zeros past cols; ldp a multiple of 64.
hipError_t launch_xent_pack(const void* src, int64_t lds, int64_t rows, int cols, void* dst, int ldp, int cus,
                            hipStream_t s);
// scaled: also forms scale, as launch_xent_scale does (likewise below).
hipError_t launch_xent_prep(const XentRows& r, bool scaled, int type, hipStream_t s);
// Power of two S that brings the largest |dloss| near 2^14 (fp16 gradients of the logits).
hipError_t launch_xent_scale(const XentRows& r, hipStream_t s);
// Few rows: up to kXentFewRows, x of at most kXentFewBytes (rows padded by 16
// bytes).  Loss side in one pass over w: parts[workgroup][row], zt, and z if
// not null.  x and w as given, any alignment; r.np workgroups.
constexpr int kXentFewRows = 64;
constexpr int64_t kXentFewBytes = 144 * 1024;
hipError_t launch_xent_few(const XentRows& r, bool scaled, float* z, int64_t ldz, int type, hipStream_t s);
// dw [V][ldo] of out_type from dz [N][ldd] and the copy xp, times *scale (null: 1).
hipError_t launch_xent_dw_few(const XentRows& r, const void* dz, int64_t ldd, void* dw, int64_t ldo, int out_type,
                              const float* scale, int type, int cus, hipStream_t s);
// dx as partial[share][N][D] sums over shares of the vocabulary, from dz [N][ldd]
// (zeros past V) and w as given.
int xent_dx_few_shares(int64_t N, int64_t V, int D, int cus);
hipError_t launch_xent_dx_few(const XentRows& r, const void* dz, int64_t ldd, float* partial, int type, int cus,
                              hipStream_t s);
// Narrow rows: D up to kXentNarrow (r.ldp 64 or 128), x and w as given, any
// alignment.  parts[share][row] in r.np shares, and zt; then dx and dw, without
// stored logits.
constexpr int kXentNarrow = 128;
enum { kNarrowStats = 0, kNarrowDx = 1, kNarrowDw = 2 };
struct XentNarrowOut {
  void* out;
  int64_t ldo;
  int type, shares;        // shares 0: not wanted
  float* partial;          // [shares][rows][ldp] where there is more than one share
  const float* scale;      // null: 1
  int64_t rows;            // set by the launch
  int row_blocks;
};
int xent_narrow_shares(int64_t own, int64_t streamed, int64_t slots);
hipError_t launch_xent_narrow_stats(const XentRows& r, bool scaled, int type, hipStream_t s);
hipError_t launch_xent_narrow_grad(const XentRows& r, XentNarrowOut dx, XentNarrowOut dw, int type, hipStream_t s);
// parts[p0 + split][row] of fp32 logits z [N][ldz], cols wide, in `splits` pieces per row.
hipError_t launch_xent_stats(const XentRows& r, const float* z, int64_t ldz, int cols, int p0, int splits,
                             hipStream_t s);
hipError_t launch_xent_lse(const XentRows& r, hipStream_t s);
// dz[row][c] = (exp(z - lse) - (v0 + c == target)) * coef for c < cols, 0 up to ldd.
hipError_t launch_xent_dz(const XentRows& r, const float* z, int64_t ldz, int64_t v0, int cols, void* dz,
                          int64_t ldd, int type, int cus, hipStream_t s);
constexpr int kXentRowCols = 32768;
// Everything between the logits of a whole row (fp32, cols wide) and the gradient
// products, one workgroup per row: loss, lse and, with dz, dz [N][ldd] and the
// copy of x in xp (if not null).  No parts, zt, lse or coef needed.
hipError_t launch_xent_rows(const XentRows& r, const float* z, int64_t ldz, int cols, void* dz, int64_t ldd, int type,
                            hipStream_t s);
// In place on the fp16 numerators of one piece, 128 columns per part from part
// p0 on: dz = numerator * factor as `type`, and the target's own from its logit.
hipError_t launch_xent_numerators(const XentRows& r, void* dz, int64_t ldd, int64_t v0, int cols, int p0, int type,
                                  hipStream_t s);
// out[i][j] = (a[i][j] + b[i][j]) * (*scale) as `type`; b and scale may be null.
hipError_t launch_xent_finish(const float* a, const float* b, const float* scale, int64_t rows, int64_t cols,
                              int64_t lda, void* out, int64_t ldo, int type, int cus, hipStream_t s);

}  // namespace ll
