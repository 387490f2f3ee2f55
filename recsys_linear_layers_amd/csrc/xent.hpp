// Row kernels of the vocabulary cross entropy: arguments and launches (xent.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ll {

// Maximum and sum of exp(z - maximum) over some of a row's logits.
struct XentPart {
  float m, s;
};

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
  float* lse;              // [N]
  float* coef;             // [N] upstream gradient times scale[0]; 0 without a target
  float* scale;            // fp16: {S, 1/S}; null otherwise
  XentPart* parts;         // [N][np]
  int32_t np;
  // outputs
  float* loss;
  float* lse_out;          // null: not wanted
};

hipError_t launch_xent_prep(const XentRows& r, int type, hipStream_t s);
// Power of two S that brings the largest |dloss| near 2^14 (fp16 gradients of the logits).
hipError_t launch_xent_scale(const XentRows& r, hipStream_t s);
// parts[row][p0 + split] of fp32 logits z [N][ldz], cols wide, in `splits` pieces per row.
hipError_t launch_xent_stats(const XentRows& r, const float* z, int64_t ldz, int cols, int p0, int splits,
                             hipStream_t s);
hipError_t launch_xent_lse(const XentRows& r, hipStream_t s);
// dz[row][c] = (exp(z - lse) - (v0 + c == target)) * coef for c < cols, 0 up to ldd.
hipError_t launch_xent_dz(const XentRows& r, const float* z, int64_t ldz, int64_t v0, int cols, void* dz,
                          int64_t ldd, int type, int cus, hipStream_t s);
// out[i][j] = (a[i][j] + b[i][j]) * (*scale) as `type`; b and scale may be null.
hipError_t launch_xent_finish(const float* a, const float* b, const float* scale, int64_t rows, int64_t cols,
                              int64_t lda, void* out, int64_t ldo, int type, int cus, hipStream_t s);

}  // namespace ll
