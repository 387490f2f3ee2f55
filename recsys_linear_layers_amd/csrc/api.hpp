// What the C entry points share: error reporting, the device check, buffer
// spans, and GEMM plans as the other operators build and run them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/linlayers.h"

namespace ll {

// Sets ll_last_error and returns the status.
ll_status fail(ll_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
ll_status ok();
ll_status hip_fail(hipError_t e, const char* what);

struct DeviceInfo {
  bool probed = false;
  bool gfx950 = false;
  int cus = 0;
  char arch[64] = {0};
};

// Current device, its CU count, and whether it is gfx950.
ll_status current_device(int* dev, const DeviceInfo** info);

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Byte extent [lo, hi) of a buffer.
struct Span {
  uintptr_t lo, hi;
};
// Of a 2-D strided view of `rows` x `cols` elements.
inline Span span_of(const void* p, int64_t rows, int64_t cols, int64_t sr, int64_t sc, int64_t esize) {
  const uintptr_t b = (uintptr_t)p;
  if (rows <= 0 || cols <= 0) return {b, b};
  const int64_t last = (rows - 1) * sr + (cols - 1) * sc;
  return {b, b + (uintptr_t)((last + 1) * esize)};
}
inline bool overlaps(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

// One GEMM operand as the kernel sees it.
struct OperandPlan {
  bool kmajor;      // K-contiguous as the kernel reads it (the original layout, or the packed copy's)
  bool pack;        // copied into the workspace (layout below)
  bool pack_mn;     // the packed copy is [K][ldp] (rows contiguous), else [rows][ldp] (K contiguous)
  bool padded;      // not copied, but laid out like a packed copy already (kPadded*)
  int64_t ldp;      // row stride of the packed copy: its row length rounded up to 64 elements, so
                    // that every packed row starts on a 128-byte line
  int64_t ld;       // leading dimension of the direct view
  int64_t s_r, s_k; // original strides (rows = M or N)
  size_t ws_off;    // workspace offset of the packed copy
};

// Operands a caller inside the library has laid out itself: rows along the
// contiguous dimension padded with zeros up to a multiple of 64 elements (the
// leading dimension at least that, a multiple of 8), 16-byte aligned.  Such an
// operand is read in place whatever its logical size.
constexpr uint32_t kPaddedA = 1u, kPaddedB = 2u;
// The hand-ordered kind in whole tiles, K not split: what a softmax epilogue
// needs (LL_ERR_UNSUPPORTED where that kind cannot take the operands).
constexpr uint32_t kWholeTiles = 4u;
// A long K beside a small C: where tiles alone would leave more than half of the
// chip idle, the hand-ordered kind with K split over the idle CUs; where C is
// one or two small tiles, up to 256 splits (otherwise 64) and a reduce to match.
constexpr uint32_t kDeepK = 8u;

}  // namespace ll

struct gemm_plan {
  gemm_desc d;
  int device;
  int cus;
  int kind;
  int layout;
  ll::OperandPlan a, b;
  int64_t Kp;       // K rounded up to a multiple of 8
  int splits;
  int deep;         // kDeepK: many splits of a small C
  int epi;          // fused-epilogue instantiation (0: none, or the split-K reduce applies it)
  int kiters, kps;
  int tiles_m, tiles_n, total, grid, group_m;
  int round_sync;   // hand-ordered kind: round barrier per XCD (counters in the workspace)
  int b_prefetch;   // hand-ordered kind: L2 prefetch of B's slice after the next
  int tail_tiles, tail_splits, tail_kps, tail_first;  // hand-ordered kind: K-split last round
  size_t ws_partial_off;
  size_t ws_sync_off;
  size_t ws_tail_off;
  size_t ws_bytes;
};

namespace ll {

struct GemmKArgs;

// gemm_plan_create into a caller's plan, with the options above.
ll_status gemm_plan_build(const gemm_desc* d, uint32_t options, gemm_plan* out);
// gemm_run on it.  softmax, with a kWholeTiles plan: launches epilogue `epi`
// (SoftmaxEpilogue) with the softmax fields of *softmax; C may be null, and has
// rows and columns up to whole tiles.  epi kScaleEpilogue, with a kWholeTiles plan
// of A^T B in fp16 or a plan with `deep` set: C is multiplied by *bias.
ll_status gemm_run_plan(const gemm_plan* p, const void* A, const void* B, void* C, const float* bias, void* ws,
                        size_t ws_bytes, void* stream, int epi = 0, const GemmKArgs* softmax = nullptr);

}  // namespace ll
