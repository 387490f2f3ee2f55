// C ABI of the 8-bit linear layers (root-mean-square norm, quantisation, scaled
// product): argument checks, workspace layout, choice of kernels and launches.
// The declarations and their contracts are in include/linlayers.h.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>

#include "api.hpp"
#include "gemm8.hpp"
#include "kernels.hpp"
#include "ops_common.hpp"
#include "quant8.hpp"
#include "rmsnorm.hpp"

using namespace ll;

namespace {

bool known_type(int ty) { return ty == LL_BF16 || ty == LL_F16 || ty == LL_F32; }
bool known_type8(int ty) { return ty == LL_E4M3 || ty == LL_E5M2; }

bool misaligned(const void* p, int64_t size) { return ((uintptr_t)p & (size - 1)) != 0; }

// A buffer's span is formed in 64 bits: rows * stride elements must stay well inside.
bool extent_fits(int64_t rows, int64_t stride) { return rows == 0 || stride <= (1ll << 58) / rows; }

int64_t blocks8(int64_t n) { return (n + kBlock8 - 1) / kBlock8; }

Span span_1d(const void* p, int64_t n, int64_t esize) { return span_of(p, n > 0 ? 1 : 0, n, 0, 1, esize); }

ll_status check_workspace(const void* ws, size_t have, size_t need) {
  if (have < need || (need > 0 && !ws))
    return fail(LL_ERR_WORKSPACE, "workspace %zu bytes, the call needs %zu", have, need);
  if (need > 0 && ((uintptr_t)ws & 255)) return fail(LL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return LL_OK;
}

// Workgroups of a launch: of 512 threads, fewer than 2^32 in all.
constexpr int64_t kG8MostTiles = 1 << 22;

ll_status check_stride(int64_t rows, int64_t cols, int64_t stride) {
  if (stride < cols) return fail(LL_ERR_INVALID_ARG, "row strides shorter than the rows");
  if (!extent_fits(rows, stride)) return fail(LL_ERR_UNSUPPORTED, "row strides too large");
  return LL_OK;
}

// Scales [rows][cols] with the strides sr, sc.
ll_status check_scale(int64_t rows, int64_t cols, int64_t sr, int64_t sc) {
  if (sr < 1 || sc < 1) return fail(LL_ERR_INVALID_ARG, "scale strides must be positive");
  if (!extent_fits(rows, sr) || !extent_fits(cols, sc)) return fail(LL_ERR_UNSUPPORTED, "scale strides too large");
  return LL_OK;
}

ll_status norm_sizes(int64_t N, int64_t D, int type, int param_type) {
  if (N < 0 || D < 0) return fail(LL_ERR_INVALID_ARG, "negative size");
  if (!known_type(type)) return fail(LL_ERR_UNSUPPORTED, "type must be LL_BF16, LL_F16 or LL_F32");
  if (param_type != type && param_type != LL_F32)
    return fail(LL_ERR_UNSUPPORTED, "param_type must be the type of x or LL_F32");
  if (D >= (1ll << 30) - 1) return fail(LL_ERR_UNSUPPORTED, "D must be below 2^30 - 1");
  if (N >= (1ll << 40)) return fail(LL_ERR_UNSUPPORTED, "N must be below 2^40");
  return LL_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// Root-mean-square norm
// ---------------------------------------------------------------------------

ll_status rmsnorm_run(const rmsnorm_desc* d, const void* x, const void* residual, const void* gamma, void* h, void* y,
                      float* scale, float* rstd, void* stream) {
  if (!d) return fail(LL_ERR_INVALID_ARG, "null desc");
  ll_status s = norm_sizes(d->N, d->D, d->type, d->param_type);
  if (s != LL_OK) return s;
  const bool eight = known_type8(d->y_type);
  if (!eight && d->y_type != d->type) return fail(LL_ERR_UNSUPPORTED, "y_type must be type, LL_E4M3 or LL_E5M2");
  s = check_stride(d->N, d->D, d->stride_x);
  if (s == LL_OK) s = check_stride(d->N, d->D, d->stride_y);
  if (s == LL_OK && residual) s = check_stride(d->N, d->D, d->stride_residual);
  if (s == LL_OK && residual) s = check_stride(d->N, d->D, d->stride_h);
  if (s == LL_OK && eight) s = check_scale(d->N, blocks8(d->D), d->stride_sn, d->stride_sb);
  if (s != LL_OK) return s;
  if (!isfinite(d->eps) || d->eps < 0.f) return fail(LL_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (d->N == 0 || d->D == 0) return ok();
  if (!x || !y || (eight && !scale)) return fail(LL_ERR_INVALID_ARG, "null pointer");
  if (!residual != !h) return fail(LL_ERR_INVALID_ARG, "h is written if and only if there is a residual");
  const int64_t e = dtype_size(d->type), pe = dtype_size(d->param_type), ye = eight ? 1 : e;
  if (misaligned(x, e) || misaligned(residual, e) || misaligned(h, e) || misaligned(y, ye) || misaligned(gamma, pe) ||
      misaligned(scale, 4) || misaligned(rstd, 4))
    return fail(LL_ERR_INVALID_ARG, "misaligned pointer");
  const int64_t hn = residual ? d->N : 0;
  const Span sx = span_of(x, d->N, d->D, d->stride_x, 1, e), sr = span_of(residual, hn, d->D, d->stride_residual, 1, e),
             sg = span_1d(gamma, gamma ? d->D : 0, pe);
  const Span out[4] = {span_of(y, d->N, d->D, d->stride_y, 1, ye), span_of(h, hn, d->D, d->stride_h, 1, e),
                       span_of(scale, eight ? d->N : 0, blocks8(d->D), d->stride_sn, d->stride_sb, 4),
                       span_1d(rstd, rstd ? d->N : 0, 4)};
  const bool y_is_x = !eight && !residual && x == y && d->stride_x == d->stride_y;
  const bool h_is_x = h == x && d->stride_h == d->stride_x, h_is_r = h == residual && d->stride_h == d->stride_residual;
  for (int i = 0; i < 4; ++i) {
    if ((overlaps(out[i], sx) && !(i == 0 && y_is_x) && !(i == 1 && h_is_x)) ||
        (overlaps(out[i], sr) && !(i == 1 && h_is_r)) || overlaps(out[i], sg))
      return fail(LL_ERR_INVALID_ARG, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return fail(LL_ERR_INVALID_ARG, "outputs overlap");
  }
  int dev = 0;
  const DeviceInfo* info = nullptr;
  s = current_device(&dev, &info);
  if (s != LL_OK) return s;
  const RmsArgs a = {x,           residual,           gamma,       h,           y,
                     scale,       rstd,               d->N,        d->stride_x, d->stride_residual,
                     d->stride_h, d->stride_y,        d->stride_sn, d->stride_sb, (int32_t)d->D,
                     d->param_type == LL_F32, d->eps};
  const hipError_t err = launch_rmsnorm(a, d->type, eight ? d->y_type : d->type, info->cus, (hipStream_t)stream);
  return err == hipSuccess ? ok() : hip_fail(err, "rmsnorm launch");
}

static size_t rms_grad_bytes(const rmsnorm_grad_desc* d) {
  return align256((size_t)rms_grad_blocks(d->N) * (size_t)d->D * 4);
}

static ll_status rms_grad_check(const rmsnorm_grad_desc* d) {
  if (!d) return fail(LL_ERR_INVALID_ARG, "null desc");
  ll_status s = norm_sizes(d->N, d->D, d->type, d->param_type);
  if (s == LL_OK) s = check_stride(d->N, d->D, d->stride_dy);
  if (s == LL_OK) s = check_stride(d->N, d->D, d->stride_h);
  if (s == LL_OK) s = check_stride(d->N, d->D, d->stride_dx);
  return s;
}

ll_status rmsnorm_grad_workspace_size(const rmsnorm_grad_desc* d, size_t* bytes) {
  const ll_status s = rms_grad_check(d);
  if (s != LL_OK) return s;
  if (!bytes) return fail(LL_ERR_INVALID_ARG, "null bytes");
  *bytes = rms_grad_bytes(d);
  return ok();
}

ll_status rmsnorm_grad_run(const rmsnorm_grad_desc* d, const void* dy, const void* h, const void* gamma,
                           const float* rstd, const void* dh, void* dx, void* dgamma, void* ws, size_t ws_bytes,
                           void* stream) {
  ll_status s = rms_grad_check(d);
  if (s == LL_OK && dh) s = check_stride(d->N, d->D, d->stride_dh);
  if (s != LL_OK) return s;
  if (d->D == 0 || (d->N == 0 && !dgamma)) return ok();
  if (d->N > 0 && (!dy || !h || !rstd || !dx)) return fail(LL_ERR_INVALID_ARG, "null pointer");
  const int64_t e = dtype_size(d->type), pe = dtype_size(d->param_type);
  if (misaligned(dy, e) || misaligned(h, e) || misaligned(dh, e) || misaligned(dx, e) || misaligned(gamma, pe) ||
      misaligned(dgamma, pe) || misaligned(rstd, 4))
    return fail(LL_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = dgamma ? rms_grad_bytes(d) : 0;
  s = check_workspace(ws, ws_bytes, need);
  if (s != LL_OK) return s;
  const Span se = span_of(dh, dh ? d->N : 0, d->D, d->stride_dh, 1, e);
  const Span in[6] = {span_of(dy, d->N, d->D, d->stride_dy, 1, e), span_of(h, d->N, d->D, d->stride_h, 1, e),
                      span_1d(gamma, gamma ? d->D : 0, pe),        span_1d(rstd, d->N, 4),
                      span_1d(ws, (int64_t)need, 1),               se};
  const Span out[2] = {span_of(dx, d->N, d->D, d->stride_dx, 1, e), span_1d(dgamma, dgamma ? d->D : 0, pe)};
  const bool in_place = dx == dh && d->stride_dx == d->stride_dh;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 6; ++j)
      if (overlaps(out[i], in[j]) && !(i == 0 && j == 5 && in_place))
        return fail(LL_ERR_INVALID_ARG, "an output overlaps an input or the workspace");
  if (overlaps(out[0], out[1])) return fail(LL_ERR_INVALID_ARG, "outputs overlap");
  int dev = 0;
  const DeviceInfo* info = nullptr;
  s = current_device(&dev, &info);
  if (s != LL_OK) return s;
  const RmsGradArgs a = {dy,          h,           gamma,        rstd,         dh,           dx,
                         dgamma,      dgamma ? (float*)ws : nullptr, d->N, d->stride_dy, d->stride_h, d->stride_dh,
                         d->stride_dx, (int32_t)d->D, d->param_type == LL_F32};
  const hipError_t err = launch_rmsnorm_grad(a, d->type, info->cus, (hipStream_t)stream);
  return err == hipSuccess ? ok() : hip_fail(err, "rmsnorm gradient launch");
}

// ---------------------------------------------------------------------------
// Quantisation
// ---------------------------------------------------------------------------

ll_status quant8_run(const quant8_desc* d, const void* x, void* q, float* scale, void* qt, float* scale_t,
                     void* stream) {
  if (!d) return fail(LL_ERR_INVALID_ARG, "null desc");
  if (d->N < 0 || d->D < 0) return fail(LL_ERR_INVALID_ARG, "negative size");
  if (!known_type(d->type)) return fail(LL_ERR_UNSUPPORTED, "type must be LL_BF16, LL_F16 or LL_F32");
  if (!known_type8(d->q_type)) return fail(LL_ERR_UNSUPPORTED, "q_type must be LL_E4M3 or LL_E5M2");
  if (d->block != 1 && d->block != kBlock8) return fail(LL_ERR_INVALID_ARG, "block must be 1 or 128");
  if (d->N >= (1ll << 30) || d->D >= (1ll << 30)) return fail(LL_ERR_UNSUPPORTED, "N and D must be below 2^30");
  if (!q != !scale || !qt != !scale_t) return fail(LL_ERR_INVALID_ARG, "a form is its values and its scales");
  ll_status s = check_stride(d->N, d->D, d->stride_x);
  const int64_t sn = d->block == 1 ? d->N : blocks8(d->N), tn = d->block == 1 ? d->D : blocks8(d->D);
  if (s == LL_OK && q) s = check_stride(d->N, d->D, d->stride_q);
  if (s == LL_OK && q) s = check_scale(sn, blocks8(d->D), d->stride_sn, d->stride_sb);
  if (s == LL_OK && qt) s = check_stride(d->D, d->N, d->stride_qt);
  if (s == LL_OK && qt) s = check_scale(tn, blocks8(d->N), d->stride_tn, d->stride_tb);
  if (s != LL_OK) return s;
  if (d->N == 0 || d->D == 0) return ok();
  if (!x || (!q && !qt)) return fail(LL_ERR_INVALID_ARG, "null pointer");
  const int64_t e = dtype_size(d->type);
  if (misaligned(x, e) || misaligned(scale, 4) || misaligned(scale_t, 4))
    return fail(LL_ERR_INVALID_ARG, "misaligned pointer");
  const Span sx = span_of(x, d->N, d->D, d->stride_x, 1, e);
  const Span out[4] = {span_of(q, q ? d->N : 0, d->D, d->stride_q, 1, 1),
                       span_of(scale, q ? sn : 0, blocks8(d->D), d->stride_sn, d->stride_sb, 4),
                       span_of(qt, qt ? d->D : 0, d->N, d->stride_qt, 1, 1),
                       span_of(scale_t, qt ? tn : 0, blocks8(d->N), d->stride_tn, d->stride_tb, 4)};
  for (int i = 0; i < 4; ++i) {
    if (overlaps(out[i], sx)) return fail(LL_ERR_INVALID_ARG, "an output overlaps x");
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return fail(LL_ERR_INVALID_ARG, "outputs overlap");
  }
  int dev = 0;
  const DeviceInfo* info = nullptr;
  s = current_device(&dev, &info);
  if (s != LL_OK) return s;
  const Quant8Args a = {x,           (uint8_t*)q,  scale,        (uint8_t*)qt, scale_t,      d->stride_x,
                        d->stride_q, d->stride_qt, d->stride_sn, d->stride_sb, d->stride_tn, d->stride_tb,
                        (int32_t)d->N, (int32_t)d->D,  !misaligned(x, 16) && d->stride_x * e % 16 == 0};
  const hipError_t err = launch_quant8(a, d->type, d->q_type, d->block, (hipStream_t)stream);
  return err == hipSuccess ? ok() : hip_fail(err, "quant8 launch");
}

// ---------------------------------------------------------------------------
// Scaled product
// ---------------------------------------------------------------------------

static ll_status gemm8_check(const gemm8_desc* d) {
  if (!d) return fail(LL_ERR_INVALID_ARG, "null desc");
  if (d->M < 0 || d->N < 0 || d->K < 0) return fail(LL_ERR_INVALID_ARG, "negative size");
  if (!known_type8(d->a_type) || d->b_type != LL_E4M3 || !known_type(d->c_type))
    return fail(LL_ERR_UNSUPPORTED, "A must be LL_E4M3 or LL_E5M2, B LL_E4M3, C LL_BF16, LL_F16 or LL_F32");
  if (d->b_block != 1 && d->b_block != kBlock8) return fail(LL_ERR_INVALID_ARG, "b_block must be 1 or 128");
  if (d->flags & ~LL_GEMM8_FULL_SUMS) return fail(LL_ERR_INVALID_ARG, "unknown flags 0x%x", d->flags);
  if (d->M >= (1ll << 26) || d->N >= (1ll << 26) || d->K >= (1ll << 22))
    return fail(LL_ERR_UNSUPPORTED, "M and N must be below 2^26, K below 2^22");
  // a launch of 2^32 threads or more is not supported
  if (((d->M + 255) / 256) * ((d->N + 255) / 256) > kG8MostTiles) return fail(LL_ERR_UNSUPPORTED, "C is too large");
  if (d->stride_a < d->K || d->stride_b < d->K || d->stride_c < d->N)
    return fail(LL_ERR_INVALID_ARG, "row strides shorter than the rows");
  if (d->stride_a % 16 || d->stride_b % 16)
    return fail(LL_ERR_INVALID_ARG, "rows of A and B must start at multiples of 16 bytes");
  if (d->stride_a >= (1ll << 22) || d->stride_b >= (1ll << 22) || !extent_fits(d->M, d->stride_c))
    return fail(LL_ERR_UNSUPPORTED, "row strides too large");
  const int64_t bn = d->b_block == 1 ? d->N : blocks8(d->N);
  ll_status s = check_scale(d->M, blocks8(d->K), d->stride_am, d->stride_ab);
  if (s == LL_OK) s = check_scale(bn, blocks8(d->K), d->stride_bn, d->stride_bb);
  if (s == LL_OK && (d->stride_am >= (1ll << 20) || (d->b_block == 1 && d->stride_bn >= (1ll << 20))))
    return fail(LL_ERR_UNSUPPORTED, "scale strides along the rows must be below 2^20");
  return s;
}

ll_status gemm8_workspace_size(const gemm8_desc* d, size_t* bytes) {
  const ll_status s = gemm8_check(d);
  if (s != LL_OK) return s;
  if (!bytes) return fail(LL_ERR_INVALID_ARG, "null bytes");
  *bytes = d->M == 0 || d->N == 0 ? 0 : gemm8_plan(*d).partial_bytes;
  return ok();
}

ll_status gemm8_describe(const gemm8_desc* d, char* buf, size_t len) {
  const ll_status s = gemm8_check(d);
  if (s != LL_OK) return s;
  if (!buf || len == 0) return fail(LL_ERR_INVALID_ARG, "null buffer");
  const Gemm8Plan p = gemm8_plan(*d);
  snprintf(buf, len, "kernel=%s tile=%dx%d tiles=%dx%d splits=%d blocks=%d ws=%zu", gemm8_kind_name(p.kind), p.bm,
           p.bn, p.tiles_m, p.tiles_n, p.splits, p.per_split, p.partial_bytes);
  return ok();
}

ll_status gemm8_run(const gemm8_desc* d, const void* A, const float* a_scale, const void* B, const float* b_scale,
                    void* C, void* ws, size_t ws_bytes, void* stream) {
  ll_status s = gemm8_check(d);
  if (s != LL_OK) return s;
  if (d->M == 0 || d->N == 0) return ok();
  if (!C || (d->K > 0 && (!A || !B || !a_scale || !b_scale))) return fail(LL_ERR_INVALID_ARG, "null pointer");
  const int64_t e = dtype_size(d->c_type);
  if (misaligned(A, 16) || misaligned(B, 16) || misaligned(a_scale, 4) || misaligned(b_scale, 4) || misaligned(C, e))
    return fail(LL_ERR_INVALID_ARG, "misaligned pointer (A and B: 16 bytes)");
  const Gemm8Plan plan = gemm8_plan(*d);
  if (plan.kind < 0) return fail(LL_ERR_UNSUPPORTED, "the forced kernel cannot take these sizes");
  s = check_workspace(ws, ws_bytes, plan.partial_bytes);
  if (s != LL_OK) return s;
  const int64_t kb = blocks8(d->K), bn = d->b_block == 1 ? d->N : blocks8(d->N);
  const Span sc = span_of(C, d->M, d->N, d->stride_c, 1, e);
  if (overlaps(sc, span_of(A, d->M, d->K, d->stride_a, 1, 1)) ||
      overlaps(sc, span_of(B, d->N, d->K, d->stride_b, 1, 1)) ||
      overlaps(sc, span_of(a_scale, d->M, kb, d->stride_am, d->stride_ab, 4)) ||
      overlaps(sc, span_of(b_scale, bn, kb, d->stride_bn, d->stride_bb, 4)) ||
      overlaps(sc, span_1d(ws, (int64_t)plan.partial_bytes, 1)))
    return fail(LL_ERR_INVALID_ARG, "C overlaps an input or the workspace");
  int dev = 0;
  const DeviceInfo* info = nullptr;
  s = current_device(&dev, &info);
  if (s != LL_OK) return s;
  Gemm8Args a = {};
  a.a = (const uint8_t*)A;
  a.b = (const uint8_t*)B;
  a.sa = a_scale;
  a.sb = b_scale;
  a.c = C;
  a.partial = plan.partial_bytes ? (float*)ws : nullptr;
  a.lda = d->stride_a;
  a.ldb = d->stride_b;
  a.ldc = d->stride_c;
  a.sam = d->stride_am;
  a.sab = d->stride_ab;
  a.sbn = d->stride_bn;
  a.sbb = d->stride_bb;
  a.M = (int32_t)d->M;
  a.N = (int32_t)d->N;
  a.K = (int32_t)d->K;
  a.c_type = d->c_type;
  a.blocks = (int32_t)kb;
  a.splits = plan.splits;
  a.per_split = plan.per_split;
  a.tiles_m = plan.tiles_m;
  a.tiles_n = plan.tiles_n;
  a.total = plan.tiles_m * plan.tiles_n * plan.splits;
  a.cus = info->cus;
  hipError_t err =
      launch_gemm8(a, plan.kind, d->a_type == LL_E5M2, d->b_block == 1, gemm8_exact(*d), (hipStream_t)stream);
  if (err == hipSuccess && a.partial)
    err = launch_splitk_reduce(a.partial, plan.splits, d->M, d->N, C, d->stride_c, 1,
                               d->c_type == LL_F32 ? 0 : d->c_type == LL_BF16 ? 1 : 2, nullptr, 0, (hipStream_t)stream);
  return err == hipSuccess ? ok() : hip_fail(err, "gemm8 launch");
}

}  // extern "C"

namespace ll {

namespace {

// step: microseconds of a step (128 of K) where all CUs hold a workgroup (tiles).
const struct {
  const char* name;
  int bm, bn;
  float step;
} kKinds[kG8Kinds] = {
    {"FEW16x16", 16, 16, 0.f},          {"FEW16x32", 16, 32, 0.f},          {"FEW32x16", 32, 16, 0.f},
    {"FEW32x32", 32, 32, 0.f},          {"FEW64x16", 64, 16, 0.f},          {"FEW64x32", 64, 32, 0.f},
    {"TILE64x128", 64, 128, 0.47f},     {"TILE128x128", 128, 128, 0.61f},   {"TILE128x256", 128, 256, 0.95f},
    {"TILE256x256", 256, 256, 1.60f}};

constexpr int kCus = 256;  // that the choice is made for

// Whether the sums go by the partials: a split K, and tiles that leave a 16-bit C in fp32.
bool gemm8_joins(const gemm8_desc& d, int kind, int64_t splits) {
  return splits > 1 || (kind >= kG8Tile64x128 && d.c_type != LL_F32 && gemm8_exact(d));
}

// What a kernel takes, in microseconds, as far as the choice needs it: 96 drawn
// problems, of 1 to 16384 rows, took 2 to 3% longer on average than with the best
// kernel and split of each.
//   Tiles: 4.2 before the first step and after the last store; a round of tiles over
//   the CUs takes its steps, each at least as long as its rows of A and B come
//   from memory (5 TB/s), and its stores (5.5); a split K adds a launch and the
//   partials' bytes, written and read.  Estimate and measured time (MI355X, bf16 C) of
//   kernels that are taken: 1024 x 4096 x 4096, 128x128 26 / 25; 2048 x 4096 x 4096,
//   128x256 39 / 36; 4096^3, 256x256 62.5 / 59; 128 x 8192 x 8192, 64x128 in two splits
//   28 / 25.5; 64 x 28672 x 8192, 64x128 53 / 54; 9690 x 1600 x 192 to fp32, 128x128 30 / 25;
//   of others: 4096^3, 128x256 73 / 71, 128x128 92 / 91; 64 x 8192 x 8192, 64x128 in four
//   splits 26 / 19.5; 29 x 19904 x 512, 64x128 7.7 / 7.0.
//   Few rows: each CU's share of B comes at 10 bytes a clock, or 11 for many small
//   workgroups (HBM; up to 25 where not all CUs ask), the rows of A, again for each
//   workgroup, at 60 (L2; 25 where rows are not whole lines), B's scales by rows take
//   some more, and kernels of more than 128 registers leave no room for a second
//   workgroup on a CU.  Taken: 1 x 8192 x 8192, 16x16 14 / 12.5; 16 x 8192 x 8192, 16x16 16 /
//   11.7; 32 x 8192 x 8192, 32x32 17 / 12.2; 64 x 8192 x 8192, 64x32 20 / 15.3; 1 x 28672 x
//   8192, 16x16 42.5 / 39; 64 x 4096 x 4096, 64x16 8.2 / 7.4; 37 x 5003 x 4099, 64x32 10.2 /
//   9.5; 29 x 19904 x 512, 32x32 4.8 / 5.2; 30 x 1624 x 10045 by rows, 32x32 in four splits
//   10.8 / 9.9.  Others: 1 x 8192 x 8192, 16x32 15 / 12.4; 16 x 8192 x 8192, 16x32 16 / 11.5; 1 x
//   28672 x 8192, 16x32 46 / 44.
float gemm8_time(const gemm8_desc& d, int kind, int64_t tiles, int64_t splits, int64_t steps) {
  const float rounds = (float)((tiles * splits + kCus - 1) / kCus);
  const float mn = (float)d.M * (float)d.N;
  const bool joins = gemm8_joins(d, kind, splits);
  const float join = joins ? 3.f + (float)splits * mn * 4.f / 3.0e6f : 0.f;
  if (kind >= kG8Tile64x128) {
    // sums of fp32's precision are formed at about half the rate
    const float work = kKinds[kind].step * (gemm8_exact(d) ? 1.9f : 1.f);
    const float memory = (float)(d.M + d.N) * 128.f * (float)splits / rounds / 5.0e6f;
    const float bytes = (float)(kKinds[kind].bm * kKinds[kind].bn * (joins ? 4 : dtype_size(d.c_type)));
    const float stores = (float)std::min<int64_t>(tiles * splits, kCus) * bytes / 5.5e6f;
    return 4.2f + rounds * (1.f + (float)steps * std::max(work, memory) + stores) + join;
  }
  const bool by_rows = d.b_block == 1;
  const float of_b = std::min(25.f, (kKinds[kind].bn == 16 ? 11.f : 10.f) * kCus / (float)std::min<int64_t>(tiles * splits, kCus));
  const float of_a = d.stride_a % 128 == 0 && d.stride_b % 128 == 0 ? 60.f : 25.f;
  const float rows = (float)std::min<int64_t>(d.M, kKinds[kind].bm);
  const float one = (float)steps * 128.f * ((float)kKinds[kind].bn / of_b + rows / of_a + (by_rows ? 0.3f : 0.f)) / 2100.f;
  const bool alone = kKinds[kind].bm == 64 || (by_rows && kKinds[kind].bn == 32);  // no room for a second on a CU
  const float turns = std::max(1.f, alone ? rounds : (float)(tiles * splits) / kCus);
  return 2.f + 0.02f * (float)kKinds[kind].bm + turns * std::max(alone ? 1.5f : 0.6f, one) + join;
}

}  // namespace

const char* gemm8_kind_name(int kind) { return kind >= 0 && kind < kG8Kinds ? kKinds[kind].name : "none"; }

// The kernel and the split of K with the smallest estimate.  The environment
// variables LL_GEMM8_KIND (a name as gemm8_describe prints it) and LL_GEMM8_SPLITS
// override the choice, for measurements.
Gemm8Plan gemm8_plan(const gemm8_desc& d) {
  const char* const forced = getenv("LL_GEMM8_KIND");
  const char* const forced_splits = getenv("LL_GEMM8_SPLITS");
  const int64_t blocks = blocks8(d.K);
  Gemm8Plan p = {};
  p.kind = -1;
  float best = 0.f;
  for (int kind = 0; kind < kG8Kinds; ++kind) {
    if (forced && strcmp(forced, kKinds[kind].name)) continue;
    if (kind < kG8Tile64x128 && (d.M > kKinds[kind].bm || (!forced && 2 * d.M <= kKinds[kind].bm && kind >= kG8Few32x16)))
      continue;  // the rows do not fit, or fit half of them
    const int64_t tm = (d.M + kKinds[kind].bm - 1) / kKinds[kind].bm, tn = (d.N + kKinds[kind].bn - 1) / kKinds[kind].bn;
    for (int64_t want = 1; want <= 16; want *= 2) {
      int64_t splits = forced_splits ? std::max(1, atoi(forced_splits)) : want;
      splits = std::max<int64_t>(1, std::min(splits, blocks));
      const int64_t steps = std::max<int64_t>(1, (blocks + splits - 1) / splits);
      splits = std::max<int64_t>(1, (blocks + steps - 1) / steps);
      if (tm * tn * splits > kG8MostTiles) break;
      const float t = gemm8_time(d, kind, tm * tn, splits, steps);
      if (p.kind >= 0 && t >= best) continue;
      best = t;
      p.kind = kind;
      p.bm = kKinds[kind].bm;
      p.bn = kKinds[kind].bn;
      p.tiles_m = (int)tm;
      p.tiles_n = (int)tn;
      p.per_split = (int)steps;
      p.splits = (int)splits;
      p.partial_bytes = gemm8_joins(d, kind, splits) ? align256((size_t)splits * (size_t)d.M * (size_t)d.N * 4) : 0;
    }
  }
  return p;
}

hipError_t launch_gemm8(const Gemm8Args& a, int kind, bool a_e5m2, bool rows, bool exact, hipStream_t s) {
  switch (kind) {
    case kG8Tile64x128:
      return exact ? launch_gemm8_tile64x128_exact(a, a_e5m2, rows, s) : launch_gemm8_tile64x128(a, a_e5m2, rows, s);
    case kG8Tile128x128:
      return exact ? launch_gemm8_tile128x128_exact(a, a_e5m2, rows, s) : launch_gemm8_tile128x128(a, a_e5m2, rows, s);
    case kG8Tile128x256:
      return exact ? launch_gemm8_tile128x256_exact(a, a_e5m2, rows, s) : launch_gemm8_tile128x256(a, a_e5m2, rows, s);
    case kG8Tile256x256:
      return exact ? launch_gemm8_tile256x256_exact(a, a_e5m2, rows, s) : launch_gemm8_tile256x256(a, a_e5m2, rows, s);
    default: return launch_gemm8_few(a, kind, a_e5m2, rows, exact, s);
  }
}

}  // namespace ll
