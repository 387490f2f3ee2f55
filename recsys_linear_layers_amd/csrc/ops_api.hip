// C ABI of the embedding and layer norm operators: argument checks, workspace
// layout and launches.  The declarations and their contracts are in
// include/linlayers.h.
#include <math.h>

#include <algorithm>

#include "api.hpp"
#include "embed.hpp"
#include "layernorm.hpp"
#include "ops_common.hpp"

using namespace ll;

namespace {

constexpr int64_t kMaxSize = (1ll << 31) - 1;
// Tokens and columns of the embedding: the kernels round their 32-bit indexes up
// to whole workgroups, chunks and steps, by less than this room.
constexpr int64_t kEmbedMaxSize = (1ll << 31) - (1ll << 12);

bool known_type(int ty) { return ty == LL_BF16 || ty == LL_F16 || ty == LL_F32; }

bool misaligned(const void* p, int64_t size) { return ((uintptr_t)p & (size - 1)) != 0; }

// A buffer's span is formed in 64 bits: rows * stride elements must stay well inside.
bool extent_fits(int64_t rows, int64_t stride) { return rows == 0 || stride <= (1ll << 58) / rows; }

Span span_1d(const void* p, int64_t n, int64_t esize) { return span_of(p, n > 0 ? 1 : 0, n, 0, 1, esize); }

ll_status check_workspace(const void* ws, size_t have, size_t need) {
  if (have < need || (need > 0 && !ws))
    return fail(LL_ERR_WORKSPACE, "workspace %zu bytes, the call needs %zu", have, need);
  if (need > 0 && ((uintptr_t)ws & 255)) return fail(LL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return LL_OK;
}

// ---------------------------------------------------------------------------
// Embedding
// ---------------------------------------------------------------------------

ll_status embed_sizes(int64_t V, int64_t T, int64_t D, int64_t s0, int64_t s1, int type, float scale) {
  if (V < 0 || T < 0 || D < 0) return fail(LL_ERR_INVALID_ARG, "negative size");
  if (!known_type(type)) return fail(LL_ERR_UNSUPPORTED, "type must be LL_BF16, LL_F16 or LL_F32");
  if (V >= kMaxSize || T > kEmbedMaxSize || D > kEmbedMaxSize)
    return fail(LL_ERR_UNSUPPORTED, "V must be below 2^31 - 1, T and D at most 2^31 - 2^12");
  if (s0 < D || s1 < D) return fail(LL_ERR_INVALID_ARG, "row strides shorter than the rows");
  if (!extent_fits(std::max(V, T), std::max(s0, s1))) return fail(LL_ERR_UNSUPPORTED, "row strides too large");
  if (!isfinite(scale)) return fail(LL_ERR_INVALID_ARG, "scale must be finite");
  return LL_OK;
}

struct EmbedGradLayout {
  bool direct = true;
  int bits = 0, passes = 0;
  size_t key[2] = {0, 0}, pos[2] = {0, 0}, hist = 0, total = 0, partial = 0, long_count = 0,
         long_rows = 0, bytes = 0;
};

// Few tokens that are added to a table take the direct path whatever its size:
// every row looks through the ids, 300 into 1000003 x 64 fp32 15 us.
// Workspace of the sorted path.  One workgroup sorts in 8-bit digits; beyond
// that, digits of at most kSortMaxBits bits, of equal width over the passes
// that cover the keys 0 .. V.
EmbedGradLayout embed_grad_layout(const embed_grad_desc* d) {
  EmbedGradLayout l;
  l.direct = d->T == 0 || d->V == 0 || d->D == 0 ||
             (d->T <= kEmbedDirect && ((d->flags & LL_EMBED_ACCUMULATE) ||
                                       d->V * d->D * (int64_t)dtype_size(d->type) <= kEmbedDirectBytes));
  if (l.direct) return l;
  const bool small = d->T <= kEmbedSmall;
  int kb = 1;
  while (kb < 31 && (1ll << kb) <= d->V) ++kb;  // V itself is a key
  const int most = small ? 8 : kSortMaxBits;
  l.passes = (kb + most - 1) / most;
  l.bits = small ? 8 : (kb + l.passes - 1) / l.passes;
  const int64_t nblk = (d->T + kSortItems - 1) / kSortItems;
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off = align256(off + n);
    return at;
  };
  for (int i = 0; i < (small ? 1 : 2); ++i) {
    l.key[i] = take((size_t)d->T * 4);
    l.pos[i] = take((size_t)d->T * 4);
  }
  if (!small) {
    l.hist = take(((size_t)nblk << l.bits) * 4);
    l.total = take((size_t)4 << l.bits);
  }
  l.partial = take((size_t)(d->T / kEmbedChunk) * (size_t)d->D * 4);
  l.long_count = take(4);
  l.long_rows = take((size_t)(d->T / kEmbedChunk) * 8);
  l.bytes = off;
  return l;
}

ll_status embed_grad_check(const embed_grad_desc* d) {
  if (!d) return fail(LL_ERR_INVALID_ARG, "null desc");
  const ll_status s = embed_sizes(d->V, d->T, d->D, d->stride_dout, d->stride_dtable, d->type, d->scale);
  if (s != LL_OK) return s;
  if (d->padding_id < -1) return fail(LL_ERR_INVALID_ARG, "padding_id must be -1 (none) or an id");
  if (d->flags & ~(uint32_t)LL_EMBED_ACCUMULATE) return fail(LL_ERR_INVALID_ARG, "unknown flag bits");
  return LL_OK;
}

}  // namespace

extern "C" {

ll_status embed_run(const embed_desc* d, const void* table, const int64_t* ids, void* out, void* stream) {
  if (!d) return fail(LL_ERR_INVALID_ARG, "null desc");
  ll_status s = embed_sizes(d->V, d->T, d->D, d->stride_table, d->stride_out, d->type, d->scale);
  if (s != LL_OK) return s;
  if (d->T == 0 || d->D == 0) return ok();
  if (!ids || !out || (d->V > 0 && !table)) return fail(LL_ERR_INVALID_ARG, "null pointer");
  const int64_t e = dtype_size(d->type);
  if (misaligned(table, e) || misaligned(out, e) || misaligned(ids, 8))
    return fail(LL_ERR_INVALID_ARG, "misaligned pointer");
  const Span so = span_of(out, d->T, d->D, d->stride_out, 1, e);
  if (overlaps(so, span_of(table, d->V, d->D, d->stride_table, 1, e)) || overlaps(so, span_1d(ids, d->T, 8)))
    return fail(LL_ERR_INVALID_ARG, "out overlaps the table or the ids");
  int dev = 0;
  const DeviceInfo* info = nullptr;
  s = current_device(&dev, &info);
  if (s != LL_OK) return s;
  const EmbedArgs a = {table, ids, out, d->V, d->stride_table, d->stride_out, (int32_t)d->T, (int32_t)d->D, d->scale};
  const hipError_t err = launch_embed(a, d->type, (hipStream_t)stream);
  return err == hipSuccess ? ok() : hip_fail(err, "embed launch");
}

ll_status embed_grad_workspace_size(const embed_grad_desc* d, size_t* bytes) {
  const ll_status s = embed_grad_check(d);
  if (s != LL_OK) return s;
  if (!bytes) return fail(LL_ERR_INVALID_ARG, "null bytes");
  *bytes = embed_grad_layout(d).bytes;
  return ok();
}

ll_status embed_grad_run(const embed_grad_desc* d, const int64_t* ids, const void* dout, void* dtable, void* ws,
                         size_t ws_bytes, void* stream) {
  ll_status s = embed_grad_check(d);
  if (s != LL_OK) return s;
  if (d->V == 0 || d->D == 0) return ok();
  if (!dtable || (d->T > 0 && (!ids || !dout))) return fail(LL_ERR_INVALID_ARG, "null pointer");
  const int64_t e = dtype_size(d->type);
  if (misaligned(dout, e) || misaligned(dtable, e) || misaligned(ids, 8))
    return fail(LL_ERR_INVALID_ARG, "misaligned pointer");
  const EmbedGradLayout l = embed_grad_layout(d);
  s = check_workspace(ws, ws_bytes, l.bytes);
  if (s != LL_OK) return s;
  const Span so = span_of(dtable, d->V, d->D, d->stride_dtable, 1, e);
  if (overlaps(so, span_of(dout, d->T, d->D, d->stride_dout, 1, e)) || overlaps(so, span_1d(ids, d->T, 8)) ||
      overlaps(so, span_1d(ws, (int64_t)l.bytes, 1)))
    return fail(LL_ERR_INVALID_ARG, "dtable overlaps dout, the ids or the workspace");
  int dev = 0;
  const DeviceInfo* info = nullptr;
  s = current_device(&dev, &info);
  if (s != LL_OK) return s;
  EmbedGradArgs a = {};
  a.ids = ids;
  a.dout = dout;
  a.dw = dtable;
  a.V = d->V;
  a.ldg = d->stride_dout;
  a.ldw = d->stride_dtable;
  a.padding = d->padding_id;
  a.T = (int32_t)d->T;
  a.D = (int32_t)d->D;
  a.accumulate = (d->flags & LL_EMBED_ACCUMULATE) != 0;
  a.scale = d->scale;
  a.direct = l.direct;
  a.bits = l.bits;
  a.passes = l.passes;
  if (l.bytes > 0) {
    char* w = (char*)ws;
    for (int i = 0; i < 2; ++i) {
      a.key[i] = (uint32_t*)(w + l.key[i]);
      a.pos[i] = (uint32_t*)(w + l.pos[i]);
    }
    a.hist = (uint32_t*)(w + l.hist);
    a.total = (uint32_t*)(w + l.total);
    a.partial = (float*)(w + l.partial);
    a.long_count = (uint32_t*)(w + l.long_count);
    a.long_rows = (int2*)(w + l.long_rows);
  }
  const hipError_t err = launch_embed_grad(a, d->type, info->cus, (hipStream_t)stream);
  return err == hipSuccess ? ok() : hip_fail(err, "embed gradient launch");
}

// ---------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------

static ll_status norm_sizes(int64_t N, int64_t D, int type, int param_type) {
  if (N < 0 || D < 0) return fail(LL_ERR_INVALID_ARG, "negative size");
  if (!known_type(type)) return fail(LL_ERR_UNSUPPORTED, "type must be LL_BF16, LL_F16 or LL_F32");
  if (param_type != type && param_type != LL_F32)
    return fail(LL_ERR_UNSUPPORTED, "param_type must be the type of x or LL_F32");
  if (D >= kMaxSize / 2) return fail(LL_ERR_UNSUPPORTED, "D must be below 2^30");
  if (N >= (1ll << 40)) return fail(LL_ERR_UNSUPPORTED, "N must be below 2^40");
  return LL_OK;
}

static ll_status norm_stride(int64_t N, int64_t D, int64_t stride) {
  if (stride < D) return fail(LL_ERR_INVALID_ARG, "row strides shorter than the rows");
  if (!extent_fits(N, stride)) return fail(LL_ERR_UNSUPPORTED, "row strides too large");
  return LL_OK;
}

ll_status layernorm_run(const layernorm_desc* d, const void* x, const void* gamma, const void* beta, void* y,
                        float* mean, float* rstd, void* stream) {
  if (!d) return fail(LL_ERR_INVALID_ARG, "null desc");
  ll_status s = norm_sizes(d->N, d->D, d->type, d->param_type);
  if (s == LL_OK) s = norm_stride(d->N, d->D, d->stride_x);
  if (s == LL_OK) s = norm_stride(d->N, d->D, d->stride_y);
  if (s != LL_OK) return s;
  if (!isfinite(d->eps) || d->eps < 0.f) return fail(LL_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (d->N == 0 || d->D == 0) return ok();
  if (!x || !y) return fail(LL_ERR_INVALID_ARG, "null pointer");
  const int64_t e = dtype_size(d->type), pe = dtype_size(d->param_type);
  if (misaligned(x, e) || misaligned(y, e) || misaligned(gamma, pe) || misaligned(beta, pe) || misaligned(mean, 4) ||
      misaligned(rstd, 4))
    return fail(LL_ERR_INVALID_ARG, "misaligned pointer");
  const Span sx = span_of(x, d->N, d->D, d->stride_x, 1, e), sg = span_1d(gamma, gamma ? d->D : 0, pe),
             sb = span_1d(beta, beta ? d->D : 0, pe);
  const Span out[3] = {span_of(y, d->N, d->D, d->stride_y, 1, e), span_1d(mean, mean ? d->N : 0, 4),
                       span_1d(rstd, rstd ? d->N : 0, 4)};
  for (int i = 0; i < 3; ++i) {
    const bool in_place = i == 0 && x == y && d->stride_x == d->stride_y;
    if ((!in_place && overlaps(out[i], sx)) || overlaps(out[i], sg) || overlaps(out[i], sb))
      return fail(LL_ERR_INVALID_ARG, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return fail(LL_ERR_INVALID_ARG, "outputs overlap");
  }
  int dev = 0;
  const DeviceInfo* info = nullptr;
  s = current_device(&dev, &info);
  if (s != LL_OK) return s;
  const NormArgs a = {x, gamma, beta, y, mean, rstd, d->N, d->stride_x, d->stride_y, (int32_t)d->D,
                      d->param_type == LL_F32, d->eps};
  const hipError_t err = launch_norm(a, d->type, info->cus, (hipStream_t)stream);
  return err == hipSuccess ? ok() : hip_fail(err, "layernorm launch");
}

static size_t norm_grad_bytes(const layernorm_grad_desc* d) {
  return align256((size_t)norm_grad_blocks(d->N) * 2 * (size_t)d->D * 4);
}

static ll_status norm_grad_check(const layernorm_grad_desc* d) {
  if (!d) return fail(LL_ERR_INVALID_ARG, "null desc");
  ll_status s = norm_sizes(d->N, d->D, d->type, d->param_type);
  if (s == LL_OK) s = norm_stride(d->N, d->D, d->stride_x);
  if (s == LL_OK) s = norm_stride(d->N, d->D, d->stride_dy);
  if (s == LL_OK) s = norm_stride(d->N, d->D, d->stride_dx);
  return s;
}

ll_status layernorm_grad_workspace_size(const layernorm_grad_desc* d, size_t* bytes) {
  const ll_status s = norm_grad_check(d);
  if (s != LL_OK) return s;
  if (!bytes) return fail(LL_ERR_INVALID_ARG, "null bytes");
  *bytes = norm_grad_bytes(d);
  return ok();
}

ll_status layernorm_grad_run(const layernorm_grad_desc* d, const void* dy, const void* x, const void* gamma,
                             const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta, void* ws,
                             size_t ws_bytes, void* stream) {
  ll_status s = norm_grad_check(d);
  if (s != LL_OK) return s;
  if (!dgamma != !dbeta) return fail(LL_ERR_INVALID_ARG, "dgamma and dbeta: both or neither");
  if (d->D == 0 || (d->N == 0 && !dgamma)) return ok();
  if (d->N > 0 && (!dy || !x || !mean || !rstd || !dx)) return fail(LL_ERR_INVALID_ARG, "null pointer");
  const int64_t e = dtype_size(d->type), pe = dtype_size(d->param_type);
  if (misaligned(x, e) || misaligned(dy, e) || misaligned(dx, e) || misaligned(gamma, pe) || misaligned(dgamma, pe) ||
      misaligned(dbeta, pe) || misaligned(mean, 4) || misaligned(rstd, 4))
    return fail(LL_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = dgamma ? norm_grad_bytes(d) : 0;
  s = check_workspace(ws, ws_bytes, need);
  if (s != LL_OK) return s;
  const Span in[6] = {span_of(dy, d->N, d->D, d->stride_dy, 1, e), span_of(x, d->N, d->D, d->stride_x, 1, e),
                      span_1d(gamma, gamma ? d->D : 0, pe),        span_1d(mean, d->N, 4),
                      span_1d(rstd, d->N, 4),                      span_1d(ws, (int64_t)need, 1)};
  const Span out[3] = {span_of(dx, d->N, d->D, d->stride_dx, 1, e), span_1d(dgamma, dgamma ? d->D : 0, pe),
                       span_1d(dbeta, dbeta ? d->D : 0, pe)};
  for (int i = 0; i < 3; ++i) {
    for (const Span& t : in)
      if (overlaps(out[i], t)) return fail(LL_ERR_INVALID_ARG, "an output overlaps an input or the workspace");
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return fail(LL_ERR_INVALID_ARG, "outputs overlap");
  }
  int dev = 0;
  const DeviceInfo* info = nullptr;
  s = current_device(&dev, &info);
  if (s != LL_OK) return s;
  const NormGradArgs a = {dy, x, gamma, mean, rstd, dx, dgamma, dbeta, dgamma ? (float*)ws : nullptr, d->N,
                          d->stride_dy, d->stride_x, d->stride_dx, (int32_t)d->D, d->param_type == LL_F32};
  const hipError_t err = launch_norm_grad(a, d->type, info->cus, (hipStream_t)stream);
  return err == hipSuccess ? ok() : hip_fail(err, "layernorm gradient launch");
}

}  // extern "C"
