// C ABI of the vocabulary cross entropy: argument checks, the pieces of the
// vocabulary, workspace layout and the sequence of launches.  The declarations
// and their contracts are in include/linlayers.h.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "api.hpp"
#include "kernels.hpp"
#include "ops_common.hpp"
#include "xent.hpp"

using namespace ll;

struct xent_plan {
  xent_desc d;
  int device, cus;
  bool dx, dw;
  int64_t ldp;        // row stride of the copy of x (and of a packed w): D rounded up to 64
  int64_t ldw;        // row stride of w as the products read it
  bool pack_w;
  int64_t cols;       // vocabulary entries per piece (the last may have fewer)
  bool fused;         // the softmax runs in the logits' product; else it reads fp32 logits
  bool few;           // few rows: w is streamed once, with fp32 logits for the gradients
  bool narrow;        // D <= kXentNarrow: logits formed in each step, never stored
  int shares[3];      // narrow: of statistics, dx, dw
  bool any_w;         // w may start at any element (the contract; few rows need no alignment either way)
  bool few_dx, few_dw;// few rows: gradients by kernels of their own, no copy of w
  bool by_row;        // one piece of at most kXentRowCols: one kernel from the logits to dz
  bool x_direct;      // by_row: the logits' product reads x itself (where it is aligned)
  int pieces, kept;   // kept: the last pieces, whose numerators stay for the gradients
  int parts, np;      // per row and piece, and over all pieces
  int64_t rows;       // N, up to whole tiles where fused
  int64_t ldz, ldd;   // row strides of the fp32 logits and of the 16-bit dz of a piece
  bool dx_direct;     // dx leaves its product in its final form
  bool dx_scaled;     // dx's product takes the scale of dz out
  bool dw_scaled;     // dw's product takes the scale of dz out
  gemm_plan logits[2], dxp[2], dwp[2];  // [1]: the last piece
  gemm_plan logits_x; // x_direct
  int dx_shares;
  size_t off_xp, off_wp, off_zt, off_lse, off_coef, off_column, off_scale, off_parts, off_z, off_dz, off_dxa, off_dxb, off_dxp, off_dwt,
      off_gemm, gemm_bytes, ws_bytes;
};

namespace {

// Bytes the logits or numerators and their gradient may take when the
// description does not say: 2 GiB, under 1% of the card's memory.
constexpr int64_t kDefaultPieceBytes = 2ll << 30;
// Rows from which a weight whose rows are not whole 64-element blocks is copied
// first: the copy costs 4 V D bytes of traffic, and lets the products run on
// the hand-ordered kind.
constexpr int64_t kPackRows = 512;

// Vocabulary entries of a piece from which the logits' product prefetches the
// next slice of w into L2, whatever D is (a plain product does from D = 8192
// on).  Loss alone, us, with and without: 4096 x 131072 x 4096 2990 / 3270, x
// 2048 1620 / 1750, x 1024 909 / 974; 300 x 131072 x 2048 204 / 225; 4096 x 32768
// x 4096 760 / 828; below that it costs: 16384 x 16384 x 2048 804 / 778, 4096 x
// 8192 x 4096 203 / 199.
constexpr int64_t kPrefetchCols = 32768;

ll_status xent_check(const xent_desc* d) {
  if (d->N < 0 || d->V < 0 || d->D < 0) return fail(LL_ERR_INVALID_ARG, "negative size");
  if (d->V == 0 || d->D == 0) return fail(LL_ERR_INVALID_ARG, "V and D must be positive");
  if (d->piece_bytes < 0) return fail(LL_ERR_INVALID_ARG, "negative piece_bytes");
  if (d->flags & ~(uint32_t)(LL_XENT_DX | LL_XENT_DW | LL_XENT_PACK_W))
    return fail(LL_ERR_INVALID_ARG, "unknown flag bits");
  if (d->type != LL_BF16 && d->type != LL_F16) return fail(LL_ERR_UNSUPPORTED, "type must be LL_BF16 or LL_F16");
  if ((d->flags & LL_XENT_DX) && d->dx_type != d->type && d->dx_type != LL_F32)
    return fail(LL_ERR_UNSUPPORTED, "dx_type must be the type of x or LL_F32");
  if ((d->flags & LL_XENT_DW) && d->dw_type != d->type && d->dw_type != LL_F32)
    return fail(LL_ERR_UNSUPPORTED, "dw_type must be the type of w or LL_F32");
  if (d->N >= (1ll << 30) || d->V >= (1ll << 30) || d->D >= (1ll << 20))
    return fail(LL_ERR_UNSUPPORTED, "N and V must be below 2^30, D below 2^20");
  if (d->stride_x < d->D || d->stride_w < d->D || ((d->flags & LL_XENT_DX) && d->stride_dx < d->D) ||
      ((d->flags & LL_XENT_DW) && d->stride_dw < d->D))
    return fail(LL_ERR_INVALID_ARG, "row strides shorter than the rows");
  for (int64_t st : {d->stride_x, d->stride_w, (d->flags & LL_XENT_DX) ? d->stride_dx : 0,
                     (d->flags & LL_XENT_DW) ? d->stride_dw : 0})
    if (st >= (1ll << 28)) return fail(LL_ERR_UNSUPPORTED, "row strides must be below 2^28");
  return LL_OK;
}

gemm_desc product(int64_t M, int64_t N, int64_t K, int64_t sam, int64_t sak, int64_t sbk, int64_t sbn, int64_t ldc,
                  int type, int c_type) {
  gemm_desc g;
  memset(&g, 0, sizeof g);
  g.M = M;
  g.N = N;
  g.K = K;
  g.stride_am = sam;
  g.stride_ak = sak;
  g.stride_bk = sbk;
  g.stride_bn = sbn;
  g.stride_cm = ldc;
  g.stride_cn = 1;
  g.a_type = g.b_type = type;
  g.c_type = c_type;
  return g;
}

}  // namespace

extern "C" {

ll_status xent_plan_create(xent_plan** out, const xent_desc* d) {
  if (!out || !d) return fail(LL_ERR_INVALID_ARG, "xent_plan_create: null argument");
  *out = nullptr;
  ll_status s = xent_check(d);
  if (s != LL_OK) return s;
  xent_plan p;
  memset(&p, 0, sizeof p);
  p.d = *d;
  p.dx = d->flags & LL_XENT_DX;
  p.dw = d->flags & LL_XENT_DW;
  const bool grads = p.dx || p.dw;
  p.ldp = round_up(d->D, 64);
  p.pack_w = (d->flags & LL_XENT_PACK_W) || d->stride_w % 8 || d->D % 8 || (d->D % 64 && d->N >= kPackRows);
  p.ldw = p.pack_w ? p.ldp : d->stride_w;
  const bool f16 = d->type == LL_F16;

  const DeviceInfo* info = nullptr;
  s = current_device(&p.device, &info);
  if (s != LL_OK) return s;
  p.cus = info->cus;

  // Whether the softmax runs in the logits' product (the hand-ordered kind's
  // 256x256 tiles, whatever kind a plain product would take): from half a
  // tile of rows on, when the tiles fill half of the CUs.  Both ways, us: loss
  // and gradients 4096 x 131072 x 4096 10128 against 13096, 16384 x 8192 x 512
  // 620 / 819, 1024 x 32768 x 2048 421 / 477, 256 x 32768 x 2048 214 / 206;
  // loss alone 2000 x 9000 x 128 37 / 87, 256 x 32768 x 1024 40 / 44; with few
  // rows the tiles' empty rows cost more: 64 x 131072 x 2048 451 / 421 and 1 x
  // 131072 x 4096 718 / 669.  LL_XENT_FUSED=0 / 1 overrides (measurement).
  const int64_t N = d->N, limit = d->piece_bytes ? d->piece_bytes : kDefaultPieceBytes;
  const int64_t tiles = (N + 255) / 256 * ((d->V + 255) / 256);
  // x, and 256 rows of w, below 2 GB; whole 64-deep slices of w
  const bool fits = N * p.ldp < (1 << 30) && p.ldw < (1 << 22) && (d->D % 64 == 0 || p.pack_w);
  p.fused = fits && N > 128 && tiles * 2 > p.cus;
  if (const char* env = getenv("LL_XENT_FUSED")) p.fused = fits && N > 0 && env[0] == '1';
  // Narrow rows: forming a logit again costs less than storing it.  Loss and
  // gradients, us, stored / formed again: bf16 16384 x 131072 x 64 5849 / 2015,
  // 8192 x 32768 x 128 804 / 545, 1746 x 68132 x 93 441 / 318, 224 x 1406 x 128
  // 44 / 34, fp16 14360 x 7374 x 64 377 / 169, 65 x 228624 x 64 173 / 86; loss
  // alone 1042 / 598, 161 / 123, 97 / 78, 16 / 17, 72 / 50, 77 / 18.  Up to 64
  // rows their own kernels win (3 x 47113 x 119 49 / 75).  LL_XENT_NARROW=0
  // overrides (measurement).
  p.narrow = d->D <= kXentNarrow && N > kXentFewRows;
  if (const char* env = getenv("LL_XENT_NARROW")) p.narrow = p.narrow && env[0] == '1';
  if (p.narrow) p.fused = false;
  p.rows = p.fused ? round_up(N, 256) : std::max<int64_t>(N, 1);

  // Pieces of the vocabulary: as many columns as the bound holds, in whole
  // tiles, all pieces alike but the last; a piece of w and of dz stays below
  // 2 GB, which the hand-ordered kind's descriptors need.  Where numerators are
  // kept but not all fit, a piece is a quarter of what fits, so that most of
  // the bound is used.  A 16-bit dw of fp16 is charged 4 D bytes per column for an
  // fp32 dw, also where its product takes the scale out (dw_scaled, below) and no
  // such buffer exists: 4096 x 131072 x 4096 is cut into 7 pieces, 11.0 ms
  // against 10.0 in one piece with bf16.
  const bool f16_dw = p.dw && f16 && d->dw_type != LL_F32;
  const bool few_rows = N >= 1 && N <= kXentFewRows && !p.fused && !p.narrow;
  const int64_t two_gb = (1 << 30) / std::max(grads ? p.rows : 1, p.ldw) - 256;
  const int64_t per_row = p.fused ? (grads ? 2 : 0) : grads ? 6 : 4;
  // few rows in one piece write dw in its own type
  const bool few_dw = few_rows && d->V <= std::min(limit / (p.rows * per_row), two_gb);
  const int64_t per_col = p.rows * per_row + (f16_dw && !few_dw ? d->D * 4 : 0);
  int64_t cols = std::min(per_col ? limit / per_col : two_gb, two_gb);
  if (p.fused && grads && cols < d->V) cols = std::min(limit / 4 / per_col, two_gb);
  cols = std::max<int64_t>(cols / 256 * 256, 256);
  p.pieces = (int)((d->V + cols - 1) / cols);
  p.cols = round_up((d->V + p.pieces - 1) / p.pieces, 256);
  p.pieces = (int)((d->V + p.cols - 1) / p.cols);
  const int64_t last = d->V - (p.pieces - 1) * p.cols;
  const int64_t first = p.pieces > 1 ? p.cols : last;
  p.ldz = round_up(first, 4);
  p.ldd = round_up(first, 256);
  const int64_t slot = p.rows * p.ldd * 2;
  p.kept = !grads ? 0 : p.fused ? (int)std::max<int64_t>(1, std::min<int64_t>(p.pieces, limit / slot)) : 1;
  // Fused: a part is 128 columns, two per tile.  Else parts of at least 1024
  // columns, up to 8 workgroups per CU over all rows.
  p.parts = p.fused ? (int)(p.ldd / 128)
                    : (int)std::max<int64_t>(1, std::min<int64_t>((first + 1023) / 1024, 8ll * p.cus / p.rows));
  p.np = (p.pieces - 1) * p.parts + (p.fused ? (int)(round_up(last, 256) / 128) : p.parts);
  p.dx_direct = p.dx && p.pieces == 1 && !f16;
  // Few rows: w streamed once past x in LDS; dw streamed out, by a kernel that
  // also serves rows that do not fit there; dx by a kernel of its own where a
  // general product would copy w first, go through fp32 (fp16) or fill one of
  // its 16-row tiles.  Loss and gradients, us, all general / logits and dw / dx
  // too: bf16 1 x 131072 x 4096 676 / 538 / 554, 4 x 233278 x 1417 1084 / 832 /
  // 609, 8 x 32000 x 2048 126 / 119 / 110, 32 x 131072 x 2048 369 / 337 / 354, 64
  // x 131072 x 1024 244 / 209 / 225; fp16 17 x 189756 x 896 307 / 274 / 229, 64 x
  // 100000 x 512 164 / 127 / 117.  LL_XENT_FEW: sum of 1 (logits), 2 (dx), 4
  // (dw) overrides (measurement).
  const bool few = few_rows && (!grads || p.pieces == 1);
  p.few = few && N * (round_up(d->D, 32) + 8) * 2 <= kXentFewBytes;
  p.few_dx = p.few && p.dx && (N <= 16 || f16 || p.pack_w);
  p.few_dw = few && p.dw;
  if (const char* env = getenv("LL_XENT_FEW")) {
    const int on = atoi(env);
    p.few = p.few && (on & 1);
    p.few_dx = few && p.dx && (on & 2);
    p.few_dw = p.few_dw && (on & 4);
  }
  // no copy of w where no general product reads it
  p.any_w = p.pack_w;
  p.pack_w = p.pack_w && !p.narrow && (!p.few || (p.dx && !p.few_dx));
  if (p.narrow) {
    p.pieces = 1;
    p.cols = round_up(d->V, 256);
    const int64_t slots = (p.ldp == 64 ? 3 : 2) * p.cus, each = p.dx && p.dw ? slots / 2 : slots;
    p.shares[0] = xent_narrow_shares(N, d->V, slots);
    p.shares[1] = p.dx ? xent_narrow_shares(N, d->V, each) : 0;
    p.shares[2] = p.dw ? xent_narrow_shares(d->V, N, each) : 0;
    p.parts = p.np = p.shares[0];
  }
  p.ldw = p.pack_w ? p.ldp : d->stride_w;
  if (p.few) {
    p.pieces = 1;
    p.cols = round_up(d->V, 256);
    p.ldz = round_up(d->V, 16);
    p.parts = p.np = (int)std::min<int64_t>((d->V + 15) / 16, p.cus);
  }
  p.by_row = !p.fused && !p.narrow && p.pieces == 1 && d->V <= kXentRowCols;
  p.x_direct = p.by_row && !p.few && d->stride_x % 8 == 0 && d->D % 8 == 0;
  // fp16: dw carries the scale of dz.  The hand-ordered kind takes it out in
  // its epilogue; where its tiles would fill less than half of the CUs, dw goes
  // through fp32 (in place for an fp32 dw).
  p.dw_scaled = p.dw && !p.few_dw && f16 && N > 0 && N * p.ldp < (1 << 30) && p.ldd * p.rows < (1 << 30) &&
                (first + 255) / 256 * ((d->D + 255) / 256) * 2 > p.cus;
  const bool dw_tmp = f16_dw && !p.dw_scaled && !p.few_dw;

  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off = align256(off + n);
    return at;
  };
  p.off_xp = take(p.narrow ? 0 : (size_t)N * p.ldp * 2);
  p.off_wp = take(p.pack_w ? (size_t)d->V * p.ldp * 2 : 0);
  p.off_zt = take((size_t)N * 4);
  p.off_lse = take((size_t)p.rows * 4);
  p.off_coef = take((size_t)p.rows * 4);
  p.off_column = take((size_t)p.rows * 4);
  p.off_scale = take(8);
  p.off_parts = take((size_t)p.rows * p.np * sizeof(float2));
  if (!p.fused && !p.narrow && (grads || !p.few)) p.off_z = take((size_t)N * p.ldz * 4);
  if (grads && !p.narrow) p.off_dz = take((size_t)slot * p.kept);
  if (p.dx && !p.dx_direct && !p.narrow) p.off_dxa = take((size_t)N * d->D * 4);
  if (p.dx && p.pieces > 1) p.off_dxb = take((size_t)N * d->D * 4);
  if (dw_tmp && !p.narrow) p.off_dwt = take((size_t)first * d->D * 4);
  p.dx_shares = p.few_dx ? xent_dx_few_shares(N, d->V, (int)d->D, p.cus) : 0;
  if (p.few_dx) p.off_dxp = take((size_t)p.dx_shares * N * d->D * 4);
  if (p.narrow) {
    if (p.shares[1] > 1) p.off_dxp = take((size_t)p.shares[1] * N * p.ldp * 4);
    if (p.shares[2] > 1) p.off_dwt = take((size_t)p.shares[2] * d->V * p.ldp * 4);
  }
  p.off_gemm = off;
  const uint32_t padded_w = p.pack_w ? kPaddedB : 0;
  for (int i = 0; i < 2 && !p.narrow; ++i) {
    const int64_t n = i ? last : first;
    gemm_desc g = p.fused ? product(N, n, d->D, p.ldp, 1, 1, p.ldw, p.ldd, d->type, d->type)
                          : product(N, n, d->D, p.ldp, 1, 1, p.ldw, p.ldz, d->type, LL_F32);
    if (!p.few) s = gemm_plan_build(&g, kPaddedA | padded_w | (p.fused ? kWholeTiles : 0), &p.logits[i]);
    if (s != LL_OK) return s;
    if (p.fused && n >= kPrefetchCols) p.logits[i].b_prefetch = 1;
    p.gemm_bytes = std::max(p.gemm_bytes, p.logits[i].ws_bytes);
    if (p.dx && !p.few_dx) {
      g = product(N, d->D, n, p.ldd, 1, p.ldw, 1, p.dx_direct ? d->stride_dx : d->D, d->type,
                  p.dx_direct ? d->dx_type : LL_F32);
      s = gemm_plan_build(&g, kPaddedA | padded_w | kDeepK, &p.dxp[i]);
      if (s != LL_OK) return s;
      if (i == 0 && p.pieces == 1 && p.dxp[0].deep) {
        // the splits' sum also takes the scale out and rounds
        p.dx_direct = p.dx_scaled = true;
        g.stride_cm = d->stride_dx;
        g.c_type = d->dx_type;
        s = gemm_plan_build(&g, kPaddedA | padded_w | kDeepK, &p.dxp[0]);
        if (s != LL_OK) return s;
      }
      p.gemm_bytes = std::max(p.gemm_bytes, p.dxp[i].ws_bytes);
    }
    if (p.dw && !p.few_dw) {
      g = product(n, d->D, N, 1, p.ldd, p.ldp, 1, dw_tmp ? d->D : d->stride_dw, d->type,
                  dw_tmp ? (int)LL_F32 : d->dw_type);
      s = gemm_plan_build(&g, kPaddedA | kPaddedB | (p.dw_scaled ? kWholeTiles : 0), &p.dwp[i]);
      if (s != LL_OK) return s;
      p.gemm_bytes = std::max(p.gemm_bytes, p.dwp[i].ws_bytes);
    }
  }
  if (p.x_direct) {
    gemm_desc g = product(N, d->V, d->D, d->stride_x, 1, 1, p.ldw, p.ldz, d->type, LL_F32);
    s = gemm_plan_build(&g, padded_w, &p.logits_x);
    if (s != LL_OK) return s;
    p.gemm_bytes = std::max(p.gemm_bytes, p.logits_x.ws_bytes);
  }
  p.ws_bytes = off + align256(p.gemm_bytes);
  xent_plan* h = new (std::nothrow) xent_plan(p);
  if (!h) return fail(LL_ERR_INVALID_ARG, "out of host memory");
  *out = h;
  return ok();
}

ll_status xent_plan_workspace_size(const xent_plan* p, size_t* bytes) {
  if (!p || !bytes) return fail(LL_ERR_INVALID_ARG, "null argument");
  *bytes = p->ws_bytes;
  return ok();
}

ll_status xent_plan_describe(const xent_plan* p, char* buf, size_t len) {
  if (!p || !buf || len == 0) return fail(LL_ERR_INVALID_ARG, "null argument");
  if (p->narrow) {
    snprintf(buf, len, "narrow shares=%d,%d,%d ws=%zu", p->shares[0], p->shares[1], p->shares[2], p->ws_bytes);
    return ok();
  }
  snprintf(buf, len, "pieces=%d cols=%lld kept=%d fused=%d packW=%d logits=%s dx=%s dw=%s ws=%zu", p->pieces,
           (long long)p->cols, p->kept, (int)p->fused, (int)p->pack_w,
           p->few ? "few_rows" : kind_info(p->logits[0].kind).name,
           !p->dx ? "-" : p->few_dx ? "few_rows" : kind_info(p->dxp[0].kind).name,
           !p->dw ? "-" : p->few_dw ? "few_rows" : kind_info(p->dwp[0].kind).name, p->ws_bytes);
  return ok();
}

ll_status xent_plan_destroy(xent_plan* p) {
  delete p;
  return ok();
}

ll_status xent_run(const xent_plan* p, const void* x, const void* w, const int64_t* target, const float* dloss,
                   float* loss, float* lse, void* dx, void* dw, void* ws, size_t ws_bytes, void* stream) {
  if (!p) return fail(LL_ERR_INVALID_ARG, "null plan");
  const xent_desc& d = p->d;
  const int64_t N = d.N;
  const bool grads = p->dx || p->dw;
  if (!w || (N > 0 && (!x || !target || !loss || (grads && !dloss) || (p->dx && !dx))) || (p->dw && !dw))
    return fail(LL_ERR_INVALID_ARG, "null pointer");
  auto bad = [](const void* q, size_t a) { return ((uintptr_t)q & (a - 1)) != 0; };
  if (bad(x, 2) || bad(w, 2) || bad(target, 8) || bad(dloss, 4) || bad(loss, 4) || bad(lse, 4) ||
      (p->dx && bad(dx, dtype_size(d.dx_type))) || (p->dw && bad(dw, dtype_size(d.dw_type))))
    return fail(LL_ERR_INVALID_ARG, "misaligned pointer");
  if (!p->any_w && bad(w, 16))
    return fail(LL_ERR_INVALID_ARG, "w must be 16-byte aligned unless packed (LL_XENT_PACK_W)");
  if (ws_bytes < p->ws_bytes || (p->ws_bytes > 0 && !ws))
    return fail(LL_ERR_WORKSPACE, "workspace %zu bytes, plan needs %zu", ws_bytes, p->ws_bytes);
  if (p->ws_bytes > 0 && bad(ws, 256)) return fail(LL_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  auto flat = [](const void* q, int64_t n, int64_t e) { return span_of(q, q && n > 0 ? 1 : 0, n, 0, 1, e); };
  const Span in[5] = {span_of(x, N, d.D, d.stride_x, 1, 2), span_of(w, d.V, d.D, d.stride_w, 1, 2),
                      flat(target, N, 8), flat(grads ? dloss : nullptr, N, 4), flat(ws, (int64_t)p->ws_bytes, 1)};
  const Span outs[4] = {flat(loss, N, 4), flat(lse, N, 4),
                        span_of(dx, p->dx ? N : 0, d.D, d.stride_dx, 1, p->dx ? dtype_size(d.dx_type) : 1),
                        span_of(dw, p->dw ? d.V : 0, d.D, d.stride_dw, 1, p->dw ? dtype_size(d.dw_type) : 1)};
  for (int i = 0; i < 4; ++i) {
    for (const Span& t : in)
      if (overlaps(outs[i], t)) return fail(LL_ERR_INVALID_ARG, "an output overlaps an input or the workspace");
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return fail(LL_ERR_INVALID_ARG, "outputs overlap");
  }
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev != p->device) return fail(LL_ERR_INVALID_ARG, "plan made for device %d, current is %d", p->device, dev);
  hipStream_t st = (hipStream_t)stream;
  char* const base = (char*)ws;
  void* const gws = base + p->off_gemm;
  const bool f16 = d.type == LL_F16;

  XentRows r;
  memset(&r, 0, sizeof r);
  r.x = x;
  r.w = w;
  r.target = target;
  r.dloss = grads ? dloss : nullptr;
  r.N = N;
  r.V = d.V;
  r.ldx = d.stride_x;
  r.ldw = d.stride_w;
  r.ignore = d.ignore_index;
  r.D = (int32_t)d.D;
  r.ldp = (int32_t)p->ldp;
  r.xp = base + p->off_xp;
  r.zt = (float*)(base + p->off_zt);
  r.lse = (float*)(base + p->off_lse);
  r.coef = (float*)(base + p->off_coef);
  r.scale = f16 && grads ? (float*)(base + p->off_scale) : nullptr;
  r.column = (int32_t*)(base + p->off_column);
  r.parts = (float2*)(base + p->off_parts);
  r.part_ld = p->rows;
  r.np = p->np;
  r.factor0 = p->fused && grads ? (p->pieces - p->kept) * p->parts : r.np;
  r.loss = loss;
  r.lse_out = lse;
  float* const z = (float*)(base + p->off_z);
  float* const dxa = (float*)(base + p->off_dxa);
  float* const dxb = (float*)(base + p->off_dxb);
  float* const dwt = (float*)(base + p->off_dwt);
  const float* const unscale = r.scale ? r.scale + 1 : nullptr;
  auto is_kept = [&](int k) { return k >= p->pieces - p->kept; };
  // kept pieces have their own place, the others the first one once its turn is over
  auto dz_of = [&](int k) -> void* {
    return base + p->off_dz + (is_kept(k) ? (size_t)(k - (p->pieces - p->kept)) * p->rows * p->ldd * 2 : 0);
  };

  const bool x_direct = p->x_direct && !bad(x, 16);
  bool scale_later = false;
  if (N > 0) {
    // fp16: the scale of dz, by the first kernel that reads no part of it
    const bool prep = !(p->few && (!grads || p->by_row)) && !x_direct && !p->narrow;
    if (prep) {
      e = launch_xent_prep(r, r.scale != nullptr, d.type, st);
      if (e != hipSuccess) return hip_fail(e, "xent prep launch");
    } else if (r.scale) {
      scale_later = p->few || p->narrow;
      if (!scale_later) e = launch_xent_scale(r, st);
      if (e != hipSuccess) return hip_fail(e, "xent scale launch");
    }
    if (p->pack_w) {
      e = launch_xent_pack(w, d.stride_w, d.V, (int)d.D, base + p->off_wp, (int)p->ldp, p->cus, st);
      if (e != hipSuccess) return hip_fail(e, "pack w launch");
    }
  }
  if (p->narrow) {
    e = launch_xent_narrow_stats(r, scale_later, d.type, st);
    if (e == hipSuccess) e = launch_xent_lse(r, st);
    if (e == hipSuccess && grads) {
      const XentNarrowOut ox = {dx, d.stride_dx, d.dx_type, p->shares[1],
                                p->shares[1] > 1 ? (float*)(base + p->off_dxp) : nullptr, unscale, 0, 0};
      const XentNarrowOut ow = {dw, d.stride_dw, d.dw_type, p->shares[2],
                                p->shares[2] > 1 ? (float*)(base + p->off_dwt) : nullptr, unscale, 0, 0};
      e = launch_xent_narrow_grad(r, ox, ow, d.type, st);
    }
    if (e != hipSuccess) return hip_fail(e, "xent narrow rows launch");
    return ok();
  }
  const uint16_t* const wk = p->pack_w ? (const uint16_t*)(base + p->off_wp) : (const uint16_t*)w;
  auto cols_of = [&](int k) { return (int)std::min(p->cols, d.V - (int64_t)k * p->cols); };
  // The logits' product of piece k, fused with softmax epilogue `epi` or into z.
  auto logits_of = [&](int k, int epi) {
    const uint16_t* const wp = wk + (int64_t)k * p->cols * p->ldw;
    const gemm_plan* const g = x_direct ? &p->logits_x : &p->logits[k + 1 == p->pieces];
    if (x_direct) return gemm_run_plan(g, x, wp, z, nullptr, gws, p->gemm_bytes, st);
    if (!p->fused) return gemm_run_plan(g, r.xp, wp, z, nullptr, gws, p->gemm_bytes, st);
    GemmKArgs x;
    memset(&x, 0, sizeof x);
    x.parts = r.parts;
    x.part_ld = r.part_ld;
    x.part0 = k * p->parts;
    x.col0 = (int32_t)(k * p->cols);
    x.lse = r.lse;
    x.coef = r.coef;
    x.column = r.column;
    return gemm_run_plan(g, r.xp, wp, epi == kSoftmaxStats ? nullptr : dz_of(k), nullptr, gws, p->gemm_bytes, st, epi,
                         &x);
  };
  ll_status s;
  if (p->few) {
    e = launch_xent_few(r, scale_later, grads ? z : nullptr, p->ldz, d.type, st);
    if (e != hipSuccess) return hip_fail(e, "xent few rows launch");
  }
  if (N > 0) {
    for (int k = 0; k < p->pieces && !p->few; ++k) {
      s = logits_of(k, grads && is_kept(k) ? kSoftmaxNumerators : kSoftmaxStats);
      if (s != LL_OK) return s;
      if (!p->fused && !p->by_row) {
        e = launch_xent_stats(r, z, p->ldz, cols_of(k), k * p->parts, p->parts, st);
        if (e != hipSuccess) return hip_fail(e, "xent stats launch");
      }
    }
    if (p->by_row && (grads || !p->few)) {
      XentRows q = r;
      if (!x_direct && !p->few) q.xp = nullptr;  // copied already
      if (!p->dw) q.xp = nullptr;
      e = launch_xent_rows(q, z, p->ldz, (int)d.V, grads ? dz_of(0) : nullptr, p->ldd, d.type, st);
      if (e != hipSuccess) return hip_fail(e, "xent rows launch");
    } else {
      e = launch_xent_lse(r, st);
      if (e != hipSuccess) return hip_fail(e, "xent lse launch");
    }
  }
  if (!grads) return ok();
  // The kept pieces first; the logits of the others are formed again.
  for (int k = p->pieces - 1, n = 0; k >= 0; --k, ++n) {
    const int li = k + 1 == p->pieces;
    const int64_t v0 = (int64_t)k * p->cols;
    const int cols = cols_of(k);
    void* const dz = dz_of(k);
    if (N > 0) {
      if (!is_kept(k)) {
        s = logits_of(k, kSoftmaxGradient);
        if (s != LL_OK) return s;
      }
      if (!p->fused && !p->by_row)
        e = launch_xent_dz(r, z, p->ldz, v0, cols, dz, p->ldd, d.type, p->cus, st);
      else if (p->fused && is_kept(k))
        e = launch_xent_numerators(r, dz, p->ldd, v0, cols, k * p->parts, d.type, st);
      if (e != hipSuccess) return hip_fail(e, "xent dz launch");
      if (p->few_dx) {
        float* const part = (float*)(base + p->off_dxp);
        e = launch_xent_dx_few(r, dz, p->ldd, part, d.type, p->cus, st);
        if (e == hipSuccess)
          e = launch_splitk_reduce_deep(part, p->dx_shares, N, d.D, dx, d.stride_dx, 1,
                                        d.dx_type == LL_BF16 ? 1 : d.dx_type == LL_F16 ? 2 : 0, unscale, st);
        if (e != hipSuccess) return hip_fail(e, "xent few rows dx launch");
      } else if (p->dx) {
        const gemm_plan* const g = &p->dxp[p->pieces == 1 ? 0 : li];
        const float* const f = p->dx_scaled ? unscale : nullptr;
        s = gemm_run_plan(g, dz, wk + v0 * p->ldw, p->dx_direct ? dx : n == 0 ? dxa : dxb, f, gws, p->gemm_bytes, st,
                          f ? kScaleEpilogue : 0);
        if (s != LL_OK) return s;
        if (!p->dx_direct) {
          if (k == 0)
            e = launch_xent_finish(dxa, n > 0 ? dxb : nullptr, unscale, N, d.D, d.D, dx, d.stride_dx, d.dx_type,
                                   p->cus, st);
          else if (n > 0)
            e = launch_xent_finish(dxa, dxb, nullptr, N, d.D, d.D, dxa, d.D, LL_F32, p->cus, st);
          if (e != hipSuccess) return hip_fail(e, "xent dx sum launch");
        }
      }
    }
    if (p->few_dw) {
      e = launch_xent_dw_few(r, dz, p->ldd, dw, d.stride_dw, d.dw_type, unscale, d.type, p->cus, st);
      if (e != hipSuccess) return hip_fail(e, "xent few rows dw launch");
    } else if (p->dw) {
      const int64_t esz = dtype_size(d.dw_type);
      char* const dst = (char*)dw + v0 * d.stride_dw * esz;
      const bool tmp = f16 && !p->dw_scaled && d.dw_type != LL_F32;
      s = gemm_run_plan(&p->dwp[li], dz, r.xp, tmp ? (void*)dwt : (void*)dst, p->dw_scaled ? unscale : nullptr, gws,
                        p->gemm_bytes, st, p->dw_scaled ? kScaleEpilogue : 0);
      if (s != LL_OK) return s;
      if (f16 && !p->dw_scaled) {
        e = launch_xent_finish(tmp ? dwt : (const float*)dst, nullptr, N > 0 ? unscale : nullptr, cols, d.D,
                               tmp ? d.D : d.stride_dw, dst, d.stride_dw, d.dw_type, p->cus, st);
        if (e != hipSuccess) return hip_fail(e, "xent dw scale launch");
      }
    }
  }
  return ok();
}

}  // extern "C"
