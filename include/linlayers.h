/*
 * linlayers.h -- C ABI of the MI355X (gfx950) GEMM and RecSys linear-compression
 * library (liblinlayers.so).
 *
 * Operations (definitions from the pages this library follows):
 *
 *  - gemm_*   : C = act(A.B + bias) with bf16 (or fp16) A and B, fp32
 *               accumulation, fp32, bf16 or fp16 C; bias and activation optional.
 *               The problem is stated as on the page "Triton 3.7 permite
 *               extender el compilador de GPU sin forks" (listings in the
 *               sections "NVIDIA H100 (Hopper): GEMM persistente" and
 *               "AMD MI350: GEMM segmentado"): pointers a/b/c, sizes M, N, K and
 *               the element strides stride_am, stride_ak, stride_bk, stride_bn,
 *               stride_cm, stride_cn.  The tile sizes and stage count those
 *               listings take as compile-time constants are chosen inside the
 *               plan here.
 *  - lincomp_*: the RecSys linear-compression layer named on the page "Meta
 *               accelere un noyau GPU d'un facteur 4 avec TLX" (section on what
 *               a four-fold speed-up means).  For request r and candidate c the
 *               layer input X is the request's user rows stacked above the
 *               candidate's item rows, and Y[r][c] = W^T . X.  The user rows are
 *               identical across a request's candidates (section on how data
 *               loading holds back compute), so this entry point takes them
 *               once per request and computes their contribution once per
 *               request, not once per candidate.
 *  - embed_*, layernorm_*: what stands in front of a model's linear layers: the
 *               lookup of its tokens' (or items') rows and the norm of the
 *               activations, each with its gradients.
 *  - xent_*   : what stands behind them: the softmax cross entropy over a
 *               vocabulary, in pieces of the vocabulary, with its gradients.
 *  - rmsnorm_*, quant8_*, gemm8_*: linear layers in 8 bits: the norm in front
 *               (with the residual's addition, its output in 8 bits or not) and
 *               its gradient, the quantisation in blocks of 128, and the product
 *               of 8-bit operands with a scale per block.
 *
 * Conventions shared by every entry point:
 *
 *  - Pointers named A, B, C, user, item, W, Y and workspace are DEVICE
 *    pointers on the device the plan (or call) runs on; descriptors and plans
 *    are host memory.  The caller owns every buffer, including the workspace;
 *    the library never allocates device memory.  It owns only host plan
 *    objects (released by gemm_plan_destroy).
 *  - bf16 values are passed as their 16-bit patterns.  All strides are in
 *    ELEMENTS, not bytes.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Run calls only
 *    enqueue work and return; results are ready when the stream is.  Errors
 *    raised by the device (faults) surface at the caller's next
 *    synchronisation, not as a return value.
 *  - No exceptions cross this ABI.  Every call returns an ll_status.
 *  - Plans are immutable and may be shared between host threads; concurrent
 *    runs need distinct workspaces.
 */
#ifndef LINLAYERS_H
#define LINLAYERS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LL_OK = 0,
  LL_ERR_INVALID_ARG = 1,  /* null pointer, negative size, bad stride, overlap, wrong device */
  LL_ERR_UNSUPPORTED = 2,  /* dtype, layout or device (not gfx950) this library does not handle */
  LL_ERR_WORKSPACE = 3,    /* workspace smaller than the queried size */
  LL_ERR_HIP = 4,          /* a HIP runtime call or kernel launch failed */
  LL_ERR_NO_DEVICE = 5     /* no HIP device is visible */
} ll_status;

typedef enum {
  LL_BF16 = 0,
  LL_F32 = 1,
  LL_F16 = 2,  /* IEEE binary16 */
  LL_E4M3 = 3, /* 8 bits, 4 of exponent: up to 448, no infinities (the operands of gemm8) */
  LL_E5M2 = 4  /* 8 bits, 5 of exponent: up to 57344 */
} ll_dtype;

/* gemm_desc.flags */
#define LL_FLAG_PACK_A 0x1u /* always copy A into an aligned workspace layout first */
#define LL_FLAG_PACK_B 0x2u /* same for B */
#define LL_FLAG_PRODUCER_CONSUMER 0x4u /* force the wave-specialised (producer/consumer) kernel */
#define LL_FLAG_COOPERATIVE 0x8u       /* force the kernel in which every wave loads and computes */

/*
 * GEMM problem.  A[i][k] = A[i*stride_am + k*stride_ak] (0 <= i < M, 0 <= k < K),
 * B[k][j] = B[k*stride_bk + j*stride_bn], C[i][j] = C[i*stride_cm + j*stride_cn].
 * a_type and b_type: both LL_BF16 or both LL_F16 (the fp16 GEMMs of the
 * tables on "Triton 3.7 permite extender el compilador de GPU sin forks");
 * c_type is LL_BF16, LL_F16 or LL_F32.  Products are accumulated in fp32.
 * For A and for B, one of the two strides must be 1 (row- or column-major, any
 * leading dimension); C may use any positive strides.  16-bit C is rounded
 * to nearest even (fp16 overflow gives infinity).
 */
/*
 * gemm_desc.epilogue: what happens to each fp32 sum z = (A.B)[i][j] before it
 * is converted to c_type (page "Meta accélère un noyau GPU d'un facteur 4 avec
 * TLX", section "Par où commencer dans votre équipe": fuse steps, then
 * measure again).  LL_EPI_BIAS adds bias[j] (fp32, one per column of C,
 * passed to gemm_run_ex); then the activation, evaluated in fp32:
 *   LL_EPI_RELU  max(z, 0)
 *   LL_EPI_GELU  z * Phi(z) = z/2 * (1 + erf(z / sqrt(2)))  (the exact form)
 *   LL_EPI_SILU  z / (1 + exp(-z))
 * 0: C = A.B as before.  Unknown bits -> LL_ERR_INVALID_ARG.
 */
#define LL_EPI_BIAS 0x1u
#define LL_EPI_RELU 0x10u
#define LL_EPI_GELU 0x20u
#define LL_EPI_SILU 0x30u
#define LL_EPI_ACT_MASK 0xF0u

typedef struct {
  int64_t M, N, K;
  int64_t stride_am, stride_ak, stride_bk, stride_bn, stride_cm, stride_cn;
  int32_t a_type, b_type, c_type; /* ll_dtype values */
  uint32_t flags;                 /* LL_FLAG_* ; unknown bits -> LL_ERR_INVALID_ARG */
  uint32_t epilogue;              /* LL_EPI_* ; 0 for a plain product */
} gemm_desc;

typedef struct gemm_plan gemm_plan; /* opaque, host-side, immutable */

/*
 * Validate `desc` and choose the kernel configuration (tile shape, stage
 * count, wave roles, split-K factor, grid) for the CURRENT HIP device.
 * On success *out receives a new plan.
 * Tile choice: 256x128 or 128x256 tiles with separate loading waves (the
 * 256-long side along the shorter of M and N); 128x256 for M <= 128; 128x128
 * for M*N <= 2^20.  The persistent grid runs ceil(tiles / CUs) passes of
 * tiles, so when A is K-contiguous (or packed) and 192x256 tiles cover the
 * problem in passes x tile area at least 3% smaller, without a K split,
 * those are used instead.  Where 256x128 remains, A is K-contiguous, B is
 * N-contiguous and no epilogue is fused, 256x256 tiles (eight computing
 * waves, one per SIMD also loading) replace it when they need no more passes
 * x tile area; for K > 8192 the 128x256 tiles take their place again under
 * the same conditions.  Last, with A K- or M-contiguous (C = X^T Y, a
 * weight gradient) and B N- or K-contiguous (C = X W^T with W stored
 * [N][K]), direct or packed, K a multiple of 64 (or every K-contiguous
 * operand packed) and each operand spanning under 2 GB from its base, any
 * of those four kinds gives way to KIND_SQ4_HO (256x256 tiles,
 * four waves of 128x128, one per SIMD, each loading and computing in one
 * hand-ordered instruction stream) when that needs at most 1.25x their
 * passes x tile area (it runs ~1.3x as fast per pass and area); with or
 * without a fused epilogue.  K is split when the tiles fill
 * fewer than half of the CUs.  KIND_SQ4_HO plans with 8 rounds or more
 * (passes of the grid over the tiles) of K >= 8192 each, on a grid of whole
 * XCDs, also keep each
 * XCD's workgroups within a round of one another (round_sync=1 in the
 * description; LL_GEMM_ROUND_SYNC=0, or 1 for two rounds or more, overrides): a bounded wait between
 * rounds, so that tiles sharing A and B panels read them from L2 together;
 * its counters take 1 KB of workspace.  When a KIND_SQ4_HO plan's last round
 * would hold at most half as many tiles as the grid has workgroups (and K
 * has at least 32 slices of 64), those tiles are split 2-4 ways along K
 * (tail=<tiles>x<splits> in the description; LL_GEMM_TAIL_SPLIT=0 turns it
 * off): each split leaves a 256x256 fp32 partial in the workspace, and a
 * reduce kernel adds them in ascending split order, then applies the
 * epilogue.  KIND_SQ4_HO plans whose B is wide (an N-contiguous B's rows, as
 * read, 16384 elements or more apart; a K-contiguous B with N >= 16384), with
 * K >= 8192, also prefetch each B slice into L2 one slice ahead (prefetch_b=1; LL_GEMM_PREFETCH_B=0 or 1 overrides).  The environment variable LL_GEMM_KIND (a
 * kernel name as printed by gemm_plan_describe, or its index) forces a
 * kernel for configuration sweeps; a forced kernel that cannot take the
 * operands (a 192-row tile with an M-contiguous A, KIND_SQ4_HO outside the
 * conditions above) gives LL_ERR_UNSUPPORTED.
 * Errors: LL_ERR_INVALID_ARG (null out/desc, negative size, zero or negative
 * stride, unknown flag bits), LL_ERR_UNSUPPORTED (dtype, neither stride of A
 * or of B equal to 1, device not gfx950), LL_ERR_NO_DEVICE, LL_ERR_HIP.
 * Argument checks run before any device query.
 */
ll_status gemm_plan_create(gemm_plan** out, const gemm_desc* desc);

/* Bytes of device workspace gemm_run needs for this plan (may be 0). */
ll_status gemm_plan_workspace_size(const gemm_plan* plan, size_t* bytes);

/*
 * Writes a one-line, NUL-terminated description of the plan's choices
 * (kernel, tile, stages, roles, split-K, grid) into buf[0..len).
 */
ll_status gemm_plan_describe(const gemm_plan* plan, char* buf, size_t len);

/*
 * C = A.B on `stream`.  A, B: device buffers of a_type (bf16 or fp16); C:
 * device buffer of c_type.  Unless the plan packs an operand (LL_FLAG_PACK_*, or a layout that
 * needs it: leading dimension not a multiple of 8, K-contiguous operand with
 * K not a multiple of 8, M- or N-contiguous operand whose M or N is not a
 * multiple of 8), that operand's pointer must be 16-byte aligned.
 * M == 0 or N == 0: nothing is written.  K == 0: C is set to zero.
 * Errors: LL_ERR_INVALID_ARG (null plan/pointer with a non-empty problem,
 * misaligned operand, C overlapping A or B, current device differs from the
 * plan's), LL_ERR_WORKSPACE (ws_bytes below gemm_plan_workspace_size, a
 * null workspace with a non-zero requirement, or a workspace not 256-byte
 * aligned), LL_ERR_HIP (launch failure).  Packed copies live in the
 * workspace with rows padded to whole 128-byte lines: A K-contiguous
 * [M][ldp], B N-contiguous [K][ldp] (K-contiguous [N][ldp] when B is given
 * K-contiguous and A is K-contiguous); so do split-K partials, the round
 * counters of plans with round_sync=1 (zeroed by the call itself) and the
 * partial tiles of a K-split last round.
 * The call only launches kernels on `stream` (pack, counter clear, GEMM,
 * split-K or tail reduce, or the K == 0 fill): it allocates nothing and records no memset or copy, so
 * it may be captured into a HIP graph; replays reuse the captured pointers.
 */
ll_status gemm_run(const gemm_plan* plan, const void* A, const void* B, void* C,
                   void* workspace, size_t ws_bytes, void* stream);

/*
 * gemm_run for a plan whose epilogue adds a bias: `bias` is a device array of
 * N fp32 values (4-byte aligned), read once per output tile.  A plan without
 * LL_EPI_BIAS ignores `bias`; gemm_run on a plan with LL_EPI_BIAS, or a null
 * bias here, is LL_ERR_INVALID_ARG.  Otherwise as gemm_run.
 */
ll_status gemm_run_ex(const gemm_plan* plan, const void* A, const void* B, void* C, const float* bias,
                      void* workspace, size_t ws_bytes, void* stream);

/*
 * gemm_run_ex without a caller workspace, for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc.  The plan's workspace (packed operand copies,
 * split-K partials, round counters, tail partials) is taken from a device array inside the library, one per
 * GPU, LL_NOALLOC_SCRATCH_BYTES long, which each GPU the library runs on
 * holds from the library's load until the process ends.  The call allocates
 * and frees nothing and calls no allocating library routine; its first call
 * on a device looks up that device's array address once.
 * Every call on one GPU shares that GPU's array: calls that overlap in time on
 * one GPU (other streams, other host threads) race on it and give undefined
 * results; serialise them.  Each call writes every workspace byte it reads
 * before reading it, so nothing left by an earlier call matters.
 * bias: as for gemm_run_ex (required iff the plan's epilogue adds one,
 * ignored otherwise).  Results are identical to gemm_run_ex's.
 * Errors: LL_ERR_WORKSPACE if the plan needs more than
 * LL_NOALLOC_SCRATCH_BYTES (gemm_plan_workspace_size tells; nothing is
 * launched), otherwise as gemm_run_ex.
 */
#define LL_NOALLOC_SCRATCH_BYTES (64u << 20) /* 64 MiB */
ll_status gemm_run_noalloc(const gemm_plan* plan, const void* A, const void* B, void* C, const float* bias,
                           void* stream);

ll_status gemm_plan_destroy(gemm_plan* plan);

/*
 * Linear compression.  Sizes: R requests, C candidates per request, Nu user
 * rows, Ni item rows, D columns (embedding width), Mo compressed rows.
 *   user[r][c][n][d] = user[r*su_r + c*su_c + n*su_n + d] (0 <= n < Nu), bf16
 *   item[r][c][n][d] = item[r*si_r + c*si_c + n*si_n + d] (0 <= n < Ni), bf16
 *   W[n][m] = W[n*sw_n + m]                               (0 <= n < Nu+Ni), bf16
 *   Y[r][c][m][d] = Y[r*sy_r + c*sy_c + m*sy_m + d], y_type LL_BF16 or LL_F32
 * Y[r][c][m][d] = sum_{n<Nu} W[n][m] user[r][c][n][d] + sum_{n<Ni} W[Nu+n][m] item[r][c][n][d],
 * accumulated in fp32.  su_c == 0: the user rows are one block per request,
 * shared by all its candidates (the request's repeated features); the first
 * sum is then computed once per request and kept in fp32 (never rounded to
 * bf16) until the final result is rounded.  su_c != 0: every candidate
 * carries its own user rows (a materialised stacked input [user; item] per
 * candidate, the layer's original form); each candidate then computes both
 * sums, in the same order, so equal rows give bit-identical results.
 * The last dimension of every tensor is contiguous; user, item and W must be
 * 16-byte aligned and every stride a non-negative multiple of 8 (su_n, si_n,
 * sw_n, sy_m at least the row length); D and Mo multiples of 8.
 * flags: 0 = user block once per request (default); LL_LINCOMP_NO_DEDUP =
 * treat the user rows as if they were repeated for every candidate (each
 * candidate recomputes the user contribution; the result is the same sum).
 */
#define LL_LINCOMP_NO_DEDUP 0x1u

/*
 * epilogue: what happens to each fp32 sum Y[r][c][m][d] before it is
 * converted to y_type, fused into the layer (page "Meta accélère un noyau GPU
 * d'un facteur 4 avec TLX", section "Par où commencer dans votre équipe":
 * fuse steps, then measure again).  The LL_EPI_* bits of gemm_desc:
 * LL_EPI_BIAS adds bias[m] (fp32, one per compressed row, Mo values, passed
 * to lincomp_run_ex / lincomp_ragged_run_ex), then the activation LL_EPI_RELU,
 * LL_EPI_GELU (z * Phi(z), the exact form) or LL_EPI_SILU, in fp32.
 * 0: Y = W^T . X as before.  Unknown bits -> LL_ERR_INVALID_ARG.
 */
typedef struct {
  int64_t R, C, Nu, Ni, D, Mo;
  int64_t su_r, su_c, su_n;
  int64_t si_r, si_c, si_n;
  int64_t sw_n;
  int64_t sy_r, sy_c, sy_m;
  int32_t y_type; /* ll_dtype */
  uint32_t flags;
  uint32_t epilogue; /* LL_EPI_* ; 0 for the plain layer */
} lincomp_desc;

/* Bytes of device workspace lincomp_run needs for `desc` (may be 0).
 * Errors as for the argument checks of lincomp_run; no device is queried. */
ll_status lincomp_workspace_size(const lincomp_desc* desc, size_t* bytes);

/*
 * Y = linear compression of (user, item) by W, on `stream` (current device,
 * must be gfx950).  R == 0 or C == 0: nothing is written.
 * Errors: LL_ERR_INVALID_ARG (null desc/pointer, negative size, stride or
 * alignment rule above broken, Y overlapping an input), LL_ERR_UNSUPPORTED
 * (y_type, device), LL_ERR_WORKSPACE, LL_ERR_NO_DEVICE, LL_ERR_HIP.
 * The call launches one kernel on `stream` and allocates nothing, so it may
 * be captured into a HIP graph.
 */
ll_status lincomp_run(const lincomp_desc* desc, const void* user, const void* item,
                      const void* W, void* Y, void* workspace, size_t ws_bytes,
                      void* stream);

/*
 * lincomp_run for a descriptor whose epilogue adds a bias: `bias` is a device
 * array of Mo fp32 values, 16-byte aligned, bias[m] added to every Y[.][.][m][.].
 * A descriptor without LL_EPI_BIAS ignores `bias`; lincomp_run on a descriptor
 * with LL_EPI_BIAS, or a null or misaligned bias here, is LL_ERR_INVALID_ARG.
 * Otherwise as lincomp_run.
 */
ll_status lincomp_run_ex(const lincomp_desc* desc, const void* user, const void* item, const void* W,
                         const float* bias, void* Y, void* workspace, size_t ws_bytes, void* stream);

/*
 * Linear compression over ragged requests (page "Meta accélère un noyau GPU
 * d'un facteur 4 avec TLX", sections "Comment le chargement des données gêne
 * le calcul" and "Par où commencer dans votre équipe": the number of
 * candidates scored per request varies).  Request r owns the candidates
 * offsets[r] .. offsets[r+1]-1 of a flat candidate axis of length Ctot:
 *   user[r][n][d] = user[r*su_r + n*su_n + d]   (0 <= n < Nu), bf16
 *   item[g][n][d] = item[g*si_c + n*si_n + d]   (0 <= g < Ctot, 0 <= n < Ni), bf16
 *   W as for lincomp_run; Y[g][m][d] = Y[g*sy_c + m*sy_m + d], y_type
 * Y[g] = sum_{n<Nu} W[n][m] user[r(g)][n][d] + sum_{n<Ni} W[Nu+n][m] item[g][n][d],
 * with the user sum formed once per (request, work item) and kept in fp32.
 * offsets: device array of R+1 int64, non-decreasing, offsets[0] = 0,
 * offsets[R] = Ctot (read on the device; values outside [0, Ctot] are
 * clamped, and malformed offsets give unspecified rows of Y but no access
 * outside the buffers).  Candidates of empty requests do not exist; every
 * g in [0, Ctot) is written.  Alignment and stride rules as for
 * lincomp_run.  No workspace.  R == 0 or Ctot == 0: nothing is written.
 * Errors as for lincomp_run, plus LL_ERR_INVALID_ARG for a null offsets.
 */
typedef struct {
  int64_t R, Ctot, Nu, Ni, D, Mo;
  int64_t su_r, su_n;
  int64_t si_c, si_n;
  int64_t sw_n;
  int64_t sy_c, sy_m;
  int32_t y_type; /* ll_dtype */
  uint32_t flags; /* LL_LINCOMP_NO_DEDUP or 0 */
  uint32_t epilogue; /* LL_EPI_* as for lincomp_desc */
} lincomp_ragged_desc;

ll_status lincomp_ragged_run(const lincomp_ragged_desc* desc, const int64_t* offsets, const void* user,
                             const void* item, const void* W, void* Y, void* stream);

/* lincomp_ragged_run with the bias of an LL_EPI_BIAS epilogue (as lincomp_run_ex). */
ll_status lincomp_ragged_run_ex(const lincomp_ragged_desc* desc, const int64_t* offsets, const void* user,
                                const void* item, const void* W, const float* bias, void* Y, void* stream);

/*
 * Embedding lookup: out[t][d] = scale * table[ids[t]][d] (0 <= t < T, 0 <= d < D),
 * formed in fp32 and rounded once to `type` (LL_BF16, LL_F16 or LL_F32; table
 * and out alike).  Row r of the table starts at table + r*stride_table, row t
 * of out at out + t*stride_out; the last dimension is contiguous; strides at
 * least D.  ids: device array of T int64.  An id outside [0, V) gives a row
 * of zeros (no access outside the table).  T == 0 or D == 0: nothing is written.
 * One kernel on `stream`; no workspace; may be captured into a HIP graph.
 * Errors: LL_ERR_INVALID_ARG (null desc/pointer, negative size, stride below
 * D, a pointer not aligned to its element, out overlapping the table or ids),
 * LL_ERR_UNSUPPORTED (type, V of 2^31 - 1 and more, T or D above 2^31 - 2^12,
 * strides that put a row 2^58 elements or more from the first, device),
 * LL_ERR_NO_DEVICE, LL_ERR_HIP.
 */
typedef struct {
  int64_t V, T, D;
  int64_t stride_table, stride_out;
  int32_t type; /* ll_dtype of table and out */
  float scale;
} embed_desc;

ll_status embed_run(const embed_desc* desc, const void* table, const int64_t* ids, void* out, void* stream);

/*
 * Gradient of the lookup with respect to the table, dense:
 *   dtable[v][d] = scale * sum over t with ids[t] == v of dout[t][d]
 * for every 0 <= v < V (rows no token refers to are written as zeros).
 * Tokens whose id is padding_id or outside [0, V) contribute nothing
 * (padding_id -1: no padding).  LL_EMBED_ACCUMULATE: the sums are added to
 * dtable instead (a tied table, several batches); rows without a token are
 * then not touched.  Tokens are sorted by id, stably; each row is summed in
 * fp32, in an order that depends on the ids alone, and rounded once to
 * `type`, so equal inputs give equal bits.
 * Workspace (256-byte aligned): embed_grad_workspace_size; 0 for few tokens
 * into a small table.
 * Only kernels are launched, so the call may be captured into a HIP graph.
 * Errors as for embed_run (dtable must not overlap dout, ids or the
 * workspace), unknown flag bits (LL_ERR_INVALID_ARG), and LL_ERR_WORKSPACE.
 */
#define LL_EMBED_ACCUMULATE 0x1u

typedef struct {
  int64_t V, T, D;
  int64_t stride_dout, stride_dtable;
  int64_t padding_id;
  int32_t type; /* ll_dtype of dout and dtable */
  float scale;
  uint32_t flags; /* LL_EMBED_ACCUMULATE or 0 */
} embed_grad_desc;

ll_status embed_grad_workspace_size(const embed_grad_desc* desc, size_t* bytes);
ll_status embed_grad_run(const embed_grad_desc* desc, const int64_t* ids, const void* dout, void* dtable,
                         void* workspace, size_t ws_bytes, void* stream);

/*
 * Layer norm over the D columns of each of N rows:
 *   y = (x - mean) * rstd * gamma + beta,  rstd = 1 / sqrt(var + eps)
 * with mean and (biased) variance in fp32 from the row itself, the variance
 * around that mean; y rounded once to `type`.  x, y: row strides stride_x,
 * stride_y (elements, at least D), last dimension contiguous.  gamma, beta:
 * D values of param_type (`type` or LL_F32), each may be NULL (ones, zeros).
 * mean, rstd: N fp32 values each for the gradient, each may be NULL.
 * y may be x itself (same pointer and stride).  N == 0 or D == 0: nothing is
 * written.  One kernel on `stream`, no workspace, graph-capturable.
 * Errors: LL_ERR_INVALID_ARG (null desc, x or y; negative size, stride below
 * D, eps negative or not finite, misaligned pointer, y overlapping an input
 * otherwise), LL_ERR_UNSUPPORTED (types, D of 2^30 - 1 and more, N of 2^40 and
 * more, strides that put a row 2^58 elements or more from the first, device),
 * LL_ERR_NO_DEVICE, LL_ERR_HIP.
 */
typedef struct {
  int64_t N, D;
  int64_t stride_x, stride_y;
  int32_t type, param_type; /* ll_dtype */
  float eps;
} layernorm_desc;

ll_status layernorm_run(const layernorm_desc* desc, const void* x, const void* gamma, const void* beta, void* y,
                        float* mean, float* rstd, void* stream);

/*
 * Gradients of layer norm, from its input and the mean and rstd it gave:
 *   xhat = (x - mean) * rstd,  h = dy * gamma,
 *   dx = rstd * (h - mean_D(h) - xhat * mean_D(h * xhat)),
 *   dgamma = sum over rows of dy * xhat,  dbeta = sum over rows of dy
 * in fp32, each result rounded once.  dgamma and dbeta: D values of
 * param_type, both or neither NULL (neither wanted: dx alone).  Sums over
 * rows are formed in an order that depends on the sizes alone.  N == 0: dgamma
 * and dbeta are written as zeros.  Workspace (256-byte aligned):
 * layernorm_grad_workspace_size.  Kernels only, graph-capturable.
 * Errors as for layernorm_run (dx must not overlap any input), and
 * LL_ERR_WORKSPACE.
 */
typedef struct {
  int64_t N, D;
  int64_t stride_dy, stride_x, stride_dx;
  int32_t type, param_type; /* ll_dtype */
} layernorm_grad_desc;

ll_status layernorm_grad_workspace_size(const layernorm_grad_desc* desc, size_t* bytes);
ll_status layernorm_grad_run(const layernorm_grad_desc* desc, const void* dy, const void* x, const void* gamma,
                             const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta,
                             void* workspace, size_t ws_bytes, void* stream);

/*
 * Softmax cross entropy of N rows against a vocabulary of V entries, in pieces
 * of the vocabulary, without the [N][V] logits:
 *   z = x w^T,  lse[i] = log sum_v exp(z[i][v]),  loss[i] = lse[i] - z[i][target[i]],
 * and, for the gradient of sum_i dloss[i] * loss[i],
 *   dz = (exp(z - lse) - onehot(target)) * dloss,  dx = dz w,  dw = dz^T x.
 * x [N][D] and w [V][D] of `type` (LL_BF16 or LL_F16), rows stride_x and
 * stride_w elements apart, last dimension contiguous (w stored as a linear
 * layer's weight).  dx [N][D] and dw [V][D] of dx_type and dw_type (`type` or
 * LL_F32), rows stride_dx and stride_dw apart; LL_XENT_DX and LL_XENT_DW say
 * which are wanted (neither: the loss alone).
 * A row whose target is ignore_index or outside [0, V) has no loss: loss, lse
 * and its row of dx are zeros, and it adds nothing to dw, whatever it holds.
 * (dx = dz w meets 0 times infinity where w holds infinities.)  Entries of the
 * vocabulary may be masked by logits of any size, -infinity included.
 * Products are accumulated in fp32, row sums carried in fp32 with their
 * maximum; the loss is never negative.
 * dz is formed from z - lse with lse rounded to fp32 (|lse| 2^-24 of each
 * probability) and, as an operand of the matrix instruction, rounded to `type`
 * before the products: half a step, 2^-8 (bf16) or 2^-11 (fp16) of each
 * element, whatever dx_type and dw_type; dx and dw are rounded once more to
 * theirs.  (Their mean error is then about 1.4 times that of rounding them
 * alone.)  Before that, pieces whose softmax numerators are kept (below) hold
 * those as fp16 times 2^15: another 2^-11 of each, and numerators below 2^-40
 * of the largest of their 128 columns become 0; so the last bits of dx and dw
 * depend on piece_bytes.  With fp16, dz is multiplied by one power of two for
 * all rows, which brings the largest |dloss| to 2^13 or more and is taken out
 * again in fp32: a row whose |dloss| is 2^k times smaller than the largest
 * loses probabilities below 2^(k - 38).
 * piece_bytes bounds the buffers that hold logits, their softmax numerators and
 * dz (0: 2 GiB); when the whole vocabulary does not fit, it is cut into pieces of
 * a multiple of 256 entries (at least one such).  The numerators of as many
 * pieces as fit stay for the gradients, the logits of the others are formed
 * again.  With D up to 128 and more than 64 rows no logits are stored at all, and
 * piece_bytes has no effect.  w must be 16-byte aligned unless LL_XENT_PACK_W is
 * set (w may then be copied into the workspace), or D or stride_w is not a
 * multiple of 8, or
 * D not a multiple of 64 with 512 rows or more.
 */
#define LL_XENT_DX 0x1u
#define LL_XENT_DW 0x2u
#define LL_XENT_PACK_W 0x4u

typedef struct {
  int64_t N, V, D;
  int64_t stride_x, stride_w, stride_dx, stride_dw;
  int64_t ignore_index;
  int64_t piece_bytes;
  int32_t type, dx_type, dw_type; /* ll_dtype */
  uint32_t flags;                 /* LL_XENT_* */
} xent_desc;

typedef struct xent_plan xent_plan; /* opaque, host-side, immutable */

/*
 * Validate `desc` and choose pieces and products for the CURRENT HIP device.
 * Errors: LL_ERR_INVALID_ARG (null argument, negative size, V or D of zero,
 * stride below D, unknown flags), LL_ERR_UNSUPPORTED (types, N or V of 2^30 and
 * more, D of 2^20 and more, device), LL_ERR_NO_DEVICE, LL_ERR_HIP.
 * Argument checks run before any device query.
 */
ll_status xent_plan_create(xent_plan** out, const xent_desc* desc);
ll_status xent_plan_workspace_size(const xent_plan* plan, size_t* bytes);
/* One line: pieces, columns per piece, the kernels of the products. */
ll_status xent_plan_describe(const xent_plan* plan, char* buf, size_t len);

/*
 * Loss (and gradients, if the plan has them) on `stream`.  target: N int64;
 * dloss: N fp32, needed with gradients, ignored otherwise; loss: N fp32; lse:
 * N fp32 or NULL; dx, dw as the plan's flags say.  N == 0: dw, if wanted, is
 * written as zeros.  Kernels only: may be captured into a HIP graph.
 * Errors: LL_ERR_INVALID_ARG (null or misaligned pointer, an output overlapping
 * an input, the workspace or another output, current device differs from the
 * plan's), LL_ERR_WORKSPACE, LL_ERR_HIP.
 */
ll_status xent_run(const xent_plan* plan, const void* x, const void* w, const int64_t* target, const float* dloss,
                   float* loss, float* lse, void* dx, void* dw, void* workspace, size_t ws_bytes, void* stream);

ll_status xent_plan_destroy(xent_plan* plan);

/*
 * Linear layers in 8 bits.
 *
 * A quantised matrix is one of 8-bit values (LL_E4M3 or LL_E5M2), K the
 * dimension a product runs over, in rows of K consecutive values, and fp32
 * scales, one for each block of 128 values along K:
 *   block 1:   scale[row][k / 128], a block is 128 consecutive values of a row;
 *   block 128: scale[row / 128][k / 128], a block is 128 x 128 values.
 * Blocks at the ends are as short as the matrix.  The value that (i, k) stands
 * for is q[i][k] * scale.  Scales may have any positive strides (scale strides
 * are in fp32 elements); consecutive rows next to each other read fastest.
 *
 * How a block is quantised (here and in rmsnorm_run): with F the type's largest
 * value (448, 57344),
 *   scale = max(amax / F, 2^-126),  q = round(x * (1 / scale))
 * amax the largest magnitude of the block, each operation rounded to fp32, the
 * last to the 8-bit type, to nearest even: half a step, 2^-4 (e4m3) or 2^-3
 * (e5m2) of each value of at least 2^-14 (2^-29) of amax.  A block that holds a
 * NaN or an infinity has the scale NaN and NaNs in q.
 */

/*
 * Root-mean-square norm of each of N rows of D columns, with the residual's
 * addition in front:
 *   h = x + residual (rounded to `type`; h = x where residual is NULL)
 *   y = h * rstd * gamma,  rstd = 1 / sqrt(mean_D(h^2) + eps)
 * of h as it is stored, in fp32 (squares are summed in fp32: h beyond 2^63
 * overflows them, and beside an eps of 0 h below 2^-63 loses them), y formed in
 * this order and rounded once to y_type: `type`, or LL_E4M3 / LL_E5M2
 * quantised in blocks of 128 of a row (block 1 above), with scale[row][d / 128]
 * at scale + row*stride_sn + (d / 128)*stride_sb.
 * x, residual, h, y: row strides in elements, at least D, last dimension
 * contiguous.  gamma: D values of param_type (`type` or LL_F32), NULL: ones.
 * h: written if there is a residual (then required, else NULL); it may be x or
 * residual (same pointer and stride).  y may be x where there is no residual and
 * y_type is `type`.  rstd: N fp32 values for the gradient, may be NULL.
 * N == 0 or D == 0: nothing is written.  One kernel on `stream`, no workspace,
 * graph-capturable.
 * Errors: LL_ERR_INVALID_ARG (null desc, x, y, or scale with an 8-bit y, negative
 * size, stride below D, scale stride below 1, eps negative or not finite,
 * misaligned pointer, an output overlapping an input otherwise or another output),
 * LL_ERR_UNSUPPORTED (types, D of 2^30 - 1 and more, N of 2^40 and more, strides
 * that put a row 2^58 elements or more from the first, device),
 * LL_ERR_NO_DEVICE, LL_ERR_HIP.
 */
typedef struct {
  int64_t N, D;
  int64_t stride_x, stride_residual, stride_h, stride_y;
  int64_t stride_sn, stride_sb;      /* of scale; ignored unless y_type is an 8-bit type */
  int32_t type, param_type, y_type;  /* ll_dtype */
  float eps;
} rmsnorm_desc;

ll_status rmsnorm_run(const rmsnorm_desc* desc, const void* x, const void* residual, const void* gamma, void* h,
                      void* y, float* scale, float* rstd, void* stream);

/*
 * Gradients of the norm, from h as it saw it and the rstd it gave:
 *   n = h * rstd,  g = dy * gamma,
 *   dx = rstd * (g - n * mean_D(g * n)) + dh,  dgamma = sum over rows of dy * n
 * in fp32, each result rounded once.  dx is the gradient of h, and so of x and of
 * the residual; dh the gradient that reaches h by its other path, may be NULL,
 * and dx may be dh (same pointer and stride).  dgamma: D values of param_type,
 * may be NULL (not wanted).  Sums over rows are formed in an order that depends
 * on the sizes alone.  N == 0: dgamma is written as zeros.  Workspace (256-byte
 * aligned): rmsnorm_grad_workspace_size; none without dgamma.  Kernels only,
 * graph-capturable.  Errors as for rmsnorm_run, and LL_ERR_WORKSPACE.
 */
typedef struct {
  int64_t N, D;
  int64_t stride_dy, stride_h, stride_dh, stride_dx;
  int32_t type, param_type; /* ll_dtype */
} rmsnorm_grad_desc;

ll_status rmsnorm_grad_workspace_size(const rmsnorm_grad_desc* desc, size_t* bytes);
ll_status rmsnorm_grad_run(const rmsnorm_grad_desc* desc, const void* dy, const void* h, const void* gamma,
                           const float* rstd, const void* dh, void* dx, void* dgamma, void* workspace, size_t ws_bytes,
                           void* stream);

/*
 * Quantises x [N][D] (`type` LL_BF16, LL_F16 or LL_F32, row stride stride_x) in
 * blocks of 128, as it lies and/or transposed, reading x once:
 *   q [N][D] of q_type, rows stride_q apart, blocks along D (block 1: 128
 *     consecutive columns of a row; block 128: 128 x 128), with
 *     scale[n or n / 128][d / 128] at n'*stride_sn + d'*stride_sb;
 *   qt [D][N], rows stride_qt apart, blocks along N (block 1: 128 consecutive
 *     rows of a column of x), with scale_t[d or d / 128][n / 128] at
 *     d'*stride_tn + n'*stride_tb.
 * q with scale, or qt with scale_t, may be NULL (not wanted), not both pairs.
 * gemm8_run takes rows at multiples of 16 bytes: round stride_q (stride_qt) up.
 * N == 0 or D == 0: nothing is written.  One kernel, no workspace,
 * graph-capturable.  Errors: LL_ERR_INVALID_ARG (null desc, x or both forms, one
 * of a pair, negative size, strides below the rows or, for scales, below 1, block
 * other than 1 or 128, misaligned pointer, an output overlapping x or another
 * output), LL_ERR_UNSUPPORTED (types, N or D of 2^30 and more, strides that put a
 * row 2^58 elements or more from the first, device), LL_ERR_NO_DEVICE, LL_ERR_HIP.
 */
typedef struct {
  int64_t N, D;
  int64_t stride_x, stride_q, stride_qt;
  int64_t stride_sn, stride_sb, stride_tn, stride_tb;
  int32_t type, q_type; /* ll_dtype */
  int32_t block;        /* 1 or 128 */
} quant8_desc;

ll_status quant8_run(const quant8_desc* desc, const void* x, void* q, float* scale, void* qt, float* scale_t,
                     void* stream);

/*
 * The product of quantised matrices, both with K contiguous (a linear layer's
 * input rows and its weight as stored):
 *   C[i][j] = sum over b of a_scale[i][b] * b_scale[j or j / 128][b] *
 *             sum over k in block b of A[i][k] * B[j][k]
 * A [M][K] of a_type (LL_E4M3 or LL_E5M2), block 1; B [N][K], LL_E4M3, b_block 1
 * or 128; C [M][N] of c_type (LL_BF16, LL_F16 or LL_F32), rows stride_c apart.
 * A block's sum is formed by the matrix unit, the scaled sums are added in fp32 in
 * an order that sizes and strides alone decide, and C is rounded once, to nearest even.
 * With an fp32 C the blocks' sums have fp32's precision.  With a 16-bit C they come
 * from the 8-bit matrix instruction, twice as fast, which drops from the products
 * of a group of eight what lies below 2^-13 of the largest's power of two: at most
 * 7 * 2^-13 of the sum of the products' magnitudes, which is much of a C that is far
 * smaller than its products.  Measured, of the result's norm: 1.4e-5 on normally
 * distributed operands, 3e-5 to 7e-5 where a hundredth of A's columns stands out by
 * 20 to 1000; C's rounding is 1.6e-3 (bf16) or 2e-4 (fp16).  LL_GEMM8_FULL_SUMS: fp32's
 * precision for a 16-bit C too, at about an fp32 C's speed (beyond few rows M * N
 * fp32 values of the workspace hold the sums until they are rounded).  Equal inputs
 * give equal bits.  A layer's gradients are the same product: dX = dY W takes W
 * quantised transposed, dW = dY^T X takes dY and X quantised transposed, b_block 1.
 * The two scales of a block are multiplied first, in fp32: where that overflows, C is
 * an infinity or a NaN (also of sums that are 0), and below 2^-126 it loses bits.
 * A and B must be 16-byte aligned, stride_a and stride_b multiples of 16; the bytes
 * from K to the next multiple of 16 are read, behind the last row too, and not used
 * (device allocations end at multiples of more than that).  Workspace (256-byte
 * aligned): gemm8_workspace_size, often 0; only the call that it is given to uses
 * it.  M == 0 or N == 0: nothing is written.  K == 0: C is zero.  Kernels only,
 * graph-capturable.
 * Errors: LL_ERR_INVALID_ARG (null desc or pointer, negative size, stride below
 * the row, misaligned operand, scale stride below 1, b_block, unknown flag bits, C
 * overlapping an input or the workspace), LL_ERR_UNSUPPORTED (types, M, N of 2^26 and more, C of
 * more than 2^22 tiles of 256 x 256, K of 2^22 and more, stride_a or stride_b of
 * 2^22 and more, scale strides along rows of 2^20 and more, strides that put a row
 * or block 2^58 elements or more from the first, device), LL_ERR_WORKSPACE,
 * LL_ERR_NO_DEVICE, LL_ERR_HIP.
 */
#define LL_GEMM8_FULL_SUMS 0x1u
typedef struct {
  int64_t M, N, K;
  int64_t stride_a, stride_b, stride_c;
  int64_t stride_am, stride_ab; /* of a_scale: from row to row, from block to block */
  int64_t stride_bn, stride_bb; /* of b_scale */
  int32_t a_type, b_type, c_type;
  int32_t b_block; /* 1 or 128 */
  uint32_t flags;  /* LL_GEMM8_FULL_SUMS or 0 */
} gemm8_desc;

ll_status gemm8_workspace_size(const gemm8_desc* desc, size_t* bytes);
/* One line: the kernel, its tile, how K is split. */
ll_status gemm8_describe(const gemm8_desc* desc, char* buf, size_t len);
ll_status gemm8_run(const gemm8_desc* desc, const void* A, const float* a_scale, const void* B, const float* b_scale,
                    void* C, void* workspace, size_t ws_bytes, void* stream);

/* Static, human-readable name of a status code ("LL_OK", ...). */
const char* ll_status_string(ll_status s);

/* Message of the most recent failing call on this host thread ("" if none). */
const char* ll_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* LINLAYERS_H */
