// Layer norm y = (x - mean) * rstd * gamma + beta over the D columns of each
// row, rstd = 1 / sqrt(var + eps), and its gradients
//   h = dy * gamma,  xhat = (x - mean) * rstd,
//   dx = rstd * (h - mean_D(h) - xhat * mean_D(h * xhat)),
//   dgamma = sum over rows of dy * xhat,  dbeta = sum over rows of dy.
//
// Both are HBM bound: a row is read once and held in registers, so the mean,
// the variance around that mean (two passes over registers: no cancellation)
// and the output need no second read.  The gradient keeps the column sums of
// dgamma and dbeta in fp32 registers over all rows a workgroup visits; one
// partial row per workgroup goes to the workspace and a second kernel adds
// them in a fixed order, so the result does not depend on timing.
// 16384 x 8192 bf16: 88 us forward (6.1 TB/s), 157 backward (5.1) and 6 for the
// second kernel; 8191 x 5003 fp32 in rows of 5006, backward, 117 us (4.2).
#include "layernorm.hpp"

#include <algorithm>

#include "norm_rows.hpp"

namespace ll {

// TPR lanes hold a row; THREADS / TPR rows per workgroup and step.  Loading the
// next row ahead of this one's barriers gains nothing once as many workgroups
// run as fit: their rows are loads enough in flight.
template <int TY, int VEC, int TPR, int NCH, int THREADS, bool TAIL, bool REG>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormArgs a) {
  typedef Chunk<TY, VEC> C;
  typedef typename Elem<TY>::raw raw;
  __shared__ float red[2][THREADS / 64 * 2];
  constexpr int ROWS = THREADS / TPR;
  const int x = threadIdx.x % TPR, y = threadIdx.x / TPR;
  const float cols = (float)a.D;
  Params<TY, VEC, NCH, TAIL, REG> gamma, beta;
  gamma.init(a.gamma, 1.f, x * VEC, TPR * VEC, a.D);
  beta.init(a.beta, 0.f, x * VEC, TPR * VEC, a.D);
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t r = (int64_t)blockIdx.x * ROWS + y;
  RowCols<TY, VEC, TPR, NCH, TAIL> cur;
  cur.load(a.x, a.ldx, r, r < a.N, x, a.D);
  // every row group takes part in each step's barriers
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.N; r0 += step, r += step) {
    const bool live = r < a.N;
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) s += cur.v[k].get(i);
    row_sum2<TPR, THREADS / 64>(s, q, red[0]);
    const float mean = s / cols;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int n = a.D - (x + k * TPR) * VEC;  // columns of the row from this chunk on
      if (n <= 0) continue;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = TAIL && i >= n ? 0.f : cur.v[k].get(i) - mean;
        s = fmaf(d, d, s);
      }
    }
    row_sum2<TPR, THREADS / 64>(s, q, red[1]);
    const float rstd = 1.f / sqrtf(s / cols + a.eps);
    if (live) {
      raw* dst = (raw*)a.y + r * a.ldy;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int d = (x + k * TPR) * VEC;
        if (d >= a.D) continue;
        float g[VEC], b[VEC];
        gamma.get(k, d, a.D - d, g);
        beta.get(k, d, a.D - d, b);
        C o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) o.put(i, fmaf((cur.v[k].get(i) - mean) * rstd, g[i], b[i]));
        o.template store<TAIL, true>(dst + d, a.D - d);  // 98 -> 94 us at 16384 x 8192 bf16
      }
      if (x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
      }
    }
    if (r0 + step < a.N) cur.load(a.x, a.ldx, r + step, r + step < a.N, x, a.D);
  }
}

template <int TY, int VEC, int TPR, int NCH, int THREADS, bool TAIL, bool REG>
static hipError_t norm_launch(const NormArgs& a, int cus, hipStream_t s) {
  constexpr int ROWS = THREADS / TPR;
  const auto kernel = norm_kernel<TY, VEC, TPR, NCH, THREADS, TAIL, REG>;
  static const int resident = per_cu((const void*)kernel, THREADS);
  const int64_t blocks = std::min<int64_t>((a.N + ROWS - 1) / ROWS, (int64_t)cus * resident);
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(THREADS), 0, s, a);
  return hipGetLastError();
}

template <int TY, int VEC, int TPR, int NCH, int THREADS, bool TAIL>
static hipError_t norm_go(const NormArgs& a, int cus, hipStream_t s) {
  if constexpr (TY != LL_F32) {
    if (a.param_f32) return norm_launch<TY, VEC, TPR, NCH, THREADS, TAIL, false>(a, cus, s);
  }
  return norm_launch<TY, VEC, TPR, NCH, THREADS, TAIL, true>(a, cus, s);
}

// Rows too wide for registers: one workgroup per row, three passes over it
// (the second and third mostly from L2), one element per lane and access: bound
// by the accesses in flight, 4096 x 32768 bf16 433 us where the bytes alone take 87.
template <int TY>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
  typedef typename Elem<TY>::raw raw;
  __shared__ float red[2][32];
  const float cols = (float)a.D;
  for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x) {
    const raw* src = (const raw*)a.x + r * a.ldx;
    float s = 0.f, q = 0.f;
    for (int c = threadIdx.x; c < a.D; c += 1024) s += elem_at<TY>(src, c);
    row_sum2<1024, 16>(s, q, red[0]);
    const float mean = s / cols;
    s = 0.f;
    for (int c = threadIdx.x; c < a.D; c += 1024) {
      const float d = elem_at<TY>(src, c) - mean;
      s = fmaf(d, d, s);
    }
    row_sum2<1024, 16>(s, q, red[1]);
    const float rstd = 1.f / sqrtf(s / cols + a.eps);
    raw* dst = (raw*)a.y + r * a.ldy;
    for (int c = threadIdx.x; c < a.D; c += 1024)
      dst[c] = Elem<TY>::put(fmaf((elem_at<TY>(src, c) - mean) * rstd, param_at<TY>(a.gamma, a.param_f32, c, 1.f),
                                  param_at<TY>(a.beta, a.param_f32, c, 0.f)));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

// A lane holds up to 32 columns before more lanes take part in a row.
template <int TY, bool TAIL>
static hipError_t launch_norm_t(const NormArgs& a, int cus, hipStream_t s) {
  constexpr int VEC = kWide<TY>, K = 32 / VEC;
  const int chunks = (a.D + VEC - 1) / VEC;
  if (chunks <= 64) return norm_go<TY, VEC, 64, 1, 256, TAIL>(a, cus, s);
  if (chunks <= 64 * (K / 2)) return norm_go<TY, VEC, 64, K / 2, 256, TAIL>(a, cus, s);
  if (chunks <= 256 * (K / 2)) return norm_go<TY, VEC, 256, K / 2, 256, TAIL>(a, cus, s);
  if (chunks <= 256 * K) return norm_go<TY, VEC, 256, K, 256, TAIL>(a, cus, s);
  if (a.D <= 16384) return norm_go<TY, VEC, 1024, K / 2, 1024, TAIL>(a, cus, s);
  const int64_t blocks = std::min<int64_t>(a.N, (int64_t)cus * 64);
  hipLaunchKernelGGL((norm_long_kernel<TY>), dim3((unsigned)blocks), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_norm(const NormArgs& a, int type, int cus, hipStream_t s) {
  switch (type) {
    case LL_BF16: return a.D % 8 ? launch_norm_t<LL_BF16, true>(a, cus, s) : launch_norm_t<LL_BF16, false>(a, cus, s);
    case LL_F16: return a.D % 8 ? launch_norm_t<LL_F16, true>(a, cus, s) : launch_norm_t<LL_F16, false>(a, cus, s);
    case LL_F32: return a.D % 4 ? launch_norm_t<LL_F32, true>(a, cus, s) : launch_norm_t<LL_F32, false>(a, cus, s);
    default: return hipErrorInvalidValue;
  }
}

// ---------------------------------------------------------------------------
// Gradients
// ---------------------------------------------------------------------------

// A lane's column sums stay in registers over all its rows; the row groups of a
// workgroup (THREADS / TPR) add theirs up at the end, in order, through LDS.
// The next row is loaded once this one is done, not ahead: the registers that
// would hold it are those that let two more waves per SIMD run, and those cover
// the loads better (16384 x 8192 bf16 184 -> 166 us, 8192 x 16384 363 -> 174 us).
template <int TY, int VEC, int TPR, int NCH, int THREADS, bool TAIL, bool REG>
__global__ void __launch_bounds__(THREADS) norm_grad_kernel(const NormGradArgs a) {
  typedef Chunk<TY, VEC> C;
  typedef typename Elem<TY>::raw raw;
  constexpr int ROWS = THREADS / TPR;
  __shared__ float red[2][THREADS / 64 * 2];
  __shared__ float col[ROWS > 1 ? THREADS * VEC : 1];
  const int x = threadIdx.x % TPR, y = threadIdx.x / TPR;
  const float cols = (float)a.D;
  Params<TY, VEC, NCH, TAIL, REG> gamma;
  gamma.init(a.gamma, 1.f, x * VEC, TPR * VEC, a.D);
  float dg[NCH][VEC], db[NCH][VEC];
#pragma unroll
  for (int k = 0; k < NCH; ++k)
#pragma unroll
    for (int i = 0; i < VEC; ++i) dg[k][i] = db[k][i] = 0.f;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t r = (int64_t)blockIdx.x * ROWS + y;
  RowCols<TY, VEC, TPR, NCH, TAIL> vx, vd;
  vx.load(a.x, a.ldx, r, r < a.N, x, a.D);
  vd.load(a.dy, a.lddy, r, r < a.N, x, a.D);
  int flip = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.N; r0 += step, r += step, flip ^= 1) {
    const bool live = r < a.N;
    const float mean = live ? a.mean[r] : 0.f, rstd = live ? a.rstd[r] : 0.f;
    float s1 = 0.f, s2 = 0.f;
    // x is 0 past the row's end: where xhat is infinite there, dy's 0 would make a
    // NaN of it although the row's own values are finite.  (8191 x 5003 bf16 stays at
    // 82 us, fp32 in rows of 5006 goes from 121 to 124; with a select on xhat in the
    // loop instead, bf16 takes 117.)
    if (__builtin_expect(fabsf(mean * rstd) == __builtin_huge_valf(), 0))
      vx.repeat_first(a.x, a.ldx, r, x, a.D);
#pragma unroll
    for (int k = 0; k < NCH; ++k) {  // dy is 0 past the row's end, so nothing is added there
      const int d = (x + k * TPR) * VEC;
      float g[VEC];
      if (REG || d < a.D) gamma.get(k, d, a.D - d, g);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float v = vd.v[k].get(i), n = (vx.v[k].get(i) - mean) * rstd;
        const float h = REG || d < a.D ? v * g[i] : 0.f;
        s1 += h;
        s2 = fmaf(h, n, s2);
        dg[k][i] = fmaf(v, n, dg[k][i]);
        db[k][i] += v;
      }
    }
    row_sum2<TPR, THREADS / 64>(s1, s2, red[flip]);
    if (live) {
      const float m1 = s1 / cols, m2 = s2 / cols;
      raw* dst = (raw*)a.dx + r * a.lddx;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int d = (x + k * TPR) * VEC;
        if (d >= a.D) continue;
        float g[VEC];
        gamma.get(k, d, a.D - d, g);
        C o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float h = vd.v[k].get(i) * g[i], n = (vx.v[k].get(i) - mean) * rstd;
          o.put(i, (h - m1 - n * m2) * rstd);
        }
        o.template store<TAIL>(dst + d, a.D - d);
      }
    }
    if (r0 + step < a.N) {
      vx.load(a.x, a.ldx, r + step, r + step < a.N, x, a.D);
      vd.load(a.dy, a.lddy, r + step, r + step < a.N, x, a.D);
    }
  }
  if (!a.partial) return;
  uint32_t* out = (uint32_t*)a.partial + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const int d = (x + k * TPR) * VEC;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      Chunk<LL_F32, VEC> v;
#pragma unroll
      for (int i = 0; i < VEC; ++i) v.put(i, which ? db[k][i] : dg[k][i]);
      if constexpr (ROWS > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VEC; ++i) col[i * THREADS + threadIdx.x] = v.get(i);
        __syncthreads();
        if (y == 0) {
#pragma unroll
          for (int w = 1; w < ROWS; ++w)
#pragma unroll
            for (int i = 0; i < VEC; ++i) v.put(i, v.get(i) + col[i * THREADS + w * TPR + x]);
        }
      }
      if (y == 0 && d < a.D) v.template store<TAIL>(out + (int64_t)which * a.D + d, a.D - d);
    }
  }
}

// Adds the partial rows: 64 columns per workgroup, 16 waves taking a
// sixteenth of the rows each, joined in order.
template <int TY>
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* partial, int nblk, int D, void* dgamma,
                                                           void* dbeta, int param_f32) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int lo = nblk * w / 16, hi = nblk * (w + 1) / 16;
  for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < 2ll * D; c0 += (int64_t)gridDim.x * 64) {
    const int64_t col = c0 + lane;  // over both sums
    float s = 0.f;
    if (col < 2ll * D) {
#pragma unroll 8
      for (int k = lo; k < hi; ++k) s += partial[(int64_t)k * 2 * D + col];
    }
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && col < 2ll * D) {
#pragma unroll
      for (int i = 1; i < 16; ++i) s += red[i][lane];
      void* out = col < D ? dgamma : dbeta;
      const int64_t c = col < D ? col : col - D;
      if (TY == LL_F32 || param_f32) ((float*)out)[c] = s;
      else ((typename Elem<TY>::raw*)out)[c] = Elem<TY>::put(s);
    }
    __syncthreads();  // red is free for the next columns
  }
}

// Rows too wide for registers: dx one workgroup per row in two passes, and
// the column sums in a kernel of their own, thread per column, workgroup y
// taking every gridDim.y-th row (4096 x 32768 bf16: 540, 178 and 23 us for the
// join, of 130 for the bytes).
template <int TY>
__global__ void __launch_bounds__(1024) norm_grad_long_kernel(const NormGradArgs a) {
  typedef typename Elem<TY>::raw raw;
  __shared__ float red[2][32];
  const float cols = (float)a.D;
  int flip = 0;
  for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x, flip ^= 1) {
    const raw* sx = (const raw*)a.x + r * a.ldx;
    const raw* sd = (const raw*)a.dy + r * a.lddy;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < a.D; c += 1024) {
      const float h = elem_at<TY>(sd, c) * param_at<TY>(a.gamma, a.param_f32, c, 1.f);
      s1 += h;
      s2 = fmaf(h, (elem_at<TY>(sx, c) - mean) * rstd, s2);
    }
    row_sum2<1024, 16>(s1, s2, red[flip]);
    const float m1 = s1 / cols, m2 = s2 / cols;
    raw* dst = (raw*)a.dx + r * a.lddx;
    for (int c = threadIdx.x; c < a.D; c += 1024) {
      const float h = elem_at<TY>(sd, c) * param_at<TY>(a.gamma, a.param_f32, c, 1.f);
      dst[c] = Elem<TY>::put((h - m1 - (elem_at<TY>(sx, c) - mean) * rstd * m2) * rstd);
    }
  }
}

template <int TY>
__global__ void __launch_bounds__(256) norm_grad_columns_kernel(const NormGradArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.D) return;
  float dg = 0.f, db = 0.f;
  for (int64_t r = blockIdx.y; r < a.N; r += gridDim.y) {
    const float d = elem_at<TY>(a.dy, r * a.lddy + c);
    const float n = (elem_at<TY>(a.x, r * a.ldx + c) - a.mean[r]) * a.rstd[r];
    dg = fmaf(d, n, dg);
    db += d;
  }
  float* out = a.partial + (int64_t)blockIdx.y * 2 * a.D;
  out[c] = dg;
  out[a.D + c] = db;
}

int norm_grad_blocks(int64_t N) { return (int)std::max<int64_t>(1, std::min<int64_t>(N, 512)); }

template <int TY, int VEC, int TPR, int NCH, int THREADS, bool TAIL>
static int norm_grad_go(const NormGradArgs& a, hipStream_t s) {
  constexpr int ROWS = THREADS / TPR;
  const int blocks = norm_grad_blocks((a.N + ROWS - 1) / ROWS);
  auto kernel = norm_grad_kernel<TY, VEC, TPR, NCH, THREADS, TAIL, true>;
  if constexpr (TY != LL_F32) {
    if (a.param_f32) kernel = norm_grad_kernel<TY, VEC, TPR, NCH, THREADS, TAIL, false>;
  }
  hipLaunchKernelGGL(kernel, dim3(blocks), dim3(THREADS), 0, s, a);
  return blocks;
}

template <int TY, bool TAIL>
static hipError_t launch_norm_grad_t(const NormGradArgs& a, int cus, hipStream_t s) {
  constexpr int VEC = kWide<TY>, K = 32 / VEC;
  const int chunks = (a.D + VEC - 1) / VEC;
  int blocks;
  if (chunks <= 64) blocks = norm_grad_go<TY, VEC, 64, 1, 256, TAIL>(a, s);
  else if (chunks <= 64 * (K / 2)) blocks = norm_grad_go<TY, VEC, 64, K / 2, 256, TAIL>(a, s);
  else if (chunks <= 64 * K) blocks = norm_grad_go<TY, VEC, 64, K, 256, TAIL>(a, s);
  else if (chunks <= 256 * (K / 2)) blocks = norm_grad_go<TY, VEC, 256, K / 2, 256, TAIL>(a, s);
  else if (chunks <= 512 * (K / 2)) blocks = norm_grad_go<TY, VEC, 512, K / 2, 512, TAIL>(a, s);
  else if (a.D <= 16384) blocks = norm_grad_go<TY, VEC, 1024, K / 2, 1024, TAIL>(a, s);
  else {
    const int64_t rows = std::min<int64_t>(a.N, (int64_t)cus * 64);
    if (rows > 0)
      hipLaunchKernelGGL((norm_grad_long_kernel<TY>), dim3((unsigned)rows), dim3(1024), 0, s, a);
    blocks = norm_grad_blocks(a.N);
    if (a.partial)
      hipLaunchKernelGGL((norm_grad_columns_kernel<TY>), dim3((a.D + 255) / 256, blocks), dim3(256), 0, s, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.partial) return e;
  // a grid of 2^32 threads or more is not supported
  const int64_t reduce = std::min<int64_t>((2ll * a.D + 63) / 64, 1 << 20);
  hipLaunchKernelGGL((norm_reduce_kernel<TY>), dim3((unsigned)reduce), dim3(1024), 0, s, a.partial, blocks, a.D,
                     a.dgamma, a.dbeta, a.param_f32);
  return hipGetLastError();
}

hipError_t launch_norm_grad(const NormGradArgs& a, int type, int cus, hipStream_t s) {
  switch (type) {
    case LL_BF16:
      return a.D % 8 ? launch_norm_grad_t<LL_BF16, true>(a, cus, s) : launch_norm_grad_t<LL_BF16, false>(a, cus, s);
    case LL_F16:
      return a.D % 8 ? launch_norm_grad_t<LL_F16, true>(a, cus, s) : launch_norm_grad_t<LL_F16, false>(a, cus, s);
    case LL_F32:
      return a.D % 4 ? launch_norm_grad_t<LL_F32, true>(a, cus, s) : launch_norm_grad_t<LL_F32, false>(a, cus, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ll
