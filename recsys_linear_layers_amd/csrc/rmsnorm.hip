// Root-mean-square norm with the residual's addition in front,
//   h = x + residual,  y = h * rstd * gamma,  rstd = 1 / sqrt(mean(h^2) + eps),
// y in x's type or quantised in blocks of 128 of a row, and the gradients
//   n = h * rstd,  g = dy * gamma,
//   dx = rstd * (g - n * mean(g * n)) + dh,  dgamma = sum over rows of dy * n.
//
// Both are HBM bound: a row is read once and held in registers as stored words,
// so the sum of squares, the 8-bit blocks' maxima and the output need no second
// read.  h is rounded before the norm, so that the norm is that of the row the
// gradient and the next layer see.  16 (fp32: 32) neighbouring lanes hold a
// block of 128 columns: its maximum is a few lane exchanges.  The gradient
// keeps the column sums of dgamma in fp32 registers over all rows a workgroup
// visits; one partial row per workgroup goes to the workspace and a second
// kernel adds them in a fixed order, so the result does not depend on timing.
// h is multiplied by rstd before gamma: their product is of the size of 1, where
// h * gamma can overflow or lose its bits though y is an ordinary number.
#include "rmsnorm.hpp"

#include <algorithm>

#include "norm_rows.hpp"
#include "quant8.hpp"

namespace ll {

// Whether a row's values are loaded as ones read once (non-temporal).  With an odd
// number of 16-bit columns rows begin anywhere: pieces straddle lines, and the next
// piece wants the line kept (8191 x 5003 in rows of 5006, non-temporal and not: norm
// bf16 38 and 31 us, with residual fp16 65 and 63, its gradient 110 and 87; but in
// fp32 102 and 105, and at whole pieces 16384 x 8192 bf16 171 and 187).
template <int TY, bool TAIL>
constexpr bool read_once = !TAIL || TY == LL_F32;

// VEC columns of a row's 8-bit output and, once per block, its scale.  Lanes
// past the row's end take part with zeros.
template <int Q, int VEC, bool TAIL>
__device__ __forceinline__ void put_block8(const float (&y)[VEC], const RmsArgs& a, int64_t r, int d) {
  constexpr int LANES = kBlock8 / VEC;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VEC; ++i) m = max(m, magnitude(y[i]));
  const Scale8 s = scale8<Q>(lanes_max<LANES>(m));
  uint32_t w[VEC / 4];
#pragma unroll
  for (int i = 0; i < VEC; i += 4)
    w[i / 4] = pack8<Q>(y[i] * s.inv, y[i + 1] * s.inv, y[i + 2] * s.inv, y[i + 3] * s.inv);
  if (d >= a.D || r >= a.N) return;
  store8<TAIL>((uint8_t*)a.y + r * a.ldy + d, w, a.D - d);
  if (d % kBlock8 == 0) a.scale[r * a.sn + (int64_t)(d / kBlock8) * a.sb] = s.scale;
}

// TPR lanes hold a row; THREADS / TPR rows per workgroup and step.  OUT: the
// 8-bit type of y, or 0 for x's own.
template <int TY, int OUT, int VEC, int TPR, int NCH, int THREADS, bool TAIL, bool REG>
__global__ void __launch_bounds__(THREADS) rms_kernel(const RmsArgs a) {
  typedef Chunk<TY, VEC> C;
  typedef typename Elem<TY>::raw raw;
  __shared__ float red[2][THREADS / 64];
  constexpr int ROWS = THREADS / TPR;
  const int x = threadIdx.x % TPR, y = threadIdx.x / TPR;
  const float cols = (float)a.D;
  Params<TY, VEC, NCH, TAIL, REG> gamma;
  gamma.init(a.gamma, 1.f, x * VEC, TPR * VEC, a.D);
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t r = (int64_t)blockIdx.x * ROWS + y;
  int flip = 0;
  // The next row's loads go out before this row's sums, unless a row is one wave's
  // (65536 x 512 bf16 to 8 bits 45.4 -> 46.6; 16384 x 8192 bf16 without a residual 80 -> 77,
  // with one 172 -> 171, in 16 bits 188 -> 190; 4096 x 16384 87 -> 83, 8192 x 4096 fp32 74 -> 72).
  constexpr bool AHEAD = TPR > 64;
  typedef RowCols<TY, VEC, TPR, NCH, TAIL, read_once<TY, TAIL>> Cols;
  Cols nx, ne;
  auto fetch = [&](int64_t r) {
    const bool live = r < a.N;
    nx.load(a.x, a.ldx, r, live, x, a.D);
    if (a.residual) ne.load(a.residual, a.ldr, r, live, x, a.D);
  };
  if constexpr (AHEAD) fetch(r);
  // every row group takes part in each step's barriers
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.N; r0 += step, r += step, flip ^= 1) {
    const bool live = r < a.N;
    if constexpr (!AHEAD) fetch(r);
    Cols cur = nx;
    const Cols res = ne;
    if (AHEAD && r0 + step < a.N) fetch(r + step);
    if (a.residual) {
      raw* dst = (raw*)a.h + r * a.ldh;
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int d = (x + k * TPR) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) cur.v[k].put(i, cur.v[k].get(i) + res.v[k].get(i));
        if (live && d < a.D) cur.v[k].template store<TAIL, true>(dst + d, a.D - d);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) s = fmaf(cur.v[k].get(i), cur.v[k].get(i), s);
    row_sum<TPR, THREADS / 64>(s, red[flip]);
    const float rstd = 1.f / sqrtf(s / cols + a.eps);
    if (live && x == 0 && a.rstd) a.rstd[r] = rstd;
    raw* dst = (raw*)a.y + r * a.ldy;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int d = (x + k * TPR) * VEC;
      float g[VEC];
      if (d < a.D) gamma.get(k, d, a.D - d, g);
      if constexpr (OUT == 0) {
        if (!live || d >= a.D) continue;
        C o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) o.put(i, cur.v[k].get(i) * rstd * g[i]);
        o.template store<TAIL, true>(dst + d, a.D - d);
      } else {
        float v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = d < a.D && (!TAIL || d + i < a.D) ? cur.v[k].get(i) * rstd * g[i] : 0.f;
        put_block8<OUT, VEC, TAIL>(v, a, r, d);
      }
    }
  }
}

// Rows too wide for registers: one workgroup per row, which reads it (or h, just
// written) a second time, mostly from L2.
template <int TY, int OUT>
__global__ void __launch_bounds__(1024) rms_long_kernel(const RmsArgs a) {
  constexpr int VEC = kWide<TY>, STEP = 1024 * VEC;
  typedef Chunk<TY, VEC> C;
  typedef typename Elem<TY>::raw raw;
  __shared__ float red[2][16];
  int flip = 0;
  for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x, flip ^= 1) {
    const raw* src = (const raw*)a.x + r * a.ldx;
    float s = 0.f;
    for (int64_t d = threadIdx.x * VEC; d < a.D; d += STEP) {
      const int n = (int)min<int64_t>(VEC, a.D - d);
      C v;
      v.template load<true>(src + d, n);
      if (a.residual) {
        C e;
        e.template load<true>((const raw*)a.residual + r * a.ldr + d, n);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v.put(i, v.get(i) + e.get(i));
        v.template store<true>((raw*)a.h + r * a.ldh + d, n);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) s = fmaf(v.get(i), v.get(i), s);
    }
    row_sum<1024, 16>(s, red[flip]);
    const float rstd = 1.f / sqrtf(s / (float)a.D + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[r] = rstd;
    const raw* again = a.residual ? (const raw*)a.h + r * a.ldh : src;  // what this lane has written itself
    // whole waves, so that a block's lanes are all there
    for (int64_t d = threadIdx.x * VEC; d - (threadIdx.x & 63) * VEC < a.D; d += STEP) {
      const int n = (int)max<int64_t>(0, min<int64_t>(VEC, a.D - d));
      C v;
      float g[VEC], y[VEC];
      if (n > 0) {
        v.template load<true>(again + d, n);
        load_param<TY, VEC, true>(a.gamma, a.param_f32, (int)d, n, 1.f, g);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) y[i] = i < n ? v.get(i) * rstd * g[i] : 0.f;
      if constexpr (OUT == 0) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v.put(i, y[i]);
        if (n > 0) v.template store<true>((raw*)a.y + r * a.ldy + d, n);
      } else {
        put_block8<OUT, VEC, true>(y, a, r, (int)d);
      }
    }
  }
}

template <int TY, int OUT, int VEC, int TPR, int NCH, int THREADS, bool TAIL, bool REG>
static hipError_t rms_launch(const RmsArgs& a, int cus, hipStream_t s) {
  constexpr int ROWS = THREADS / TPR;
  const auto kernel = rms_kernel<TY, OUT, VEC, TPR, NCH, THREADS, TAIL, REG>;
  static const int resident = per_cu((const void*)kernel, THREADS);
  const int64_t blocks = std::min<int64_t>((a.N + ROWS - 1) / ROWS, (int64_t)cus * resident);
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(THREADS), 0, s, a);
  return hipGetLastError();
}

template <int TY, int OUT, int VEC, int TPR, int NCH, int THREADS, bool TAIL>
static hipError_t rms_go(const RmsArgs& a, int cus, hipStream_t s) {
  if constexpr (TY != LL_F32) {
    if (a.param_f32) return rms_launch<TY, OUT, VEC, TPR, NCH, THREADS, TAIL, false>(a, cus, s);
  }
  return rms_launch<TY, OUT, VEC, TPR, NCH, THREADS, TAIL, true>(a, cus, s);
}

// A lane holds up to 32 columns before more lanes take part in a row.
template <int TY, int OUT, bool TAIL>
static hipError_t launch_rms_t(const RmsArgs& a, int cus, hipStream_t s) {
  constexpr int VEC = kWide<TY>, K = 32 / VEC;
  const int chunks = (int)(((int64_t)a.D + VEC - 1) / VEC);
  if (chunks <= 64) return rms_go<TY, OUT, VEC, 64, 1, 256, TAIL>(a, cus, s);
  if (chunks <= 64 * (K / 2)) return rms_go<TY, OUT, VEC, 64, K / 2, 256, TAIL>(a, cus, s);
  if (chunks <= 256 * (K / 2)) return rms_go<TY, OUT, VEC, 256, K / 2, 256, TAIL>(a, cus, s);
  if (chunks <= 256 * K) return rms_go<TY, OUT, VEC, 256, K, 256, TAIL>(a, cus, s);
  if (a.D <= 16384) return rms_go<TY, OUT, VEC, 1024, K / 2, 1024, TAIL>(a, cus, s);
  const int64_t blocks = std::min<int64_t>(a.N, (int64_t)cus * 64);
  hipLaunchKernelGGL((rms_long_kernel<TY, OUT>), dim3((unsigned)blocks), dim3(1024), 0, s, a);
  return hipGetLastError();
}

template <int TY>
static hipError_t launch_rms_y(const RmsArgs& a, int y_type, int cus, hipStream_t s) {
  const bool tail = a.D % kWide<TY> != 0;
  if (y_type == LL_E4M3)
    return tail ? launch_rms_t<TY, LL_E4M3, true>(a, cus, s) : launch_rms_t<TY, LL_E4M3, false>(a, cus, s);
  if (y_type == LL_E5M2)
    return tail ? launch_rms_t<TY, LL_E5M2, true>(a, cus, s) : launch_rms_t<TY, LL_E5M2, false>(a, cus, s);
  return tail ? launch_rms_t<TY, 0, true>(a, cus, s) : launch_rms_t<TY, 0, false>(a, cus, s);
}

hipError_t launch_rmsnorm(const RmsArgs& a, int type, int y_type, int cus, hipStream_t s) {
  switch (type) {
    case LL_BF16: return launch_rms_y<LL_BF16>(a, y_type, cus, s);
    case LL_F16: return launch_rms_y<LL_F16>(a, y_type, cus, s);
    case LL_F32: return launch_rms_y<LL_F32>(a, y_type, cus, s);
    default: return hipErrorInvalidValue;
  }
}

// ---------------------------------------------------------------------------
// Gradients
// ---------------------------------------------------------------------------

// A lane's column sums stay in registers over all its rows; the row groups of a
// workgroup (THREADS / TPR) add theirs up at the end, in order, through LDS.
template <int TY, int VEC, int TPR, int NCH, int THREADS, bool TAIL, bool REG>
__global__ void __launch_bounds__(THREADS) rms_grad_kernel(const RmsGradArgs a) {
  typedef Chunk<TY, VEC> C;
  typedef typename Elem<TY>::raw raw;
  constexpr int ROWS = THREADS / TPR;
  __shared__ float red[2][THREADS / 64];
  __shared__ float col[ROWS > 1 ? THREADS * VEC : 1];
  const int x = threadIdx.x % TPR, y = threadIdx.x / TPR;
  const float cols = (float)a.D;
  Params<TY, VEC, NCH, TAIL, REG> gamma;
  gamma.init(a.gamma, 1.f, x * VEC, TPR * VEC, a.D);
  float dg[NCH][VEC];
#pragma unroll
  for (int k = 0; k < NCH; ++k)
#pragma unroll
    for (int i = 0; i < VEC; ++i) dg[k][i] = 0.f;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t r = (int64_t)blockIdx.x * ROWS + y;
  int flip = 0;
  // The next row's loads go out before this row's sums (4096 x 16384 104.5 -> 103, 65536 x
  // 512 53 -> 48; 8191 x 5003 in rows of 5006, fp16 86 -> 80, fp32 102 -> 93), but not in
  // whole pieces by 512 lanes, where many rows are in flight as it is and the registers
  // cost more (bf16, not ahead and ahead, 65536 x 4352 397 and 440, 16384 x 5120 116 and 126,
  // 16384 x 8192 188 and 193, without dh 137 and 146, in fp32 361 and 378; few rows gain 1 to
  // 3%: 4096 x 8192 54.6 and 52.9, 1024 x 8192 24.2 and 23.6, 8192 x 5120 fp32 119 and 116).
  constexpr bool AHEAD = TAIL || TPR != 512;
  typedef RowCols<TY, VEC, TPR, NCH, TAIL, read_once<TY, TAIL>> Cols;
  Cols nh, nd, ne;
  float nr;
  auto fetch = [&](int64_t r) {
    const bool live = r < a.N;
    nh.load(a.h, a.ldh, r, live, x, a.D);
    nd.load(a.dy, a.lddy, r, live, x, a.D);
    if (a.dh) ne.load(a.dh, a.lddh, r, live, x, a.D);
    nr = live ? a.rstd[r] : 0.f;
  };
  if constexpr (AHEAD) fetch(r);
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.N; r0 += step, r += step, flip ^= 1) {
    const bool live = r < a.N;
    if constexpr (!AHEAD) fetch(r);
    const Cols vh = nh, vd = nd, ve = ne;
    const float rstd = nr;
    if (AHEAD && r0 + step < a.N) fetch(r + step);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {  // dy and h are 0 past the row's end, so nothing is added there
      const int d = (x + k * TPR) * VEC;
      if (!REG && d >= a.D) continue;
      float g[VEC];
      gamma.get(k, d, a.D - d, g);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float v = vd.v[k].get(i), n = vh.v[k].get(i) * rstd;
        s = fmaf(v * g[i], n, s);
        dg[k][i] = fmaf(v, n, dg[k][i]);
      }
    }
    row_sum<TPR, THREADS / 64>(s, red[flip]);
    if (live) {
      const float m = s / cols;
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
          const float n = vh.v[k].get(i) * rstd;
          const float v = (vd.v[k].get(i) * g[i] - n * m) * rstd;
          o.put(i, a.dh ? v + ve.v[k].get(i) : v);
        }
        o.template store<TAIL, true>(dst + d, a.D - d);
      }
    }
  }
  if (!a.dgamma) return;
  const bool all = gridDim.x == 1;  // these sums are the result
  uint32_t* out = (uint32_t*)a.partial + (int64_t)blockIdx.x * a.D;
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const int d = (x + k * TPR) * VEC;
    Chunk<LL_F32, VEC> v;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v.put(i, dg[k][i]);
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
    if (y > 0 || d >= a.D) continue;
    if (!all) {
      v.template store<TAIL>(out + d, a.D - d);
    } else if (TY == LL_F32 || a.param_f32) {
      v.template store<TAIL>((uint32_t*)a.dgamma + d, a.D - d);
    } else {
      C c;
#pragma unroll
      for (int i = 0; i < VEC; ++i) c.put(i, v.get(i));
      c.template store<TAIL>((raw*)a.dgamma + d, a.D - d);
    }
  }
}

// Adds the partial rows: 64 columns per workgroup, 16 waves taking a
// sixteenth of the rows each, joined in order.
template <int TY>
__global__ void __launch_bounds__(1024) rms_reduce_kernel(const float* partial, int nblk, int D, void* dgamma,
                                                          int param_f32) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int lo = nblk * w / 16, hi = nblk * (w + 1) / 16;
  for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < D; c0 += (int64_t)gridDim.x * 64) {
    const int64_t c = c0 + lane;
    float s = 0.f;
    if (c < D) {
#pragma unroll 8
      for (int k = lo; k < hi; ++k) s += partial[(int64_t)k * D + c];
    }
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < D) {
#pragma unroll
      for (int i = 1; i < 16; ++i) s += red[i][lane];
      if (TY == LL_F32 || param_f32) ((float*)dgamma)[c] = s;
      else ((typename Elem<TY>::raw*)dgamma)[c] = Elem<TY>::put(s);
    }
    __syncthreads();  // red is free for the next columns
  }
}

// Rows too wide for registers: dx one workgroup per row in two passes, and the
// column sums in a kernel of their own, VEC columns per lane, workgroup y taking
// every gridDim.y-th row.
template <int TY>
__global__ void __launch_bounds__(1024) rms_grad_long_kernel(const RmsGradArgs a) {
  constexpr int VEC = kWide<TY>, STEP = 1024 * VEC;
  typedef Chunk<TY, VEC> C;
  typedef typename Elem<TY>::raw raw;
  __shared__ float red[2][16];
  int flip = 0;
  for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x, flip ^= 1) {
    const raw* sh = (const raw*)a.h + r * a.ldh;
    const raw* sd = (const raw*)a.dy + r * a.lddy;
    const float rstd = a.rstd[r];
    float s = 0.f;
    for (int64_t d = threadIdx.x * VEC; d < a.D; d += STEP) {
      const int n = (int)min<int64_t>(VEC, a.D - d);
      C vh, vd;
      float g[VEC];
      vh.template load<true>(sh + d, n);
      vd.template load<true>(sd + d, n);
      load_param<TY, VEC, true>(a.gamma, a.param_f32, (int)d, n, 1.f, g);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s = fmaf(vd.get(i) * g[i], vh.get(i) * rstd, s);
    }
    row_sum<1024, 16>(s, red[flip]);
    const float m = s / (float)a.D;
    for (int64_t d = threadIdx.x * VEC; d < a.D; d += STEP) {
      const int n = (int)min<int64_t>(VEC, a.D - d);
      C vh, vd, ve;
      float g[VEC];
      vh.template load<true>(sh + d, n);
      vd.template load<true>(sd + d, n);
      if (a.dh) ve.template load<true>((const raw*)a.dh + r * a.lddh + d, n);
      load_param<TY, VEC, true>(a.gamma, a.param_f32, (int)d, n, 1.f, g);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float v = (vd.get(i) * g[i] - vh.get(i) * rstd * m) * rstd;
        vd.put(i, a.dh ? v + ve.get(i) : v);
      }
      vd.template store<true>((raw*)a.dx + r * a.lddx + d, n);
    }
  }
}

template <int TY>
__global__ void __launch_bounds__(256) rms_grad_columns_kernel(const RmsGradArgs a) {
  constexpr int VEC = kWide<TY>;
  typedef Chunk<TY, VEC> C;
  typedef typename Elem<TY>::raw raw;
  const int64_t d = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
  if (d >= a.D) return;
  const int n = (int)min<int64_t>(VEC, a.D - d);
  Chunk<LL_F32, VEC> sum;
  sum.clear();
#pragma unroll 2
  for (int64_t r = blockIdx.y; r < a.N; r += gridDim.y) {
    C vh, vd;
    vh.template load<true>((const raw*)a.h + r * a.ldh + d, n);
    vd.template load<true>((const raw*)a.dy + r * a.lddy + d, n);
    const float rstd = a.rstd[r];
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum.put(i, fmaf(vd.get(i), vh.get(i) * rstd, sum.get(i)));
  }
  sum.template store<true>((uint32_t*)a.partial + (int64_t)blockIdx.y * a.D + d, n);
}

int rms_grad_blocks(int64_t N) { return (int)std::max<int64_t>(1, std::min<int64_t>(N, 512)); }

template <int TY, int VEC, int TPR, int NCH, int THREADS, bool TAIL>
static int rms_grad_go(const RmsGradArgs& a, hipStream_t s) {
  // Up to two rows per row group are one workgroup's, which saves the launch that
  // adds up (a call of 4 x 2048: 16.5 -> 12.4 us).
  constexpr int ROWS = THREADS / TPR;
  const int64_t steps = (a.N + ROWS - 1) / ROWS;
  const int blocks = steps <= 2 ? 1 : rms_grad_blocks(steps);
  auto kernel = rms_grad_kernel<TY, VEC, TPR, NCH, THREADS, TAIL, true>;
  if constexpr (TY != LL_F32) {
    if (a.param_f32) kernel = rms_grad_kernel<TY, VEC, TPR, NCH, THREADS, TAIL, false>;
  }
  hipLaunchKernelGGL(kernel, dim3(blocks), dim3(THREADS), 0, s, a);
  return blocks;
}

template <int TY, bool TAIL>
static hipError_t launch_rms_grad_t(const RmsGradArgs& a, int cus, hipStream_t s) {
  constexpr int VEC = kWide<TY>, K = 32 / VEC;
  const int chunks = (int)(((int64_t)a.D + VEC - 1) / VEC);
  int blocks;
  if (chunks <= 64) blocks = rms_grad_go<TY, VEC, 64, 1, 256, TAIL>(a, s);
  else if (chunks <= 64 * (K / 2)) blocks = rms_grad_go<TY, VEC, 64, K / 2, 256, TAIL>(a, s);
  else if (chunks <= 64 * K) blocks = rms_grad_go<TY, VEC, 64, K, 256, TAIL>(a, s);
  else if (chunks <= 256 * (K / 2)) blocks = rms_grad_go<TY, VEC, 256, K / 2, 256, TAIL>(a, s);
  else if (chunks <= 512 * (K / 2)) blocks = rms_grad_go<TY, VEC, 512, K / 2, 512, TAIL>(a, s);
  else if (a.D <= 16384) blocks = rms_grad_go<TY, VEC, 1024, K / 2, 1024, TAIL>(a, s);
  else {
    const int64_t rows = std::min<int64_t>(a.N, (int64_t)cus * 64);
    if (rows > 0)
      hipLaunchKernelGGL((rms_grad_long_kernel<TY>), dim3((unsigned)rows), dim3(1024), 0, s, a);
    const int across = (chunks + 255) / 256;  // a grid of 2^32 threads or more is not supported
    blocks = std::min(rms_grad_blocks(a.N), std::max(1, (1 << 23) / across));
    if (a.partial)
      hipLaunchKernelGGL((rms_grad_columns_kernel<TY>), dim3(across, blocks), dim3(256), 0, s, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.dgamma || (blocks == 1 && a.D <= 16384)) return e;
  // a grid of 2^32 threads or more is not supported
  const int64_t reduce = std::min<int64_t>(((int64_t)a.D + 63) / 64, 1 << 20);
  hipLaunchKernelGGL((rms_reduce_kernel<TY>), dim3((unsigned)reduce), dim3(1024), 0, s, a.partial, blocks, a.D,
                     a.dgamma, a.param_f32);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_grad(const RmsGradArgs& a, int type, int cus, hipStream_t s) {
  switch (type) {
    case LL_BF16:
      return a.D % 8 ? launch_rms_grad_t<LL_BF16, true>(a, cus, s) : launch_rms_grad_t<LL_BF16, false>(a, cus, s);
    case LL_F16:
      return a.D % 8 ? launch_rms_grad_t<LL_F16, true>(a, cus, s) : launch_rms_grad_t<LL_F16, false>(a, cus, s);
    case LL_F32:
      return a.D % 4 ? launch_rms_grad_t<LL_F32, true>(a, cus, s) : launch_rms_grad_t<LL_F32, false>(a, cus, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ll
