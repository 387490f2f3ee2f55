// The cross entropy of few rows: kernels that stream the vocabulary (or write its
// gradient) once at any alignment, where the tiles of a general product would
// be mostly empty and misaligned rows would have to be copied first.
#include <algorithm>

#include "ops_common.hpp"
#include "xent.hpp"
#include "xent_rows.hpp"

namespace ll {

// The logits of up to 64 rows (as far as x fits in LDS), w streamed
// once.
//
// HBM bound: 2 V D bytes of w against 2 N V D flops.  A wave takes 16 entries of
// the vocabulary: the 16x16x32 matrix instruction with w's rows as its rows and
// x's as its columns, NT times 16 of them (columns past N repeat row 0 and are
// dropped).  w goes straight from memory into the operand registers, 16 bytes
// per lane and instruction (64 bytes of each of the 16 rows), the next U loads
// always in flight while U are used: with U = 8 and 16 waves that is 128 KB per
// CU, what HBM latency takes.  x sits in LDS, rows 16 bytes apart beyond their
// length so that the 16 rows of a read fall on different banks.  Each lane keeps
// (maximum, sum) of its own entries over all its wave's tiles; lanes and waves
// are joined at the end, so a workgroup leaves one pair per row.
// 1 x 50021 x 2048: 35 us, 5.9 TB/s; the whole call at 64 x 131072 x 1024 58 us, 89
// with the logits through a product of their own.  (128 rows: the state of 8
// tiles does not fit in registers, 80 us against 58 at 128 x 131072 x 512.)

template <int TY, bool TAIL, int NT>
__global__ void __launch_bounds__(1024) xent_few_kernel(const XentRows r, float* z, int64_t ldz) {
  constexpr int U = NT <= 2 ? 8 : 4;
  typedef Chunk<TY, 8> C;
  extern __shared__ __attribute__((aligned(16))) uint16_t xs[];  // [N][Dp + 8], Dp: D up to whole 32s
  __shared__ float red[16][2][16];
  if ((int)blockIdx.x == r.np) {
    scale_block<1024>(r, red[0][0]);
    return;
  }
  const int N = (int)r.N, D = r.D, steps = (D + 31) / 32, pitch = steps * 32 + 8;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c16 = lane & 15, g = lane >> 4;
  for (int q = threadIdx.x; q < N * steps * 4; q += 1024) {
    const int i = q / (steps * 4), c = q % (steps * 4);
    C v;
    v.clear();
    if (8 * c < D) v.template load<TAIL>((const uint16_t*)r.x + i * r.ldx + 8 * c, D - 8 * c);
    __builtin_memcpy(xs + i * pitch + 8 * c, &v, 16);
  }
  int64_t t[NT];
  const uint16_t* xrow[NT];
  float m[NT], s[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int n = 16 * q + c16;
    t[q] = n < N ? r.target[n] : -1;
    xrow[q] = xs + (n < N ? n : 0) * pitch + 8 * g;
    m[q] = kNegInf;
    s[q] = 0.f;
  }
  __syncthreads();
  const int tiles = (int)((r.V + 15) / 16);
  const int full = D / 32 / U * U;  // steps taken U at a time, whole
  for (int tile = blockIdx.x + r.np * wave; tile < tiles; tile += r.np * 16) {
    const int64_t row = min((int64_t)tile * 16 + c16, r.V - 1);
    const uint16_t* const wrow = (const uint16_t*)r.w + row * r.ldw + 8 * g;
    f32x4 acc[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
    C cur[U];
    if (full > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u].template load<false>(wrow + 32 * u, 8);
    }
    for (int k = 0; k < full; k += U) {
      C next[U];
      if (k + U < full) {
#pragma unroll
        for (int u = 0; u < U; ++u) next[u].template load<false>(wrow + 32 * (k + U + u), 8);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          C b;
          __builtin_memcpy(&b, xrow[q] + 32 * (k + u), 16);
          acc[q] = mfma16(cur[u], b, acc[q]);
        }
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = next[u];
    }
    for (int k = full; k < steps; ++k) {
      const int left = D - 32 * k - 8 * g;
      C a;
      if (left > 0) a.template load<TAIL>(wrow + 32 * k, left);
      else a.clear();
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        C b;
        __builtin_memcpy(&b, xrow[q] + 32 * k, 16);
        acc[q] = mfma16(a, b, acc[q]);
      }
    }
    // lane: rows 16 q + c16 of x, entries 16 tile + 4 g + 0 .. 3
    const int64_t v0 = (int64_t)tile * 16 + 4 * g;
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const int n = 16 * q + c16;
      float m4 = kNegInf;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (v0 + i >= r.V) acc[q][i] = kNegInf;
        else if (v0 + i == t[q]) r.zt[n] = acc[q][i];
        m4 = fmaxf(m4, acc[q][i]);
      }
      float s4 = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) s4 += acc[q][i] == kNegInf ? 0.f : __expf(acc[q][i] - m4);
      join(m[q], s[q], m4, s4);
      if (z && n < N) *(f32x4*)(z + n * ldz + v0) = acc[q];  // ldz: whole groups of 16
    }
  }
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int n = 16 * q + (threadIdx.x & 15);
    join(m[q], s[q], __shfl_xor(m[q], 16, 64), __shfl_xor(s[q], 16, 64));
    join(m[q], s[q], __shfl_xor(m[q], 32, 64), __shfl_xor(s[q], 32, 64));
    if (q > 0) __syncthreads();  // red is still read for the rows before
    if (lane < 16) {
      red[wave][0][lane] = m[q];
      red[wave][1][lane] = s[q];
    }
    __syncthreads();
    if (threadIdx.x < 16 && n < N) {
      for (int k = 1; k < 16; ++k) join(m[q], s[q], red[k][0][lane], red[k][1][lane]);
      r.parts[(int64_t)blockIdx.x * r.part_ld + n] = float2{m[q], s[q]};
    }
  }
}

template <int TY, bool TAIL>
static void few_go(const XentRows& r, bool scaled, float* z, int64_t ldz, size_t lds, hipStream_t s) {
  if (r.N <= 16) hipLaunchKernelGGL((xent_few_kernel<TY, TAIL, 1>), dim3(r.np + scaled), dim3(1024), lds, s, r, z, ldz);
  else if (r.N <= 32) hipLaunchKernelGGL((xent_few_kernel<TY, TAIL, 2>), dim3(r.np + scaled), dim3(1024), lds, s, r, z, ldz);
  else hipLaunchKernelGGL((xent_few_kernel<TY, TAIL, 4>), dim3(r.np + scaled), dim3(1024), lds, s, r, z, ldz);
}

hipError_t launch_xent_few(const XentRows& r, bool scaled, float* z, int64_t ldz, int type, hipStream_t s) {
  const size_t lds = (size_t)r.N * ((r.D + 31) / 32 * 32 + 8) * 2;
  if (r.N < 1 || r.N > kXentFewRows || lds > (size_t)kXentFewBytes) return hipErrorInvalidValue;
  if (type == LL_BF16) {
    if (r.D % 8) few_go<LL_BF16, true>(r, scaled, z, ldz, lds, s);
    else few_go<LL_BF16, false>(r, scaled, z, ldz, lds, s);
  } else {
    if (r.D % 8) few_go<LL_F16, true>(r, scaled, z, ldz, lds, s);
    else few_go<LL_F16, false>(r, scaled, z, ldz, lds, s);
  }
  return hipGetLastError();
}

// Operand of a 16x16x32 matrix instruction from a row-major LDS tile whose rows
// are the inner dimension: lane l gets column c0 + l % 16, inner rows k0 + 8 (l /
// 16) + 0 .. 7, by two transposing reads.
template <int TY>
__device__ __forceinline__ Chunk<TY, 8> frag_tr(const uint16_t LL_LDS* tile, int pitch, int k0, int c0, int lane) {
  const int g = lane >> 4, sl = lane & 15;
  const uint16_t LL_LDS* const p = tile + (k0 + 8 * g + (sl >> 2)) * pitch + c0 + 4 * (sl & 3);
  return frag_pair<TY>(p, p + 4 * pitch);
}

// ---------------------------------------------------------------------------
// dw of few rows: dw[v][d] = *scale * sum_n dz[n][v] x[n][d].
//
// Bound by writing dw: 2 V D bytes against 2 N V D flops.  The matrix
// instruction's rows are columns d of x and its columns entries v, the inner
// dimension the rows n.  A wave keeps the operands of its 64 columns of x in
// registers for its whole life and takes dz 64 entries at a time from LDS.  Row
// m of the instruction's tile i is column 16 (m / 4) + 4 i + m % 4 of the 64, so
// that a lane ends up with 16 consecutive values of one row of dw.  They leave
// through LDS, 16 rows of 512 bytes together, 16 bytes per lane: stored straight
// from the registers each instruction would write half of every 32 bytes, which
// took 500 us instead of 185 for 131072 x 4096 of one row (1.07 GB, 5.8 TB/s; 64
// rows of 131072 x 1024 65 us, 4.1 TB/s).  Where rows are not 16-byte aligned, the
// 16-byte pieces are taken where dw is, at any element of the row in LDS, and the
// up to 7 elements left at its two ends by one 2-byte store per lane: 233278 x
// 1417 160 us, against 265 with 16-byte stores at odd addresses.
// ---------------------------------------------------------------------------

constexpr int kDwCols = 256, kDwEntries = 64;

template <int TY, int OT, int KS>
__global__ void __launch_bounds__(256) xent_dw_few_kernel(const XentRows r, const uint16_t* dz, int64_t ldd, void* dw,
                                                          int64_t ldo, const float* scale, int col_blocks) {
  constexpr int PITCH = kDwEntries + 8;
  typedef Chunk<TY, 8> C;
  typedef typename Elem<OT>::raw O;
  __shared__ __attribute__((aligned(16))) uint16_t tile[2][32 * KS * PITCH];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, c16 = lane & 15;
  const int d0 = (blockIdx.x % col_blocks) * kDwCols + wave * 64;
  const int N = (int)r.N;
  const float f = scale ? *scale : 1.f;
  // x's operands: lane: column d(c16, i), rows n = 32 k + 8 g + 0 .. 7
  C a[4][KS];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = d0 + 16 * (c16 >> 2) + 4 * i + (c16 & 3);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      a[i][k].clear();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int n = 32 * k + 8 * g + j;
        if (n < N && d < r.D) a[i][k].put_raw(j, ((const uint16_t*)r.xp)[(int64_t)n * r.ldp + d]);
      }
    }
  }
  const int blocks = (int)((r.V + kDwEntries - 1) / kDwEntries), step = gridDim.x / col_blocks;
  constexpr int OP = kDwCols + 32 / (int)sizeof(O);
  __shared__ __attribute__((aligned(16))) O out[16 * OP];
  const bool aligned = (((uintptr_t)dw | (uint64_t)ldo * sizeof(O)) & 15) == 0;
  const int left = r.D - (blockIdx.x % col_blocks) * kDwCols;  // columns from this workgroup's first on
  auto stage = [&](int b, int slot) {  // rows n of dz, entries 64 b ..; ldd covers whole 256s
    for (int q = threadIdx.x; q < 32 * KS * (kDwEntries / 8); q += 256) {
      const int n = q / (kDwEntries / 8), c = q % (kDwEntries / 8) * 8;
      C v;
      v.clear();
      if (n < N) v.template load<false>(dz + n * ldd + (int64_t)b * kDwEntries + c, 8);
      __builtin_memcpy(&tile[slot][n * PITCH + c], &v, 16);
    }
  };
  int b = blockIdx.x / col_blocks, slot = 0;
  if (b < blocks) stage(b, 0);
  for (; b < blocks; b += step, slot ^= 1) {
    __syncthreads();  // this block's dz is there, and the other slot is free
    if (b + step < blocks) stage(b + step, slot ^ 1);
    const uint16_t LL_LDS* const t = (const uint16_t LL_LDS*)tile[slot];
#pragma unroll
    for (int vt = 0; vt < kDwEntries / 16; ++vt) {
      f32x4 acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const C o = frag_tr<TY>(t, PITCH, 32 * k, 16 * vt, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = mfma16(a[i][k], o, acc[i]);
      }
      constexpr int W = kWide<OT>, LANES = kDwCols / W;
      __syncthreads();  // the 16 entries before have left
#pragma unroll
      for (int h = 0; h < 16; h += W) {
        Chunk<OT, W> o;
#pragma unroll
        for (int j = 0; j < W; ++j) o.put(j, acc[(h + j) >> 2][(h + j) & 3] * f);
        __builtin_memcpy(&out[c16 * OP + wave * 64 + 16 * g + h], &o, 16);
      }
      __syncthreads();
      const int l = threadIdx.x % LANES, cols = min(kDwCols, left);
#pragma unroll
      for (int e = threadIdx.x / LANES; e < 16; e += 256 / LANES) {
        const int64_t v = (int64_t)b * kDwEntries + 16 * vt + e;
        if (v >= r.V) break;
        O* const dst = (O*)dw + v * ldo + d0 - wave * 64;
        const O* const src = &out[e * OP];
        Chunk<OT, W> o;
        if (aligned) {
          if (W * l >= cols) continue;
          __builtin_memcpy(&o, src + W * l, 16);
          o.template store<true, true>(dst + W * l, cols - W * l);
        } else {
          const int at = (int)((uintptr_t)dst / sizeof(O)) & (W - 1), c = W * l - at;
          if (c >= 0 && c + W <= cols) {
            __builtin_memcpy(&o, src + c, 16);
            o.template store<false>(dst + c, W);
          }
          const int head = min(-at & (W - 1), cols), tail = max(head, ((cols + at) & -W) - at);
          const int q = l < W ? l : tail + l - W;
          if (l < 2 * W && q < (l < W ? head : cols)) dst[q] = src[q];
        }
      }
    }
  }
}

template <int TY, int OT>
static void dw_few_go(const XentRows& r, const void* dz, int64_t ldd, void* dw, int64_t ldo, const float* scale,
                      int cus, hipStream_t s) {
  const int cb = (r.D + kDwCols - 1) / kDwCols;
  const int64_t blocks = (r.V + kDwEntries - 1) / kDwEntries;
  // four workgroups per CU, each with several blocks of entries for its x
  const int64_t share = std::max<int64_t>(1, std::min<int64_t>(blocks, 4ll * cus / cb));
  const dim3 grid((unsigned)(share * cb));
  if (r.N <= 32)
    hipLaunchKernelGGL((xent_dw_few_kernel<TY, OT, 1>), grid, dim3(256), 0, s, r, (const uint16_t*)dz, ldd, dw, ldo,
                       scale, cb);
  else
    hipLaunchKernelGGL((xent_dw_few_kernel<TY, OT, 2>), grid, dim3(256), 0, s, r, (const uint16_t*)dz, ldd, dw, ldo,
                       scale, cb);
}

hipError_t launch_xent_dw_few(const XentRows& r, const void* dz, int64_t ldd, void* dw, int64_t ldo, int out_type,
                              const float* scale, int type, int cus, hipStream_t s) {
  if (r.N < 1 || r.N > kXentFewRows) return hipErrorInvalidValue;
  if (type == LL_BF16) {
    if (out_type == LL_F32) dw_few_go<LL_BF16, LL_F32>(r, dz, ldd, dw, ldo, scale, cus, s);
    else dw_few_go<LL_BF16, LL_BF16>(r, dz, ldd, dw, ldo, scale, cus, s);
  } else {
    if (out_type == LL_F32) dw_few_go<LL_F16, LL_F32>(r, dz, ldd, dw, ldo, scale, cus, s);
    else dw_few_go<LL_F16, LL_F16>(r, dz, ldd, dw, ldo, scale, cus, s);
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// dx of few rows: dx[n][d] = sum_v dz[n][v] w[v][d], w streamed once.
//
// HBM bound like the logits.  A workgroup takes 256 columns and a share of the
// vocabulary, 64 entries at a time through LDS (from registers, so w may start
// anywhere; the next 64 are loaded while these are used), a wave 64 of the
// columns: NT x 4 tiles of sums.  The shares' sums go to the workspace and are
// added by the reduce of a split product.  One row of 131072 x 4096 170 us (6.3
// TB/s), 4 rows of 233278 x 1417 134 us (4.9 TB/s), 64 rows of 131072 x 1024 69
// us (3.9 TB/s).
// ---------------------------------------------------------------------------

constexpr int kDxCols = 256, kDxEntries = 64;

template <int TY, int NT>
__global__ void __launch_bounds__(256) xent_dx_few_kernel(const XentRows r, const uint16_t* dz, int64_t ldd,
                                                          float* partial, int col_blocks) {
  constexpr int PITCH = kDxCols + 8, PER = kDxEntries * kDxCols / 8 / 256;  // 16-byte loads per thread
  typedef Chunk<TY, 8> C;
  __shared__ __attribute__((aligned(16))) uint16_t tile[kDxEntries * PITCH];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, c16 = lane & 15;
  const int d0 = (blockIdx.x % col_blocks) * kDxCols;
  const int N = (int)r.N, share = blockIdx.x / col_blocks, shares = gridDim.x / col_blocks;
  const int64_t blocks = (r.V + kDxEntries - 1) / kDxEntries;
  const int64_t b0 = blocks * share / shares, b1 = blocks * (share + 1) / shares;
  f32x4 acc[NT][4];
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[q][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  // thread: column chunk threadIdx % 32, entries threadIdx / 32 + 8 j
  const int wc = (threadIdx.x & 31) * 8, wv = threadIdx.x >> 5;
  C w[PER];
  auto load = [&](int64_t b) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int64_t v = b * kDxEntries + wv + 8 * j;
      if (v < r.V && d0 + wc < r.D)
        w[j].template load<true>((const uint16_t*)r.w + v * r.ldw + d0 + wc, r.D - d0 - wc);
      else w[j].clear();
    }
  };
  // dz: lane: row 16 q + c16, entries 32 k + 8 g + 0 .. 7 (zeros past V)
  C a[kDxEntries / 32][NT];
  auto load_a = [&](int64_t b) {
#pragma unroll
    for (int k = 0; k < kDxEntries / 32; ++k)
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const int n = min(16 * q + c16, N - 1);  // rows past N are not stored
        a[k][q].template load<false>(dz + n * ldd + b * kDxEntries + 32 * k + 8 * g, 8);
      }
  };
  if (b0 < b1) {
    load(b0);
    load_a(b0);
  }
  for (int64_t b = b0; b < b1; ++b) {
    __syncthreads();  // every wave is done with the entries before
#pragma unroll
    for (int j = 0; j < PER; ++j) __builtin_memcpy(&tile[(wv + 8 * j) * PITCH + wc], &w[j], 16);
    __syncthreads();
    if (b + 1 < b1) load(b + 1);
#pragma unroll
    for (int k = 0; k < kDxEntries / 32; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const C o = frag_tr<TY>((const uint16_t LL_LDS*)tile, PITCH, 32 * k, wave * 64 + 16 * i, lane);
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[q][i] = mfma16(a[k][q], o, acc[q][i]);
      }
    if (b + 1 < b1) load_a(b + 1);
  }
  float* const out = partial + (int64_t)share * N * r.D;
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = d0 + wave * 64 + 16 * i + c16;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = 16 * q + 4 * g + e;
        if (n < N && d < r.D) out[(int64_t)n * r.D + d] = acc[q][i][e];
      }
    }
}

// Shares: the chip filled once, and more as long as their sums (4 N D bytes each)
// stay an eighth of w, up to three workgroups per CU.
int xent_dx_few_shares(int64_t N, int64_t V, int D, int cus) {
  const int64_t cb = (D + kDxCols - 1) / kDxCols, blocks = (V + kDxEntries - 1) / kDxEntries;
  const int64_t most = std::min<int64_t>(std::min<int64_t>(blocks, 256), std::max<int64_t>(1, 3ll * cus / cb));
  const int64_t least = std::min<int64_t>(most, std::max<int64_t>(1, cus / cb));
  return (int)std::max(least, std::min(most, V / (16 * N)));
}

template <int TY>
static void dx_few_go(const XentRows& r, const void* dz, int64_t ldd, float* partial, int cus, hipStream_t s) {
  const int cb = (r.D + kDxCols - 1) / kDxCols;
  const dim3 grid((unsigned)(xent_dx_few_shares(r.N, r.V, r.D, cus) * cb));
  const uint16_t* const z = (const uint16_t*)dz;
  if (r.N <= 16) hipLaunchKernelGGL((xent_dx_few_kernel<TY, 1>), grid, dim3(256), 0, s, r, z, ldd, partial, cb);
  else if (r.N <= 32) hipLaunchKernelGGL((xent_dx_few_kernel<TY, 2>), grid, dim3(256), 0, s, r, z, ldd, partial, cb);
  else hipLaunchKernelGGL((xent_dx_few_kernel<TY, 4>), grid, dim3(256), 0, s, r, z, ldd, partial, cb);
}

hipError_t launch_xent_dx_few(const XentRows& r, const void* dz, int64_t ldd, float* partial, int type, int cus,
                              hipStream_t s) {
  if (r.N < 1 || r.N > kXentFewRows) return hipErrorInvalidValue;
  if (type == LL_BF16) dx_few_go<LL_BF16>(r, dz, ldd, partial, cus, s);
  else dx_few_go<LL_F16>(r, dz, ldd, partial, cus, s);
  return hipGetLastError();
}

}  // namespace ll
