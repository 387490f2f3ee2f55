// Row kernels of the vocabulary cross entropy: everything around its three
// matrix products.
//
//   z = x w^T,  lse = log sum_v exp(z_v),  loss = lse - z_target,
//   dz = (exp(z - lse) - onehot(target)) * dloss,  dx = dz w,  dw = dz^T x
//
// Row work beside the products, HBM or launch bound: 4096 x 131072 numerators into
// dz 371 us (2.1 GB, 5.8 TB/s), 32003 x 1000 of w packed 20 us (6.4 TB/s), the copy of
// 4096 x 4096 and its target logits 18 us, the join of 4096 x 1024 parts 18 us.
//
// The row sums are carried as pairs (m, s) with sum = s * exp(m), so any
// number of pieces of a row can be joined in any grouping without overflow.
#include "xent.hpp"

#include <algorithm>

#include "kernels.hpp"
#include "ops_common.hpp"
#include "xent_rows.hpp"

namespace ll {

// Over the 256 threads of a workgroup; every thread gets it.
__device__ __forceinline__ void block_join(float& m, float& s, float* red) {
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) join(m, s, __shfl_xor(m, k, 64), __shfl_xor(s, k, 64));
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    red[2 * wave] = m;
    red[2 * wave + 1] = s;
  }
  __syncthreads();
  m = red[0];
  s = red[1];
#pragma unroll
  for (int w = 1; w < 4; ++w) join(m, s, red[2 * w], red[2 * w + 1]);
}

// The aligned copy of x (a row without a target becomes zeros, so that whatever
// it holds cannot reach dw through 0 * inf), and the target's logit as a dot
// product of its own.  LANES lanes per row.
// One workgroup more forms the scale (scaled): a launch of its own costs 4 us.
template <int TY, int LANES>
__global__ void __launch_bounds__(256) xent_prep_kernel(const XentRows r, int scaled) {
  __shared__ float red[4];
  const int blocks = gridDim.x - scaled;
  if ((int)blockIdx.x == blocks) {
    scale_block<256>(r, red);
    return;
  }
  constexpr int ROWS = 256 / LANES;
  typedef Chunk<TY, 8> C;
  const int l = threadIdx.x % LANES, y = threadIdx.x / LANES;
  for (int64_t i0 = (int64_t)blockIdx.x * ROWS; i0 < r.N; i0 += (int64_t)blocks * ROWS) {
    const int64_t i = i0 + y;
    const int64_t t = i < r.N ? r.target[i] : -1;
    const bool live = has_target(r, t);
    const uint16_t* x = (const uint16_t*)r.x + i * r.ldx;
    const uint16_t* w = (const uint16_t*)r.w + (live ? t : 0) * r.ldw;
    uint16_t* dst = (uint16_t*)r.xp + i * r.ldp;
    float acc = 0.f;
    if (i < r.N) {
      for (int c = 8 * l; c < r.ldp; c += 8 * LANES) {
        C v, u;
        v.clear();
        u.clear();
        if (live && c < r.D) {
          v.template load<true>(x + c, r.D - c);
          u.template load<true>(w + c, r.D - c);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) acc = fmaf(v.get(k), u.get(k), acc);
        v.template store<false>(dst + c, 8);
      }
    }
    acc = lanes_sum<(LANES < 64 ? LANES : 64)>(acc);
    if constexpr (LANES == 256) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
      __syncthreads();
      acc = red[0] + red[1] + red[2] + red[3];
    }
    if (l == 0 && i < r.N) r.zt[i] = acc;
  }
}

// 16 bytes of a packed row per thread, rows of any alignment and width.
__global__ void __launch_bounds__(256) xent_pack_kernel(const uint16_t* src, int64_t lds, int64_t rows, int cols,
                                                        uint16_t* dst, int ldp) {
  const int chunks = ldp / 8;
  const int64_t n = rows * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = n >> 31 ? i / chunks : (int64_t)((uint32_t)i / (uint32_t)chunks);
    const int c = (int)(i - r * chunks) * 8;
    Chunk<LL_F16, 8> v;
    if (c < cols) v.load<true>(src + r * lds + c, cols - c);
    else v.clear();
    v.store<false>(dst + i * 8, 8);
  }
}

hipError_t launch_xent_pack(const void* src, int64_t lds, int64_t rows, int cols, void* dst, int ldp, int cus,
                            hipStream_t s) {
  const int64_t blocks = std::min<int64_t>((rows * (ldp / 8) + 1023) / 1024, 64ll * cus);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(xent_pack_kernel, dim3((unsigned)blocks), dim3(256), 0, s, (const uint16_t*)src, lds, rows, cols,
                     (uint16_t*)dst, ldp);
  return hipGetLastError();
}

hipError_t launch_xent_prep(const XentRows& r, bool scaled, int type, hipStream_t s) {
  const int lanes = r.ldp <= 128 ? 16 : r.ldp <= 512 ? 64 : 256, rows = 256 / lanes;
  const dim3 grid((unsigned)std::min<int64_t>((r.N + rows - 1) / rows, 1 << 16) + scaled);
#define LL_PREP(TY)                                                                                         \
  if (lanes == 16) hipLaunchKernelGGL((xent_prep_kernel<TY, 16>), grid, dim3(256), 0, s, r, (int)scaled);   \
  else if (lanes == 64) hipLaunchKernelGGL((xent_prep_kernel<TY, 64>), grid, dim3(256), 0, s, r, (int)scaled);\
  else hipLaunchKernelGGL((xent_prep_kernel<TY, 256>), grid, dim3(256), 0, s, r, (int)scaled);
  if (type == LL_BF16) {
    LL_PREP(LL_BF16)
  } else {
    LL_PREP(LL_F16)
  }
#undef LL_PREP
  return hipGetLastError();
}

__global__ void __launch_bounds__(1024) xent_scale_kernel(const XentRows r) {
  __shared__ float red[16];
  scale_block<1024>(r, red);
}

hipError_t launch_xent_scale(const XentRows& r, hipStream_t s) {
  hipLaunchKernelGGL(xent_scale_kernel, dim3(1), dim3(1024), 0, s, r);
  return hipGetLastError();
}

// Columns [lo, hi) of a split, in whole groups of four.
__device__ __forceinline__ void split_range(int cols, int splits, int k, int& lo, int& hi) {
  const int quads = (cols + 3) / 4;
  lo = (int)((int64_t)quads * k / splits) * 4;
  hi = min((int)((int64_t)quads * (k + 1) / splits) * 4, cols);
}

__global__ void __launch_bounds__(256) xent_stats_kernel(const XentRows r, const float* z, int64_t ldz, int cols,
                                                         int p0, int splits) {
  __shared__ float red[8];
  const int64_t items = r.N * splits;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t i = it / splits;
    const int k = (int)(it % splits);
    int lo, hi;
    split_range(cols, splits, k, lo, hi);
    const float* row = z + i * ldz;
    float m = kNegInf, s = 0.f;
    for (int c = lo + 4 * threadIdx.x; c < hi; c += 1024) {
      float v[4];
      const float4 q = *(const float4*)(row + c);  // ldz covers whole groups of four
      v[0] = q.x;
      v[1] = c + 1 < hi ? q.y : kNegInf;
      v[2] = c + 2 < hi ? q.z : kNegInf;
      v[3] = c + 3 < hi ? q.w : kNegInf;
      const float m4 = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
      float s4 = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) s4 += v[e] == kNegInf ? 0.f : __expf(v[e] - m4);
      join(m, s, m4, s4);
    }
    __syncthreads();
    block_join(m, s, red);
    if (threadIdx.x == 0) r.parts[(int64_t)(p0 + k) * r.part_ld + i] = float2{m, s};
  }
}

hipError_t launch_xent_stats(const XentRows& r, const float* z, int64_t ldz, int cols, int p0, int splits,
                             hipStream_t s) {
  const int64_t items = r.N * splits;
  hipLaunchKernelGGL(xent_stats_kernel, dim3((unsigned)std::min<int64_t>(items, 1 << 20)), dim3(256), 0, s, r, z, ldz,
                     cols, p0, splits);
  return hipGetLastError();
}

// Joins each row's parts: 16 rows per workgroup (a 128-byte line of each part),
// 64 lanes taking every 64th part of a row, joined in a fixed order.  The
// chain is a few loads long and the rows spread over the chip; 64 rows by 16
// lanes took 38 us at 4096 rows of 1024 parts.
__global__ void __launch_bounds__(1024) xent_lse_kernel(const XentRows r, int64_t first_row) {
  __shared__ float red[16][2][16];
  __shared__ float row_lse[16], row_coef[16];
  const int y = threadIdx.x & 15, g = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int64_t i = first_row + (int64_t)blockIdx.x * 16 + y;
  float m = kNegInf, s = 0.f;
  if (i < r.N) {
#pragma unroll 4
    for (int p = g; p < r.np; p += 64) {
      const float2 q = r.parts[(int64_t)p * r.part_ld + i];
      join(m, s, q.x, q.y);
    }
  }
  join(m, s, __shfl_xor(m, 16, 64), __shfl_xor(s, 16, 64));
  join(m, s, __shfl_xor(m, 32, 64), __shfl_xor(s, 32, 64));
  if ((threadIdx.x & 63) < 16) {
    red[wave][0][y] = m;
    red[wave][1][y] = s;
  }
  __syncthreads();
  if (threadIdx.x < 16 && i < r.N) {
    for (int k = 1; k < 16; ++k) join(m, s, red[k][0][y], red[k][1][y]);
    const int64_t t = r.target[i];
    const bool live = has_target(r, t);
    const float lse = live ? m + logf(s) : 0.f;
    const float coef = live && r.dloss ? r.dloss[i] * (r.scale ? r.scale[0] : 1.f) : 0.f;
    r.lse[i] = lse;
    r.coef[i] = coef;
    r.column[i] = live ? (int32_t)t : -1;
    // zt is a sum of its own, in another order than the logits: where the target has
    // almost all of the probability the difference of the roundings may be negative
    const float loss = lse - r.zt[i];
    r.loss[i] = live && !(loss < 0.f) ? loss : 0.f;
    if (r.lse_out) r.lse_out[i] = lse;
    row_lse[y] = lse;
    row_coef[y] = coef * (1.f / kNumeratorScale);
  }
  if (r.factor0 >= r.np) return;  // uniform
  __syncthreads();
  if (i >= r.N) return;
  for (int p = r.factor0 + g; p < r.np; p += 64) {
    float2* const q = &r.parts[(int64_t)p * r.part_ld + i];
    q->x = __expf(q->x - row_lse[y]) * row_coef[y];
  }
}

hipError_t launch_xent_lse(const XentRows& r, hipStream_t s) {
  // A grid of 2^32 threads or more is not supported.  (Rows in a loop of the kernel
  // instead: 5.5 -> 11 us at 14360 rows.)
  const int64_t most = 16ll << 20;
  for (int64_t i = 0; i < r.N; i += most)
    hipLaunchKernelGGL(xent_lse_kernel, dim3((unsigned)((std::min(r.N - i, most) + 15) / 16)), dim3(1024), 0, s, r, i);
  return hipGetLastError();
}

// The logits are read twice, the second time from L2 (a row is at most
// kXentRowCols values); a launch for each step instead took 4 us more apiece.
template <int TY>
__global__ void __launch_bounds__(256) xent_rows_kernel(const XentRows r, const float* z, int64_t ldz, int cols,
                                                        uint16_t* dz, int64_t ldd) {
  __shared__ float red[8];
  typedef Chunk<TY, 8> C;
  for (int64_t i = blockIdx.x; i < r.N; i += gridDim.x) {
    const int64_t t = r.target[i];
    const bool live = has_target(r, t);
    const float* row = z + i * ldz;
    float m = kNegInf, s = 0.f;
    if (live) {
      for (int c = 4 * threadIdx.x; c < cols; c += 1024) {
        const float4 q = *(const float4*)(row + c);  // ldz covers whole groups of four
        const float v[4] = {q.x, c + 1 < cols ? q.y : kNegInf, c + 2 < cols ? q.z : kNegInf,
                            c + 3 < cols ? q.w : kNegInf};
        const float m4 = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
        float s4 = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) s4 += v[e] == kNegInf ? 0.f : __expf(v[e] - m4);
        join(m, s, m4, s4);
      }
    }
    __syncthreads();  // red may still be read for the row before
    block_join(m, s, red);
    const float lse = live ? m + logf(s) : 0.f;
    if (threadIdx.x == 0) {
      r.loss[i] = live ? lse - row[t] : 0.f;
      if (r.lse_out) r.lse_out[i] = lse;
    }
    if (!dz) continue;
    const float coef = live ? r.dloss[i] * (r.scale ? r.scale[0] : 1.f) : 0.f;
    for (int c = 8 * threadIdx.x; c < ldd; c += 2048) {
      C o;
      o.clear();
      if (live) {
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
          if (c + h >= cols) continue;
          const float4 q = *(const float4*)(row + c + h);
          const float v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + h + e < cols) o.put(h + e, (__expf(v[e] - lse) - (c + h + e == t ? 1.f : 0.f)) * coef);
        }
      }
      o.template store<false>(dz + i * ldd + c, 8);
    }
    if (!r.xp) continue;
    const uint16_t* x = (const uint16_t*)r.x + i * r.ldx;
    for (int c = 8 * threadIdx.x; c < r.ldp; c += 2048) {
      C v;
      v.clear();
      if (live && c < r.D) v.template load<true>(x + c, r.D - c);
      v.template store<false>((uint16_t*)r.xp + i * r.ldp + c, 8);
    }
  }
}

hipError_t launch_xent_rows(const XentRows& r, const float* z, int64_t ldz, int cols, void* dz, int64_t ldd, int type,
                            hipStream_t s) {
  const dim3 grid((unsigned)std::min<int64_t>(r.N, 1 << 16));
  if (type == LL_BF16)
    hipLaunchKernelGGL((xent_rows_kernel<LL_BF16>), grid, dim3(256), 0, s, r, z, ldz, cols, (uint16_t*)dz, ldd);
  else
    hipLaunchKernelGGL((xent_rows_kernel<LL_F16>), grid, dim3(256), 0, s, r, z, ldz, cols, (uint16_t*)dz, ldd);
  return hipGetLastError();
}

// 64 rows by 256 columns (two parts) per workgroup, 8 columns per thread and
// step.  Rows without a target become zeros whatever their numerators are.
template <int TY>
__global__ void __launch_bounds__(256) xent_numerators_kernel(const XentRows r, uint16_t* dz, int64_t ldd, int64_t v0,
                                                              int p0) {
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = blockIdx.x * 256 + 8 * x;
  const float2* f = r.parts + (int64_t)(p0 + c / 128) * r.part_ld;
  for (int64_t i0 = (int64_t)blockIdx.y * 64; i0 < r.N; i0 += (int64_t)gridDim.y * 64)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t i = i0 + 8 * k + y;
      if (i >= r.N) break;
      Chunk<LL_F16, 8> e;
      Chunk<TY, 8> o;
      uint16_t* const p = dz + i * ldd + c;
      e.template load<false>(p, 8);
      const float g = f[i].x;
      const int32_t t = r.column[i];
#pragma unroll
      for (int j = 0; j < 8; ++j) o.put(j, t < 0 ? 0.f : e.get(j) * g);
      const int64_t at = t - v0 - c;  // the numerator's rounding would be lost against the 1
      if (t >= 0 && at >= 0 && at < 8) {
        const float d = r.zt[i] - r.lse[i];
        const float own = (__expf(d > 0.f ? 0.f : d) - 1.f) * r.coef[i];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at == j) o.put(j, own);
      }
      o.template store<false>(p, 8);
    }
}

hipError_t launch_xent_numerators(const XentRows& r, void* dz, int64_t ldd, int64_t v0, int cols, int p0, int type,
                                  hipStream_t s) {
  const dim3 grid((unsigned)((cols + 255) / 256), (unsigned)std::min<int64_t>((r.N + 63) / 64, 1 << 15));  // y ends at 2^16
  if (type == LL_BF16)
    hipLaunchKernelGGL((xent_numerators_kernel<LL_BF16>), grid, dim3(256), 0, s, r, (uint16_t*)dz, ldd, v0, p0);
  else
    hipLaunchKernelGGL((xent_numerators_kernel<LL_F16>), grid, dim3(256), 0, s, r, (uint16_t*)dz, ldd, v0, p0);
  return hipGetLastError();
}

// Four columns per thread.  dz is rounded to the 16-bit type of the products
// that follow (the matrix instruction takes no wider operand): relative to
// each element, half a step of the type, as any 16-bit gradient is.
template <int TY>
__global__ void __launch_bounds__(256) xent_dz_kernel(const XentRows r, const float* z, int64_t ldz, int64_t v0,
                                                      int cols, uint16_t* dz, int64_t ldd, int splits) {
  const int64_t items = r.N * splits;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t i = it / splits;
    int lo, hi;
    split_range((int)ldd, splits, (int)(it % splits), lo, hi);
    const float coef = r.coef[i], lse = r.lse[i];
    const bool live = r.column[i] >= 0;
    const int64_t t = r.column[i] - v0;
    for (int c = lo + 4 * threadIdx.x; c < hi; c += 1024) {
      uint16_t o[4] = {};
      if (live && c < cols) {
        const float4 q = *(const float4*)(z + i * ldz + c);
        const float v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < cols) o[e] = Elem<TY>::put((__expf(v[e] - lse) - (c + e == t ? 1.f : 0.f)) * coef);
      }
      uint2 w;
      __builtin_memcpy(&w, o, 8);
      *(uint2*)(dz + i * ldd + c) = w;
    }
  }
}

hipError_t launch_xent_dz(const XentRows& r, const float* z, int64_t ldz, int64_t v0, int cols, void* dz, int64_t ldd,
                          int type, int cus, hipStream_t s) {
  const int splits = (int)std::max<int64_t>(1, std::min<int64_t>((ldd + 1023) / 1024, 8ll * cus / r.N));
  const dim3 grid((unsigned)std::min<int64_t>(r.N * splits, 1 << 20));
  if (type == LL_BF16)
    hipLaunchKernelGGL((xent_dz_kernel<LL_BF16>), grid, dim3(256), 0, s, r, z, ldz, v0, cols, (uint16_t*)dz, ldd,
                       splits);
  else
    hipLaunchKernelGGL((xent_dz_kernel<LL_F16>), grid, dim3(256), 0, s, r, z, ldz, v0, cols, (uint16_t*)dz, ldd,
                       splits);
  return hipGetLastError();
}

template <int TY>
__global__ void __launch_bounds__(256) xent_finish_kernel(const float* a, const float* b, const float* scale,
                                                          int64_t rows, int64_t cols, int64_t lda, void* out,
                                                          int64_t ldo) {
  const float f = scale ? *scale : 1.f;
  for (int64_t i = blockIdx.x; i < rows; i += gridDim.x)
    for (int64_t c = threadIdx.x; c < cols; c += 256) {
      float v = a[i * lda + c];
      if (b) v += b[i * lda + c];
      ((typename Elem<TY>::raw*)out)[i * ldo + c] = Elem<TY>::put(v * f);
    }
}

hipError_t launch_xent_finish(const float* a, const float* b, const float* scale, int64_t rows, int64_t cols,
                              int64_t lda, void* out, int64_t ldo, int type, int cus, hipStream_t s) {
  if (rows == 0 || cols == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>(rows, 64ll * cus));
#define LL_FINISH(TY) \
  hipLaunchKernelGGL((xent_finish_kernel<TY>), grid, dim3(256), 0, s, a, b, scale, rows, cols, lda, out, ldo)
  if (type == LL_BF16) LL_FINISH(LL_BF16);
  else if (type == LL_F16) LL_FINISH(LL_F16);
  else LL_FINISH(LL_F32);
#undef LL_FINISH
  return hipGetLastError();
}

}  // namespace ll
