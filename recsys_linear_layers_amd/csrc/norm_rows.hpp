// Rows of the norms (layer norm, root-mean-square norm) in registers: a row's
// columns and its parameters as stored words, and sums over its lanes.
#pragma once

#include "ops_common.hpp"

namespace ll {

// Parameter columns [d, d + VEC) as fp32, stored as TY or (param_f32) as fp32; n of them exist.
template <int TY, int VEC, bool TAIL>
__device__ __forceinline__ void load_param(const void* p, int param_f32, int d, int n, float dflt, float (&v)[VEC]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = dflt;
  } else if (TY == LL_F32 || param_f32) {
    Chunk<LL_F32, VEC> c;
    c.template load<TAIL>((const uint32_t*)p + d, n);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = c.get(i);
  } else {
    Chunk<TY, VEC> c;
    c.template load<TAIL>((const typename Elem<TY>::raw*)p + d, n);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = c.get(i);
  }
}

// The parameter columns of a lane, kept over its rows: as stored where that is
// x's own type, else (REG false: fp32 beside 16-bit rows, twice the registers)
// read again for each row, from L2 (16384 x 8192 bf16 rows, parameters bf16 / fp32:
// forward 88 / 89 us, backward 172 / 184).
template <int TY, int VEC, int NCH, bool TAIL, bool REG>
struct Params {
  Chunk<TY, VEC> v[REG ? NCH : 1];
  const void* p;
  float dflt;
  __device__ __forceinline__ void init(const void* p_, float dflt_, int d0, int step, int D) {
    p = p_;
    dflt = dflt_;
    if constexpr (REG) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int d = d0 + k * step;
        if (p && d < D) v[k].template load<TAIL>((const typename Elem<TY>::raw*)p + d, D - d);
        else
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[k].put(i, dflt);
      }
    }
  }
  __device__ __forceinline__ void get(int k, int d, int n, float (&out)[VEC]) {
    if constexpr (REG) {
      v[k].keep_packed();
#pragma unroll
      for (int i = 0; i < VEC; ++i) out[i] = v[k].get(i);
    } else {
      load_param<TY, VEC, TAIL>(p, 1, d, n, dflt, out);
    }
  }
};

// Sum over the TPR lanes of one row (64: one wave; more: the row's waves,
// through red, two floats per wave of the workgroup).  One barrier: calls in a
// row alternate between two areas, so that a slow wave may still read the last.
template <int TPR, int WAVES>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* red) {
  a = lanes_sum<64>(a);
  b = lanes_sum<64>(b);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      red[2 * wave] = a;
      red[2 * wave + 1] = b;
    }
    __syncthreads();
    const int w0 = wave / W * W;
    a = 0.f;
    b = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      a += red[2 * (w0 + w)];
      b += red[2 * (w0 + w) + 1];
    }
  }
}

// The same for one sum.
template <int TPR, int WAVES>
__device__ __forceinline__ void row_sum(float& a, float* red) {
  a = lanes_sum<64>(a);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = a;
    __syncthreads();
    const int w0 = wave / W * W;
    a = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) a += red[w0 + w];
  }
}

// One row of a lane's columns: NCH chunks of VEC, TPR chunks apart.  Lanes past
// the row's end and rows past the last hold zeros.
template <int TY, int VEC, int TPR, int NCH, bool TAIL, bool NT = false>
struct RowCols {
  Chunk<TY, VEC> v[NCH];
  __device__ __forceinline__ void load(const void* base, int64_t ld, int64_t r, bool live, int x, int D) {
    const typename Elem<TY>::raw* row = (const typename Elem<TY>::raw*)base + (live ? r : 0) * ld;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int d = (x + k * TPR) * VEC;
      if (live && d < D) v[k].template load<TAIL, NT>(row + d, D - d);
      else v[k].clear();
    }
  }
  // Columns past the row's end hold its first value instead.
  __device__ __forceinline__ void repeat_first(const void* base, int64_t ld, int64_t r, int x, int D) {
    const typename Elem<TY>::raw first = ((const typename Elem<TY>::raw*)base)[r * ld];
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if ((x + k * TPR) * VEC + i >= D) v[k].put_raw(i, first);
  }
};

// Workgroups of `threads` of a kernel that a CU holds at once.
inline int per_cu(const void* kernel, int threads) {
  int n = 0;
  if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != hipSuccess || n < 1) n = 1;
  return n;
}

// One element of a row, or of a parameter.
template <int TY>
__device__ __forceinline__ float elem_at(const void* p, int64_t i) {
  return Elem<TY>::get(((const typename Elem<TY>::raw*)p)[i]);
}
template <int TY>
__device__ __forceinline__ float param_at(const void* p, int param_f32, int d, float dflt) {
  if (!p) return dflt;
  return TY == LL_F32 || param_f32 ? ((const float*)p)[d] : elem_at<TY>(p, d);
}

}  // namespace ll
