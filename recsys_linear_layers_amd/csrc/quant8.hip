// Quantises a matrix in blocks of 128 to 8 bits: as it lies, transposed, or both.
//
// HBM bound (2 bytes read and 1 or 2 written per 16-bit value), so x is read
// once for both forms: a workgroup takes a 128 x 128 tile, which holds whole
// blocks of either.  A lane holds 8 rows x 8 columns in registers as stored
// words.  Next to the loads it is vector instructions that count (about five per
// value and form): maxima are formed on pairs of 16-bit magnitudes, and a block's
// scale and reciprocal once, by one lane per block, and handed out through LDS.
// The 8 bytes that 8 rows of one column make are one LDS write of the transposed
// image, which leaves in 16-byte pieces, 128 bytes of a row of qt together.
#include "quant8.hpp"

#include <algorithm>

namespace ll {

namespace {

constexpr int kThreads = 256;

// Maxima of magnitudes, of pairs of 16-bit elements or of one of 32 bits, in their
// own bit patterns (which order as the values do, infinity and NaN on top).
template <int TY>
struct Mags {
  typedef uint16_t pair __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ uint32_t of(uint32_t w) { return w & (TY == LL_F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu); }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (TY == LL_F32) return max(a, b);
    else return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(pair, a), __builtin_bit_cast(pair, b)));
  }
  // As an fp32 bit pattern: element `high` of the pair.
  static __device__ __forceinline__ uint32_t wide(uint32_t w, bool high) {
    if constexpr (TY == LL_F32) return w;
    else if constexpr (TY == LL_BF16) return high ? w & 0xFFFF0000u : w << 16;
    else return __builtin_bit_cast(uint32_t, Elem<TY>::get((uint16_t)(high ? w >> 16 : w)));
  }
  static __device__ __forceinline__ uint32_t widest(uint32_t w) {
    if constexpr (TY == LL_F32) return w;
    else return wide(max(w & 0xFFFFu, w >> 16), false);
  }
};

template <int TY, int Q, bool SQUARE, bool PLAIN, bool TRANSPOSED, bool ONCE>
__global__ void __launch_bounds__(kThreads) quant8_kernel(const Quant8Args a, int tiles_d, int64_t tiles) {
  typedef typename Elem<TY>::raw raw;
  typedef Chunk<TY, 8> C;
  typedef Mags<TY> M;
  constexpr int WORDS = sizeof(C) / 4, PER = 8 / WORDS;
  __shared__ __align__(16) uint64_t image[TRANSPOSED ? kBlock8 * 16 : 1];  // [column][8 rows each]
  uint32_t(*const part)[kBlock8] = (uint32_t(*)[kBlock8])image;            // column maxima, before the image: [8 rows each][column]
  __shared__ __align__(16) uint32_t row_max[kBlock8];
  __shared__ __align__(16) float inv_row[kBlock8], inv_col[kBlock8];
  __shared__ uint32_t one_max[4];
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    int tn = (int)(t / tiles_d), td = (int)(t - (int64_t)tn * tiles_d);
    if constexpr (!ONCE) {  // eight rows of tiles, which the eight XCDs take in turn
      const int first = tn & ~7, rows = min(8, (a.N + kBlock8 - 1) / kBlock8 - first);
      const int64_t in = t - (int64_t)first * tiles_d;
      td = (int)(in / rows);
      tn = first + (int)(in - (int64_t)td * rows);
    }
    const int n0 = tn * kBlock8 + rg * 8, d0 = td * kBlock8 + cg * 8;
    const int rows = min(8, a.N - n0), cols = a.D - d0;
    const raw* const src = (const raw*)a.x + (int64_t)n0 * a.ldx + d0;
    C v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < rows && cols > 0) v[i].template load<true, ONCE>(src + i * a.ldx, cols);
      else v[i].clear();
    }
    uint32_t rmax[8], cmax[WORDS];
#pragma unroll
    for (int w = 0; w < WORDS; ++w) cmax[w] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      rmax[i] = 0;
#pragma unroll
      for (int w = 0; w < WORDS; ++w) {
        const uint32_t m = M::of(v[i].w[w]);
        if (SQUARE || PLAIN) rmax[i] = M::larger(rmax[i], m);
        if (!SQUARE && TRANSPOSED) cmax[w] = M::larger(cmax[w], m);
      }
    }
    float ir[8], ic[8];
    if constexpr (SQUARE) {
      uint32_t m = rmax[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) m = M::larger(m, rmax[i]);
      m = lanes_max<32>(M::widest(m));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      if ((threadIdx.x & 63) == 0) one_max[wave] = m;
      __syncthreads();
      const Scale8 s = scale8<Q>(max(max(one_max[0], one_max[1]), max(one_max[2], one_max[3])));
      if (threadIdx.x == 0) {
        if (PLAIN) a.scale[(int64_t)tn * a.sn + (int64_t)td * a.sb] = s.scale;
        if (TRANSPOSED) a.scale_t[(int64_t)td * a.tn + (int64_t)tn * a.tb] = s.scale;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ir[i] = ic[i] = s.inv;
    } else {
      if constexpr (PLAIN) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t m = lanes_max<16>(M::widest(rmax[i]));
          if (cg == i) row_max[rg * 8 + i] = m;
        }
      }
      if constexpr (TRANSPOSED) {
#pragma unroll
        for (int w = 0; w < WORDS; ++w)
#pragma unroll
          for (int e = 0; e < PER; ++e) part[rg][cg * 8 + w * PER + e] = M::wide(cmax[w], e);
      }
      __syncthreads();
      const int l = threadIdx.x & (kBlock8 - 1);
      if (TRANSPOSED && threadIdx.x < kBlock8) {
        uint32_t m = part[0][l];
#pragma unroll
        for (int k = 1; k < 16; ++k) m = max(m, part[k][l]);
        const Scale8 s = scale8<Q>(m);
        inv_col[l] = s.inv;
        const int d = td * kBlock8 + l;
        if (d < a.D) a.scale_t[(int64_t)d * a.tn + (int64_t)tn * a.tb] = s.scale;
      }
      if (PLAIN && threadIdx.x >= kBlock8) {
        const Scale8 s = scale8<Q>(row_max[l]);
        inv_row[l] = s.inv;
        const int n = tn * kBlock8 + l;
        if (n < a.N) a.scale[(int64_t)n * a.sn + (int64_t)td * a.sb] = s.scale;
      }
      __syncthreads();
      if constexpr (PLAIN) __builtin_memcpy(ir, &inv_row[rg * 8], sizeof ir);
      if constexpr (TRANSPOSED) __builtin_memcpy(ic, &inv_col[cg * 8], sizeof ic);
    }
    if constexpr (PLAIN) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v[i].get(j) * ir[i];
        const uint32_t w[2] = {pack8<Q>(f[0], f[1], f[2], f[3]), pack8<Q>(f[4], f[5], f[6], f[7])};
        if (i < rows && cols > 0) store8<true>(a.q + (int64_t)(n0 + i) * a.ldq + d0, w, cols);
      }
    }
    if constexpr (TRANSPOSED) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v[i].get(j) * ic[j];
        const uint64_t lo = pack8<Q>(f[0], f[1], f[2], f[3]), hi = pack8<Q>(f[4], f[5], f[6], f[7]);
        // the groups of 8 rows of a column are permuted, so that the 16 columns one write covers spread over the banks
        image[(cg * 8 + j) * 16 + (rg ^ ((cg & 3) << 2))] = lo | hi << 32;
      }
      __syncthreads();
      const int left = a.N - tn * kBlock8;  // rows of x from this tile on: bytes of a row of qt
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = (threadIdx.x >> 3) + 32 * k, p = threadIdx.x & 7, d = td * kBlock8 + c;
        uint32_t w[4];
        __builtin_memcpy(w, &image[c * 16 + ((2 * p) ^ (((c >> 3) & 3) << 2))], 16);
        if (d < a.D && 16 * p < left)
          store8<true>(a.qt + (int64_t)d * a.ldqt + (int64_t)tn * kBlock8 + 16 * p, w, left - 16 * p);
      }
    }
    __syncthreads();  // LDS is free for the next tile
  }
}

template <int TY, int Q, bool SQUARE, bool ONCE>
auto pick(const Quant8Args& a) {
  return a.q ? (a.qt ? quant8_kernel<TY, Q, SQUARE, true, true, ONCE> : quant8_kernel<TY, Q, SQUARE, true, false, ONCE>)
             : quant8_kernel<TY, Q, SQUARE, false, true, ONCE>;
}

template <int TY, int Q, bool SQUARE>
hipError_t launch(const Quant8Args& a, hipStream_t s) {
  const int tiles_d = (a.D + kBlock8 - 1) / kBlock8;
  const int64_t tiles = (int64_t)((a.N + kBlock8 - 1) / kBlock8) * tiles_d;
  // Each value is read once (non-temporal); but pieces that straddle lines, and
  // fp32's two per lane, ask for a line twice and want it kept (non-temporal,
  // 16384 x 8192 bf16: 75 -> 70 us, 8191 x 5003 fp16 in rows of 5006: 30 -> 43,
  // 8192 x 8192 fp32 80 -> 83).  Such tiles are also dealt out so that those beside
  // each other, which share lines, run on one XCD and find them in its L2 (8191 x 5003
  // fp16 in rows of 5006, both forms 40.7 -> 33.8, as it lies 30.3 -> 24.3; whole pieces 8192 x 4096 transposed 20.5 -> 21.4).
  auto kernel = pick<TY, Q, SQUARE, false>(a);
  if constexpr (TY != LL_F32) {
    if (a.aligned) kernel = pick<TY, Q, SQUARE, true>(a);
  }
  const int64_t blocks = std::min<int64_t>(tiles, 1 << 22);  // a grid of 2^32 threads or more is not supported
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a, tiles_d, tiles);
  return hipGetLastError();
}

template <int TY>
hipError_t launch_t(const Quant8Args& a, int q_type, int block, hipStream_t s) {
  if (q_type == LL_E4M3)
    return block == 1 ? launch<TY, LL_E4M3, false>(a, s) : launch<TY, LL_E4M3, true>(a, s);
  return block == 1 ? launch<TY, LL_E5M2, false>(a, s) : launch<TY, LL_E5M2, true>(a, s);
}

}  // namespace

hipError_t launch_quant8(const Quant8Args& a, int type, int q_type, int block, hipStream_t s) {
  switch (type) {
    case LL_BF16: return launch_t<LL_BF16>(a, q_type, block, s);
    case LL_F16: return launch_t<LL_F16>(a, q_type, block, s);
    case LL_F32: return launch_t<LL_F32>(a, q_type, block, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ll
