// Quantises a matrix in blocks of 128 to 8 bits: as it lies, transposed, or both.
//
// HBM bound (2 bytes read and 1 or 2 written per 16-bit value), so x is read
// once for both forms: a workgroup takes a 128 x 128 tile, which holds whole
// blocks of either.  A lane holds 8 rows x 8 columns in registers as stored
// words.  A row of the tile lies in 16 neighbouring lanes, a column in four
// lanes of each wave and the four waves: the row maxima are formed by lane
// exchanges, the column maxima by those and one trip through LDS.  The 8 bytes
// that 8 rows of one column make are one LDS write of the transposed image,
// which leaves in 16-byte pieces, 128 bytes of a row of qt together.
#include "quant8.hpp"

#include <algorithm>

namespace ll {

namespace {

constexpr int kThreads = 256;

template <int TY, int Q, bool SQUARE, bool PLAIN, bool TRANSPOSED>
__global__ void __launch_bounds__(kThreads) quant8_kernel(const Quant8Args a, int tiles_d, int64_t tiles) {
  typedef typename Elem<TY>::raw raw;
  typedef Chunk<TY, 8> C;
  __shared__ uint32_t col_max[4][kBlock8];
  __shared__ uint32_t one_max[4];
  __shared__ uint64_t image[TRANSPOSED ? kBlock8 * 16 : 1];  // [column][8 rows each]
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int tn = (int)(t / tiles_d), td = (int)(t - (int64_t)tn * tiles_d);
    const int n0 = tn * kBlock8 + rg * 8, d0 = td * kBlock8 + cg * 8;
    const int rows = min(8, a.N - n0), cols = a.D - d0;
    const raw* const src = (const raw*)a.x + (int64_t)n0 * a.ldx + d0;
    C v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < rows && cols > 0) v[i].template load<true>(src + i * a.ldx, cols);
      else v[i].clear();
    }
    uint32_t rmax[8], cmax[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rmax[i] = cmax[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t m = magnitude(v[i].get(j));
        if (SQUARE || PLAIN) rmax[i] = max(rmax[i], m);
        if (!SQUARE && TRANSPOSED) cmax[j] = max(cmax[j], m);
      }
    Scale8 one;
    if constexpr (SQUARE) {
      uint32_t m = rmax[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) m = max(m, rmax[i]);
      m = lanes_max<64>(m);
      if ((threadIdx.x & 63) == 0) one_max[wave] = m;
      __syncthreads();
      one = scale8<Q>(max(max(one_max[0], one_max[1]), max(one_max[2], one_max[3])));
      if (threadIdx.x == 0) {
        if (PLAIN) a.scale[(int64_t)tn * a.sn + (int64_t)td * a.sb] = one.scale;
        if (TRANSPOSED) a.scale_t[(int64_t)td * a.tn + (int64_t)tn * a.tb] = one.scale;
      }
    } else if constexpr (TRANSPOSED) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cmax[j] = max(cmax[j], (uint32_t)__shfl_xor((int)cmax[j], 16, 64));
        cmax[j] = max(cmax[j], (uint32_t)__shfl_xor((int)cmax[j], 32, 64));
      }
      if ((threadIdx.x & 63) < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) col_max[wave][cg * 8 + j] = cmax[j];
      }
      __syncthreads();
    }
    if constexpr (PLAIN) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        Scale8 s = one;
        if constexpr (!SQUARE) {
          s = scale8<Q>(lanes_max<16>(rmax[i]));
          if (cg == 0 && i < rows) a.scale[(int64_t)(n0 + i) * a.sn + (int64_t)td * a.sb] = s.scale;
        }
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v[i].get(j) * s.inv;
        const uint32_t w[2] = {pack8<Q>(f[0], f[1], f[2], f[3]), pack8<Q>(f[4], f[5], f[6], f[7])};
        if (i < rows && cols > 0) store8<true>(a.q + (int64_t)(n0 + i) * a.ldq + d0, w, cols);
      }
    }
    if constexpr (TRANSPOSED) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        Scale8 s = one;
        if constexpr (!SQUARE) {
          const int c = cg * 8 + j;
          s = scale8<Q>(max(max(col_max[0][c], col_max[1][c]), max(col_max[2][c], col_max[3][c])));
          if (rg == 0 && j < cols) a.scale_t[(int64_t)(d0 + j) * a.tn + (int64_t)tn * a.tb] = s.scale;
        }
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v[i].get(j) * s.inv;
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

template <int TY, int Q, bool SQUARE>
hipError_t launch(const Quant8Args& a, int cus, hipStream_t s) {
  const int tiles_d = (a.D + kBlock8 - 1) / kBlock8;
  const int64_t tiles = (int64_t)((a.N + kBlock8 - 1) / kBlock8) * tiles_d;
  auto kernel = a.q ? (a.qt ? quant8_kernel<TY, Q, SQUARE, true, true> : quant8_kernel<TY, Q, SQUARE, true, false>)
                    : quant8_kernel<TY, Q, SQUARE, false, true>;
  const int64_t blocks = std::min<int64_t>(tiles, 1 << 22);  // a grid of 2^32 threads or more is not supported
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a, tiles_d, tiles);
  return hipGetLastError();
}

template <int TY>
hipError_t launch_t(const Quant8Args& a, int q_type, int block, int cus, hipStream_t s) {
  if (q_type == LL_E4M3)
    return block == 1 ? launch<TY, LL_E4M3, false>(a, cus, s) : launch<TY, LL_E4M3, true>(a, cus, s);
  return block == 1 ? launch<TY, LL_E5M2, false>(a, cus, s) : launch<TY, LL_E5M2, true>(a, cus, s);
}

}  // namespace

hipError_t launch_quant8(const Quant8Args& a, int type, int q_type, int block, int cus, hipStream_t s) {
  switch (type) {
    case LL_BF16: return launch_t<LL_BF16>(a, q_type, block, cus, s);
    case LL_F16: return launch_t<LL_F16>(a, q_type, block, cus, s);
    case LL_F32: return launch_t<LL_F32>(a, q_type, block, cus, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ll
