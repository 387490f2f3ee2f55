// The 8-bit product for few rows of A (serving: one token, or a small batch of
// sequences), bound by the bytes of B.
//
// A workgroup takes 16 NF rows of B (columns of C) and all rows of A; its waves
// deal the blocks of 128 k among them, 128 consecutive bytes of a row each, so
// that neighbouring waves read neighbouring pieces.  Fragments go from memory to
// registers: no byte of B is used twice, and A's few rows come from the caches.
// A wave keeps the loads of several blocks in flight.  The waves' sums are joined
// in LDS in wave order; where N alone leaves the chip empty K is also split over
// workgroups, whose partials a second kernel joins.
#include "gemm8_common.hpp"

namespace ll {

namespace {

constexpr int kFewWaves = 8;

// 32 bytes of row `r` (16 at k, 16 at k + 64), in two halves.
struct Piece8 {
  i32x4 lo, hi;
};

__device__ __forceinline__ Piece8 load_piece(const uint8_t* row, int k) {
  return {*(const i32x4*)(row + k), *(const i32x4*)(row + k + 64)};
}

// The 16 bytes from k on; those at K and beyond are zeros.
__device__ __forceinline__ i32x4 load_masked(const uint8_t* row, int k, int K) {
  i32x4 v = {0, 0, 0, 0};
  if (k >= K) return v;
  v = *(const i32x4*)(row + k);
  const int n = K - k;  // bytes there are
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int have = n - 4 * i;
    if (have <= 0) v[i] = 0;
    else if (have < 4) v[i] &= (int)((1u << (8 * have)) - 1u);
  }
  return v;
}

template <int MF, int NF, int U, bool E5M2, bool ROWS, bool EXACT>
__global__ void __launch_bounds__(kFewWaves * 64) gemm8_few_kernel(const Gemm8Args p) {
  typedef Block8<E5M2, EXACT> Block;
  __shared__ f32x4 red[kFewWaves][MF * NF][64];
  const int lane = threadIdx.x & 63, row16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x / p.tiles_n, n0 = (blockIdx.x - split * p.tiles_n) * (16 * NF);
  const int kb0 = split * p.per_split, kb1 = min(p.blocks, kb0 + p.per_split);

  // rows past the last stand for the last: read, and not stored
  const uint8_t* brow[NF];
  const uint8_t* arow[MF];
  const float* sarow[MF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
    brow[f] = p.b + (int64_t)min(p.N - 1, n0 + (row16 >> 2) * 4 * NF + 4 * f + (row16 & 3)) * p.ldb;
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int m = min(p.M - 1, 16 * i + row16);
    arow[i] = p.a + (int64_t)m * p.lda;
    sarow[i] = p.sa + (int64_t)m * p.sam;
  }
  f32x4 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto scale_b = [&](int kb, f32x4 (&sb)[NF]) {
    if constexpr (ROWS) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          sb[f][r] = p.sb[(int64_t)min(p.N - 1, n0 + 4 * NF * g + 4 * f + r) * p.sbn + (int64_t)kb * p.sbb];
    } else {
      const float s = p.sb[(int64_t)(n0 / kBlock8) * p.sbn + (int64_t)kb * p.sbb];
#pragma unroll
      for (int f = 0; f < NF; ++f) sb[f] = f32x4{s, s, s, s};
    }
  };
  auto add = [&](const Piece8 (&w)[NF], const Piece8& x, float sa, const f32x4 (&sb)[NF], int i) {
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const f32x4 d = Block::product(Block::w(frag8(w[f].lo, w[f].hi)), Block::x(frag8(x.lo, x.hi)));
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][f][r] = fmaf(d[r], sa * sb[f][r], acc[i][f][r]);
    }
  };

  const int whole = min(kb1, p.K / kBlock8);  // blocks up to here have 128 k
  int kb = kb0 + wave;
  for (; kb + (U - 1) * kFewWaves < whole; kb += U * kFewWaves) {
    Piece8 w[U][NF], x[U][MF];
    float sa[U][MF];
    f32x4 sb[U][NF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = kb + u * kFewWaves, k = b * kBlock8 + 16 * g;
#pragma unroll
      for (int f = 0; f < NF; ++f) w[u][f] = load_piece(brow[f], k);
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        x[u][i] = load_piece(arow[i], k);
        sa[u][i] = sarow[i][(int64_t)b * p.sab];
      }
      scale_b(b, sb[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MF; ++i) add(w[u], x[u][i], sa[u][i], sb[u], i);
  }
  for (; kb < kb1; kb += kFewWaves) {
    const int k = kb * kBlock8 + 16 * g;
    Piece8 w[NF];
    f32x4 sb[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) w[f] = {load_masked(brow[f], k, p.K), load_masked(brow[f], k + 64, p.K)};
    scale_b(kb, sb);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const Piece8 x = {load_masked(arow[i], k, p.K), load_masked(arow[i], k + 64, p.K)};
      add(w, x, sarow[i][(int64_t)kb * p.sab], sb, i);
    }
  }

#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int f = 0; f < NF; ++f) red[wave][i * NF + f][lane] = acc[i][f];
  __syncthreads();
  if (wave >= MF) return;
  float v[4 * NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    f32x4 s = red[0][wave * NF + f][lane];
#pragma unroll
    for (int k = 1; k < kFewWaves; ++k) s += red[k][wave * NF + f][lane];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[4 * f + r] = s[r];
  }
  store_c8<4 * NF>(p, split, 16 * wave + row16, n0 + 4 * NF * g, v);
}

template <int MF, int NF, int U, bool EXACT>
hipError_t launch(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  auto kernel =
      a_e5m2 ? (rows ? gemm8_few_kernel<MF, NF, U, true, true, EXACT> : gemm8_few_kernel<MF, NF, U, true, false, EXACT>)
             : (rows ? gemm8_few_kernel<MF, NF, U, false, true, EXACT>
                     : gemm8_few_kernel<MF, NF, U, false, false, EXACT>);
  hipLaunchKernelGGL(kernel, dim3((unsigned)a.total), dim3(kFewWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <int MF, int NF, int U>
hipError_t launch(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  return a.c_type == LL_F32 ? launch<MF, NF, U, true>(a, a_e5m2, rows, s)
                            : launch<MF, NF, U, false>(a, a_e5m2, rows, s);
}

}  // namespace

hipError_t launch_gemm8_few(const Gemm8Args& a, int kind, bool a_e5m2, bool rows, hipStream_t s) {
  switch (kind) {
    case kG8Few16: return launch<1, 1, 4>(a, a_e5m2, rows, s);
    case kG8Few32: return launch<2, 1, 2>(a, a_e5m2, rows, s);
    default: return launch<4, 2, 1>(a, a_e5m2, rows, s);
  }
}

}  // namespace ll
