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
__global__ void __launch_bounds__(kFewWaves * 64, 2) gemm8_few_kernel(const Gemm8Args p) {
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

  // U blocks' fragments and scales
  struct Set {
    Piece8 w[U][NF], x[U][MF];
    float sa[U][MF];
    f32x4 sb[U][NF];
  };
  typedef const float __attribute__((address_space(4))) scalar_float;  // read by scalar loads
  auto scales = [&](Set& s, int u, int kb) {
#pragma unroll
    for (int i = 0; i < MF; ++i) s.sa[u][i] = sarow[i][(int64_t)kb * p.sab];
    if constexpr (ROWS) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          s.sb[u][f][r] = p.sb[(int64_t)min(p.N - 1, n0 + 4 * NF * g + 4 * f + r) * p.sbn + (int64_t)kb * p.sbb];
    } else {
      const float v = *(scalar_float*)(p.sb + (int64_t)(n0 / kBlock8) * p.sbn + (int64_t)kb * p.sbb);
#pragma unroll
      for (int f = 0; f < NF; ++f) s.sb[u][f] = f32x4{v, v, v, v};
    }
  };
  // Workgroups begin at different blocks and go round, so that they do not all ask
  // for the same columns at once (1 x 28672 x 8192 41.2 -> 38.9 us, 16 x 8192 x 8192
  // 16.8 -> 13.6).  The order in which a column's blocks are added up depends on
  // the sizes alone.
  const int whole = min(kb1, p.K / kBlock8);  // blocks up to here have 128 k
  const int turn = whole > kb0 ? (blockIdx.x - split * p.tiles_n) % (whole - kb0) : 0;
  auto load = [&](Set& s, int kb) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int b = kb + u * kFewWaves + turn;
      if (b >= whole) b -= whole - kb0;
      const int k = b * kBlock8 + 16 * g;
#pragma unroll
      for (int f = 0; f < NF; ++f) s.w[u][f] = load_piece(brow[f], k);
#pragma unroll
      for (int i = 0; i < MF; ++i) s.x[u][i] = load_piece(arow[i], k);
      scales(s, u, b);
    }
    __builtin_amdgcn_sched_barrier(0);  // all in flight before the sums go on: the compiler would load where they are used
  };
  auto add = [&](const Set& s, int u) {
    typename Block::W w[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) w[f] = Block::w(frag8(s.w[u][f].lo, s.w[u][f].hi));
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const typename Block::X x = Block::x(frag8(s.x[u][i].lo, s.x[u][i].hi));
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const f32x4 d = Block::product(w[f], x);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][f][r] = fmaf(d[r], s.sa[u][i] * s.sb[u][f][r], acc[i][f][r]);
      }
    }
  };

  int kb = kb0 + wave;
  constexpr int STEP = U * kFewWaves;
  // steps of U blocks that are there in full for this wave
  int steps = whole - kb - (U - 1) * kFewWaves;
  steps = steps > 0 ? (steps + STEP - 1) / STEP : 0;
  auto add_all = [&](const Set& s) {
#pragma unroll
    for (int u = 0; u < U; ++u) add(s, u);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (steps > 0) {  // one step's loads ahead
    Set s0, s1;
    load(s0, kb);
#pragma unroll 1
    for (; steps > 2; steps -= 2, kb += 2 * STEP) {
      load(s1, kb + STEP);
      add_all(s0);
      load(s0, kb + 2 * STEP);
      add_all(s1);
    }
    if (steps == 2) {
      load(s1, kb + STEP);
      add_all(s0);
      add_all(s1);
    } else {
      add_all(s0);
    }
    kb += steps * STEP;
  }
  for (; kb < kb1; kb += kFewWaves) {  // the rest, and the short block
    int b = kb;
    if (b < whole) b = b + turn < whole ? b + turn : b + turn - (whole - kb0);
    const int k = b * kBlock8 + 16 * g;
    Set s;
#pragma unroll
    for (int f = 0; f < NF; ++f) s.w[0][f] = {load_masked(brow[f], k, p.K), load_masked(brow[f], k + 64, p.K)};
#pragma unroll
    for (int i = 0; i < MF; ++i) s.x[0][i] = {load_masked(arow[i], k, p.K), load_masked(arow[i], k + 64, p.K)};
    scales(s, 0, b);
    add(s, 0);
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
    case kG8Few16x16: return launch<1, 1, 2>(a, a_e5m2, rows, s);
    case kG8Few16x32: return launch<1, 2, 2>(a, a_e5m2, rows, s);
    case kG8Few32x16: return launch<2, 1, 2>(a, a_e5m2, rows, s);
    case kG8Few32x32: return launch<2, 2, 1>(a, a_e5m2, rows, s);
    case kG8Few64x16: return launch<4, 1, 1>(a, a_e5m2, rows, s);
    default: return launch<4, 2, 1>(a, a_e5m2, rows, s);
  }
}

}  // namespace ll
