// The 8-bit product for few rows of A (serving: one token, or a small batch of
// sequences), bound by the bytes of B.
//
// A workgroup takes 16 NF rows of B (columns of C) and all rows of A; its waves
// deal the blocks of 128 k among them, 128 consecutive bytes of a row each, so
// that neighbouring waves read neighbouring pieces.  Rows go from memory to
// registers: no byte of B is used twice, and A's few rows come from the caches.
// A wave keeps two blocks' loads in flight (of four, half as many workgroups fit a CU:
// 2 x 8704 x 7168, 16x32, 18.7 and 13.6 us).  The waves' sums are joined
// in LDS in wave order; where N alone leaves the chip empty K is also split over
// workgroups, whose partials a second kernel joins.
#include "gemm8_common.hpp"

namespace ll {

namespace {

constexpr int kFewWaves = 8;

// A lane's share of 16 rows of 128 bytes.  LINES: 16 bytes (l % 8) of row l / 8 and of
// row 8 + l / 8, so that eight lanes ask for a line together, and an exchange in LDS
// hands them to the lanes that the matrix unit takes them from.  Else what the lane
// itself needs, pieces l / 16 and l / 16 + 4 of row l % 16: sixteen lanes then ask for
// sixteen rows, in the same banks of the cache where rows are whole lines.  Where
// they are not LINES would fetch most lines twice.  (LINES and not, whole lines: 64 x
// 4096 x 4096 7.5 and 11.8 us, 64 x 8192 x 8192 15.8 and 24.6, 16 x 8192 x 8192 11.6 and 16.6, 2 x
// 8704 x 7168 12.2 and 14.8, 1 x 5120 x 5120 7.1 and 8.2, 1 x 8192 x 8192 12.5 and 12.4, 1 x 28672 x
// 8192 39.2 and 39.4, 1 x 8192 x 28672 41.4 and 41.0; rows of 4112 or 8208 bytes: 64 x 4096 10.0
// and 8.8, 1 x 28672 46 and 41.)
struct Piece8 {
  i32x4 lo, hi;
};

// The 16 bytes of piece `piece` at p + at, of a row's block that has `left` more bytes;
// what lies past them is zeros.  Without branches (a piece past the end is read as
// piece 0, which is there), so that the words are no merge of two branches' values.
__device__ __forceinline__ i32x4 load_masked(const uint8_t* p, uint32_t at, int piece, int left) {
  const int n = left - (piece << 4);
  i32x4 v = *(const i32x4*)(p + (n > 0 ? at : at - (piece << 4)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int have = min(max(n - 4 * i, 0), 4);
    v[i] &= have == 4 ? -1 : (1 << (8 * have)) - 1;
  }
  return v;
}

template <int MF, int NF, bool E5M2, bool ROWS, bool EXACT, bool LINES>
__global__ void __launch_bounds__(kFewWaves * 64, 2) gemm8_few_kernel(const Gemm8Args p) {
  typedef Block8<E5M2, EXACT> Block;
  constexpr int STAGE = LINES ? (MF + NF) * 2048 : 0;  // of a wave
  constexpr int RED = kFewWaves * MF * NF * 1024;
  __shared__ __align__(16) char lds[kFewWaves * STAGE > RED ? kFewWaves * STAGE : RED];
  f32x4(*const red)[MF * NF][64] = (f32x4(*)[MF * NF][64])lds;
  const int lane = threadIdx.x & 63, row16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x / p.tiles_n, n0 = (blockIdx.x - split * p.tiles_n) * (16 * NF);
  const int kb0 = split * p.per_split, kb1 = min(p.blocks, kb0 + p.per_split);

  // rows past the last stand for the last: read, and not stored
  const uint8_t* const b0 = p.b + (int64_t)n0 * p.ldb;
  uint32_t brow[NF][2], arow[MF][2];
  int piece[2];  // of the 128 bytes
  const float* sarow[MF];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    piece[h] = LINES ? lane & 7 : g + 4 * h;
    const int r = LINES ? 8 * h + (lane >> 3) : row16;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int n = LINES ? 16 * f + r : (r >> 2) * 4 * NF + 4 * f + (r & 3);
      brow[f][h] = (uint32_t)min(p.N - 1 - n0, n) * (uint32_t)p.ldb + (piece[h] << 4);
    }
#pragma unroll
    for (int i = 0; i < MF; ++i)
      arow[i][h] = (uint32_t)min(p.M - 1, 16 * i + r) * (uint32_t)p.lda + (piece[h] << 4);
  }
#pragma unroll
  for (int i = 0; i < MF; ++i) sarow[i] = p.sa + (int64_t)min(p.M - 1, 16 * i + row16) * p.sam;
  // A wave's exchange goes through its own part of LDS.
  char* const mine = lds + wave * STAGE;
  const int put_c = lane & 7;
  auto exchange = [&](const Piece8* x, const Piece8* w, i32x8* xf, i32x8* wf) {
    if constexpr (!LINES) {
#pragma unroll
      for (int i = 0; i < MF; ++i) xf[i] = frag8(x[i].lo, x[i].hi);
#pragma unroll
      for (int f = 0; f < NF; ++f) wf[f] = frag8(w[f].lo, w[f].hi);
      return;
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int r = lane >> 3;
      *(i32x4*)(mine + i * 2048 + r * 128 + ((put_c ^ swz8_a(r)) << 4)) = x[i].lo;
      *(i32x4*)(mine + i * 2048 + (r + 8) * 128 + ((put_c ^ swz8_a(r + 8)) << 4)) = x[i].hi;
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int r = 16 * f + (lane >> 3);
      *(i32x4*)(mine + MF * 2048 + r * 128 + ((put_c ^ swz8_b<NF>(r)) << 4)) = w[f].lo;
      *(i32x4*)(mine + MF * 2048 + (r + 8) * 128 + ((put_c ^ swz8_b<NF>(r + 8)) << 4)) = w[f].hi;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int at = i * 2048 + row16 * 128 + ((g ^ swz8_a(row16)) << 4);
      xf[i] = frag8(*(const i32x4*)(mine + at), *(const i32x4*)(mine + (at ^ 64)));
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int r = (row16 >> 2) * 4 * NF + 4 * f + (row16 & 3), at = MF * 2048 + r * 128 + ((g ^ swz8_b<NF>(r)) << 4);
      wf[f] = frag8(*(const i32x4*)(mine + at), *(const i32x4*)(mine + (at ^ 64)));
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  f32x4 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Set {  // a block's rows and scales
    Piece8 w[NF], x[MF];
    float sa[MF];
    f32x4 sb[NF];
  };
  typedef const float __attribute__((address_space(4))) scalar_float;  // read by scalar loads
  auto scales = [&](Set& s, int kb) {
#pragma unroll
    for (int i = 0; i < MF; ++i) s.sa[i] = sarow[i][(int64_t)kb * p.sab];
    if constexpr (ROWS) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          s.sb[f][r] = p.sb[(int64_t)min(p.N - 1, n0 + 4 * NF * g + 4 * f + r) * p.sbn + (int64_t)kb * p.sbb];
    } else {
      const float v = *(scalar_float*)(p.sb + (int64_t)(n0 / kBlock8) * p.sbn + (int64_t)kb * p.sbb);
#pragma unroll
      for (int f = 0; f < NF; ++f) s.sb[f] = f32x4{v, v, v, v};
    }
  };
  // Workgroups begin at different blocks and go round, so that they do not all ask
  // for the same columns at once (1 x 28672 x 8192 41.2 -> 38.9 us, 16 x 8192 x 8192
  // 16.8 -> 13.6).  The order in which a column's blocks are added up depends on
  // the sizes alone.
  const int whole = min(kb1, p.K / kBlock8);  // blocks up to here have 128 k
  const int turn = whole > kb0 ? (blockIdx.x - split * p.tiles_n) % (whole - kb0) : 0;
  auto load = [&](Set& s, int kb) {
    const int b = kb + turn < whole ? kb + turn : kb + turn - (whole - kb0);
    const uint8_t* const bk = b0 + b * kBlock8;
    const uint8_t* const ak = p.a + b * kBlock8;
#pragma unroll
    for (int f = 0; f < NF; ++f) s.w[f] = {*(const i32x4*)(bk + brow[f][0]), *(const i32x4*)(bk + brow[f][1])};
#pragma unroll
    for (int i = 0; i < MF; ++i) s.x[i] = {*(const i32x4*)(ak + arow[i][0]), *(const i32x4*)(ak + arow[i][1])};
    scales(s, b);
    __builtin_amdgcn_sched_barrier(0);  // all in flight before the sums go on: the compiler would load where they are used
  };
  auto add = [&](const Set& s) {
    i32x8 xf[MF], wf[NF];
    exchange(s.x, s.w, xf, wf);
    typename Block::W w[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) w[f] = Block::w(wf[f]);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const typename Block::X x = Block::x(xf[i]);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const f32x4 d = Block::product(w[f], x);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][f][r] = fmaf(d[r], s.sa[i] * s.sb[f][r], acc[i][f][r]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  int kb = kb0 + wave;
  int steps = whole > kb ? (whole - kb + kFewWaves - 1) / kFewWaves : 0;  // blocks of 128 k of this wave
  if (steps > 0) {  // one block's loads ahead
    Set s0, s1;
    load(s0, kb);
#pragma unroll 1
    for (; steps > 2; steps -= 2, kb += 2 * kFewWaves) {
      load(s1, kb + kFewWaves);
      add(s0);
      load(s0, kb + 2 * kFewWaves);
      add(s1);
    }
    if (steps == 2) {
      load(s1, kb + kFewWaves);
      add(s0);
      add(s1);
    } else {
      add(s0);
    }
    kb += steps * kFewWaves;
  }
  // The short block, behind the loop.  Loaded inside it, by a branch in load(), an
  // earlier form of this kernel (16x16, 16-bit C, two blocks ahead; clang 22 of ROCm
  // 7.2.0) gave wrong sums: half of a matrix operand that the branch had made a merge
  // of two values held an address when the instruction read it.  The kernel as it is
  // now passes its tests that way too; test_every_variant with K = 3333 and 4100 finds it.
  if (kb < kb1) {
    const int k = kb * kBlock8, left = p.K - k;
    Set s;
#pragma unroll
    for (int f = 0; f < NF; ++f)
      s.w[f] = {load_masked(b0 + k, brow[f][0], piece[0], left), load_masked(b0 + k, brow[f][1], piece[1], left)};
#pragma unroll
    for (int i = 0; i < MF; ++i)
      s.x[i] = {load_masked(p.a + k, arow[i][0], piece[0], left), load_masked(p.a + k, arow[i][1], piece[1], left)};
    scales(s, kb);
    add(s);
  }

  __syncthreads();  // the sums take the place of the rows
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

template <int MF, int NF, bool EXACT, bool LINES>
hipError_t launch(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  auto kernel = a_e5m2 ? (rows ? gemm8_few_kernel<MF, NF, true, true, EXACT, LINES>
                               : gemm8_few_kernel<MF, NF, true, false, EXACT, LINES>)
                       : (rows ? gemm8_few_kernel<MF, NF, false, true, EXACT, LINES>
                               : gemm8_few_kernel<MF, NF, false, false, EXACT, LINES>);
  hipLaunchKernelGGL(kernel, dim3((unsigned)a.total), dim3(kFewWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <int MF, int NF>
hipError_t launch(const Gemm8Args& a, bool a_e5m2, bool rows, bool exact, hipStream_t s) {
  const bool lines = (((uintptr_t)a.a | (uintptr_t)a.b | (uint64_t)a.lda | (uint64_t)a.ldb) & 127) == 0;
  if (exact)
    return lines ? launch<MF, NF, true, true>(a, a_e5m2, rows, s) : launch<MF, NF, true, false>(a, a_e5m2, rows, s);
  return lines ? launch<MF, NF, false, true>(a, a_e5m2, rows, s) : launch<MF, NF, false, false>(a, a_e5m2, rows, s);
}

}  // namespace

hipError_t launch_gemm8_few(const Gemm8Args& a, int kind, bool a_e5m2, bool rows, bool exact, hipStream_t s) {
  switch (kind) {
    case kG8Few16x16: return launch<1, 1>(a, a_e5m2, rows, exact, s);
    case kG8Few16x32: return launch<1, 2>(a, a_e5m2, rows, exact, s);
    case kG8Few32x16: return launch<2, 1>(a, a_e5m2, rows, exact, s);
    case kG8Few32x32: return launch<2, 2>(a, a_e5m2, rows, exact, s);
    case kG8Few64x16: return launch<4, 1>(a, a_e5m2, rows, exact, s);
    default: return launch<4, 2>(a, a_e5m2, rows, exact, s);
  }
}

}  // namespace ll
