// Tiles of the 8-bit product C = sum over blocks b of sa[i][b] sb[j][b] (A B^T)_b.
//
// The matrix unit forms a block's sum over its 128 k in one 16x16x128
// instruction per 16x16 of C, from zero; four vector fmas then add the scaled
// sums to the fp32 accumulators, which therefore live in vector registers.  The
// rows of B take the instruction's first operand: a lane then holds one row of C
// (its scale of A is one register) and, with the rows of B dealt out as
// 4 FN g + 4 f + r to instruction f, lane group g and register r, 4 FN
// consecutive columns, which leave in 16-byte stores.
//
// A step is one block of 128 k: A's and B's rows of 128 bytes go straight from
// memory to LDS (1 KB per instruction), two steps deep; one barrier per step.
// The chunks of 16 bytes of a row are permuted so that the fragment reads touch
// every bank once.  Rows and k outside the matrices are given an offset out of
// the buffer's range, which reads zeros; the bytes of a last piece past K are
// cleared in LDS.
#pragma once

#include "gemm8_common.hpp"

namespace ll {

template <int BM_, int BN_, int WM_, int WN_>
struct G8Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, WAVES = WM * WN, THREADS = WAVES * 64;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, SLOT = A_BYTES + B_BYTES;
  static constexpr int QA = BM / 8 / WAVES, QB = BN / 8 / WAVES;  // 1-KB loads of a wave
  static constexpr int SLOTS = 2;
  static constexpr int SCALES = (BM + BN) * 4;  // of a step; three steps' worth, as those of one are read until its end
  static constexpr int LDS = SLOTS * SLOT + 3 * SCALES;
  static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0 && TN <= 128 && 128 % TN == 0, "tile");
};

// Chunk c of A's row r sits at c ^ swz8_a(r), of B's at c ^ swz8_b(r).  One pass
// of a 16-byte LDS read serves lanes 8p..8p+7 and 32+8p..32+8p+7: 8 rows, each at
// chunks x and x ^ 2, a row's 128 bytes being half of the banks (which half goes
// by the row's parity).  The four rows of each parity need one value from each
// of {0, 2}, {1, 3}, {4, 6}, {5, 7}.  A's eight rows follow one another; B's are
// 4 and 4, 4 FN rows apart.
__device__ __forceinline__ int swz8_a(int r) { return ((r >> 1) & 1) | (r & 4); }
template <int FN>
__device__ __forceinline__ int swz8_b(int r) {
  return ((r >> 1) & 1) | (((r / (4 * FN)) & 1) << 2);
}

template <class Cfg, bool E5M2, bool ROWS, bool EXACT>
__global__ void __launch_bounds__(Cfg::THREADS, 2) gemm8_tile_kernel(const Gemm8Args p) {
  typedef Block8<E5M2, EXACT> Block;
  __shared__ __align__(1024) char lds[Cfg::LDS];
  constexpr int FM = Cfg::FM, FN = Cfg::FN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;

  // work item -> (split, tile); the XCDs take runs of neighbouring tiles, in
  // groups of 8 tile rows, so that those in flight share panels in L2
  const int item = xcd_remap(blockIdx.x, gridDim.x);
  const int split = item / (p.tiles_m * p.tiles_n), tile = item - split * (p.tiles_m * p.tiles_n);
  const int group = tile / (8 * p.tiles_n), in_group = tile - group * 8 * p.tiles_n;
  const int height = min(8, p.tiles_m - group * 8);
  const int tm = group * 8 + in_group % height, tn = in_group / height;
  const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
  const int kb0 = split * p.per_split, kb1 = min(p.blocks, kb0 + p.per_split);

  // loads: instruction q takes rows 8q .. 8q+7 of the tile, lane l row l / 8, position l % 8
  uint32_t va[Cfg::QA], vb[Cfg::QB];
  const i32x4 ra = make_rsrc(p.a + (int64_t)m0 * p.lda, records8((int64_t)(p.M - m0 - 1) * p.lda + p.K));
  const i32x4 rb = make_rsrc(p.b + (int64_t)n0 * p.ldb, records8((int64_t)(p.N - n0 - 1) * p.ldb + p.K));
#pragma unroll
  for (int i = 0; i < Cfg::QA; ++i) {
    const int row = (wave + i * Cfg::WAVES) * 8 + (lane >> 3);
    va[i] = m0 + row < p.M ? (uint32_t)(row * (int)p.lda + (((lane & 7) ^ swz8_a(row)) << 4)) : kOOB;
  }
#pragma unroll
  for (int i = 0; i < Cfg::QB; ++i) {
    const int row = (wave + i * Cfg::WAVES) * 8 + (lane >> 3);
    vb[i] = n0 + row < p.N ? (uint32_t)(row * (int)p.ldb + (((lane & 7) ^ swz8_b<FN>(row)) << 4)) : kOOB;
  }
  // scales: a wave takes 64 rows of A's (and, with ROWS, B's)
  constexpr int SA_WAVES = Cfg::BM / 64, SB_WAVES = ROWS ? Cfg::BN / 64 : 0;
  static_assert(SA_WAVES <= Cfg::WAVES && SB_WAVES <= Cfg::WAVES, "scale loads");
  const uint32_t vsa = m0 + wave * 64 + lane < p.M ? (uint32_t)((wave * 64 + lane) * (int)p.sam) * 4u : kOOB;
  const uint32_t vsb = n0 + wave * 64 + lane < p.N ? (uint32_t)((wave * 64 + lane) * (int)p.sbn) * 4u : kOOB;
  const float* sa_base = p.sa + (int64_t)m0 * p.sam;
  const float* sb_base = ROWS ? p.sb + (int64_t)n0 * p.sbn : nullptr;

  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_u32((const char LL_LDS*)lds));
  constexpr uint32_t SC = Cfg::SLOTS * Cfg::SLOT;  // scales: per slot, A's then B's
  auto issue = [&](int kb, int slot, int sslot) {
    const uint32_t dst = lds0 + slot * Cfg::SLOT + wave * 1024;
    const int k0 = kb * 128;
    if (k0 + 128 <= p.K) {
#pragma unroll
      for (int i = 0; i < Cfg::QA; ++i) dma16s(ra, dst + i * Cfg::WAVES * 1024, va[i], (uint32_t)k0);
#pragma unroll
      for (int i = 0; i < Cfg::QB; ++i)
        dma16s(rb, dst + Cfg::A_BYTES + i * Cfg::WAVES * 1024, vb[i], (uint32_t)k0);
    } else {
      // the last, short block: pieces that start at K or beyond are zeros
#pragma unroll
      for (int i = 0; i < Cfg::QA; ++i) {
        const int row = (wave + i * Cfg::WAVES) * 8 + (lane >> 3);
        const bool in = k0 + (((lane & 7) ^ swz8_a(row)) << 4) < p.K;
        dma16s(ra, dst + i * Cfg::WAVES * 1024, in ? va[i] : kOOB, (uint32_t)k0);
      }
#pragma unroll
      for (int i = 0; i < Cfg::QB; ++i) {
        const int row = (wave + i * Cfg::WAVES) * 8 + (lane >> 3);
        const bool in = k0 + (((lane & 7) ^ swz8_b<FN>(row)) << 4) < p.K;
        dma16s(rb, dst + Cfg::A_BYTES + i * Cfg::WAVES * 1024, in ? vb[i] : kOOB, (uint32_t)k0);
      }
    }
    const uint32_t sdst = lds0 + SC + sslot * Cfg::SCALES + wave * 256;
    if (wave < SA_WAVES) dma4(make_rsrc(sa_base + (int64_t)kb * p.sab, 0x7FFFFFF0u), sdst, vsa);
    if (ROWS && wave < SB_WAVES) dma4(make_rsrc(sb_base + (int64_t)kb * p.sbb, 0x7FFFFFF0u), sdst + Cfg::BM * 4, vsb);
  };

  // fragments: lane l takes row l % 16 and chunks l / 16 and l / 16 + 4
  const int row16 = lane & 15, g = lane >> 4;
  const int arow = wm * Cfg::TM + row16;
  const int brow = wn * Cfg::TN + (row16 >> 2) * 4 * FN + (row16 & 3);
  const int a_off = arow * 128 + ((g ^ swz8_a(arow)) << 4);                            // + 2048 i
  const int b_off = Cfg::A_BYTES + brow * 128 + ((g ^ swz8_b<FN>(brow)) << 4);         // + 512 f
  const int sb_row = (n0 + wn * Cfg::TN) / 128;                                         // block row of B, unless ROWS

  const float __attribute__((address_space(4))) * sbs =
      (const float __attribute__((address_space(4)))*)(p.sb + (int64_t)min(sb_row, (p.N - 1) / 128) * p.sbn);

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int f = 0; f < FN; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Clears the bytes past K of the piece that K ends in.
  auto clear_tail = [&](int slot) {
    const int c = (p.K & 127) >> 4;
    for (int row = threadIdx.x; row < Cfg::BM + Cfg::BN; row += Cfg::THREADS) {
      const bool of_a = row < Cfg::BM;
      const int r = of_a ? row : row - Cfg::BM;
      char* q = lds + slot * Cfg::SLOT + row * 128 + ((c ^ (of_a ? swz8_a(r) : swz8_b<FN>(r))) << 4);
      for (int i = p.K & 15; i < 16; ++i) q[i] = 0;
    }
    __syncthreads();
  };
  // The rows of the slot of step kb are there, for every wave.
  auto arrive = [&](int kb, int slot) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
    if (kb * 128 + 128 > p.K && (p.K & 15)) clear_tail(slot);
  };
  auto read_x = [&](const char* st, int i) {
    return frag8(*(const i32x4*)(st + a_off + 2048 * i), *(const i32x4*)(st + (a_off ^ 64) + 2048 * i));
  };
  auto read_w = [&](const char* st, int f) {
    return frag8(*(const i32x4*)(st + b_off + 512 * f), *(const i32x4*)(st + (b_off ^ 64) + 512 * f));
  };
  const int sa_off = SC + (wm * Cfg::TM + row16) * 4;                              // + 64 i
  const int sb_off = SC + (Cfg::BM + wn * Cfg::TN + 4 * FN * g) * 4;               // + 16 f

  // A step is FM x FN products, in the order below.  A product's fmas follow LAG
  // products later, when its result is there; the fragments of A are read one
  // row of products ahead, those of the next step during the last row, after the
  // barrier that says that its rows have landed and that nobody reads this step's.
  constexpr bool FEW_SB = EXACT;
  constexpr int T = FM * FN, LAG = EXACT ? 1 : 2, ND = EXACT ? 2 : 4;
  static_assert(T % ND == 0 && LAG < ND && LAG <= FN && FM % 2 == 0, "ring of results");
  f32x4 d[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i) d[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (kb0 < kb1) {
    issue(kb0, 0, 0);
    arrive(kb0, 0);
    if (kb0 + 1 < kb1) issue(kb0 + 1, 1, 1);
    i32x8 wr[FN], xr[2];
    f32x4 sbv[FEW_SB ? 1 : FN];  // ROWS: of all f, or (EXACT, whose operands take the registers) of the last product
    typename Block::W w[FN];
    float s_last = 0.f, sa_next, sb = 0.f;
    if constexpr (!ROWS) sb = sbs[(int64_t)kb0 * p.sbb];
    xr[0] = read_x(lds, 0);
    sa_next = *(const float*)(lds + sa_off);
#pragma unroll
    for (int f = 0; f < FN; ++f) wr[f] = read_w(lds, f);
#pragma unroll
    for (int f = 0; f < (FEW_SB ? 1 : FN); ++f) sbv[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto add = [&](int t, float s) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[t / FN][t % FN][r] =
            fmaf(d[t % ND][r], ROWS ? s * sbv[FEW_SB ? 0 : t % FN][r] : s, acc[t / FN][t % FN][r]);
      asm volatile("" : "+v"(acc[t / FN][t % FN]));  // here, not where the compiler would sink them to
    };
    int s0 = 0, s1 = 1, s2 = 2;  // scale slots of this step and of the next two
    for (int kb = kb0; kb < kb1; ++kb) {
      const int slot = (kb - kb0) & 1;
      const char* st = lds + slot * Cfg::SLOT;
      const char* next = lds + (slot ^ 1) * Cfg::SLOT;
      const char* sc = lds + s0 * Cfg::SCALES;
      float sb_next = 0.f;
      if constexpr (!ROWS) sb_next = sbs[(int64_t)min(kb + 1, kb1 - 1) * p.sbb];
      float s = 0.f;
      typename Block::X x;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int i = t / FN, f = t % FN;
        if (f == 0) {
          if (i == FM - 1 && kb + 1 < kb1) {
            arrive(kb + 1, slot ^ 1);
            if (kb + 2 < kb1) issue(kb + 2, slot, s2);
          }
          x = Block::x(xr[i & 1]);
        }
        if (i == 0) w[f] = Block::w(wr[f]);
        d[t % ND] = Block::product(w[f], x);
        if (t < LAG) add(T + t - LAG, s_last);
        else add(t - LAG, s);
        if (f == LAG - 1) s = ROWS ? sa_next : sa_next * sb;  // of this row of products from here on
        if (ROWS && FEW_SB) sbv[0] = *(const f32x4*)(sc + sb_off + 16 * f);
        if (ROWS && !FEW_SB && t == LAG - 1) {
#pragma unroll
          for (int q = 0; q < FN; ++q) sbv[q] = *(const f32x4*)(sc + sb_off + 16 * q);
        }
        if (f == 0) xr[(i + 1) & 1] = i + 1 < FM ? read_x(st, i + 1) : read_x(next, 0);
        if (f == LAG)
          sa_next = *(const float*)(i + 1 < FM ? sc + sa_off + 64 * (i + 1) : lds + s1 * Cfg::SCALES + sa_off);
        if (i == FM - 1) wr[f] = read_w(next, f);
        __builtin_amdgcn_sched_barrier(0);
      }
      s_last = s;
      sb = sb_next;
      const int first = s0;
      s0 = s1, s1 = s2, s2 = first;
    }
#pragma unroll
    for (int t = T - LAG; t < T; ++t) add(t, s_last);
  }

#pragma unroll
  for (int i = 0; i < FM; ++i) {
    float v[4 * FN];
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[4 * f + r] = acc[i][f][r];
    store_c8<4 * FN>(p, split, m0 + wm * Cfg::TM + 16 * i + row16, n0 + wn * Cfg::TN + 4 * FN * g, v);
  }
}

template <class Cfg, bool EXACT>
hipError_t launch_gemm8_tile(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  auto kernel = a_e5m2 ? (rows ? gemm8_tile_kernel<Cfg, true, true, EXACT> : gemm8_tile_kernel<Cfg, true, false, EXACT>)
                       : (rows ? gemm8_tile_kernel<Cfg, false, true, EXACT>
                               : gemm8_tile_kernel<Cfg, false, false, EXACT>);
  hipLaunchKernelGGL(kernel, dim3((unsigned)a.total), dim3(Cfg::THREADS), 0, s, a);
  return hipGetLastError();
}

}  // namespace ll
