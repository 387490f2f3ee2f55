// Tiles of the 8-bit product C = sum over blocks b of sa[i][b] sb[j][b] (A B^T)_b.
//
// The matrix unit forms a block's sum over its 128 k in one 16x16x128
// instruction per 16x16 of C, from zero; four vector fmas then add the scaled
// sums to the fp32 accumulators, which therefore live in vector registers.  The
// rows of B take the instruction's first operand: a lane then holds one row of C
// (its scale of A is one register) and, in four registers, four consecutive
// columns; with a 16-bit C the rows of B are dealt out so that two instructions
// make eight (8 g + 4 (f % 2) + r of 32 to instruction f, lane group g, register
// r).  So a store is 16 bytes, and a row's 64 bytes leave together.
//
// A workgroup stays on its CU and takes tile after tile; the loads run ahead over a
// tile's end, so that the next tile's rows arrive while C is stored.  With a workgroup
// per tile each began with empty LDS: 16384 x 28672 x 512 took 426 us, now 394; 3000 x
// 28672 x 1000 (128x256) 135 and 120; 500 x 28672 x 4096 (64x128) 135 and 117; one
// tile per CU (4096^3) 59.8 and 60.5; where the card's power is the bound (16384 x
// 28672 x 8192) 3140 and 3112.
//
// What bounds the large tiles: a step of a 256x256 tile takes 3000 to 3400 cycles, of
// which the matrix unit works 2048 (without the loads into LDS 2830, without the fmas
// 3100), at the clock that the card's power allows: on random bytes 1.9 to 2.0 GHz,
// on zeros 2.4 (8192^3 436 and 358 us).  So fewer cycles pay a third of what they save.
//
// A step is one block of 128 k: A's and B's rows of 128 bytes go straight from
// memory to LDS (1 KB per instruction), two to six steps deep; one barrier per step.
// The chunks of 16 bytes of a row are permuted so that the fragment reads touch
// every bank once.  Rows and k outside the matrices are given an offset out of
// the buffer's range, which reads zeros; the bytes of a last piece past K are
// cleared in LDS.
#pragma once

#include <algorithm>
#include <type_traits>

#include "gemm8_common.hpp"

namespace ll {

template <int BM_, int BN_, int WM_, int WN_, int SLOTS_>
struct G8Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, WAVES = WM * WN, THREADS = WAVES * 64;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, SLOT = A_BYTES + B_BYTES;
  static constexpr int QA = BM / 8 / WAVES, QB = BN / 8 / WAVES;  // 1-KB loads of a wave
  static constexpr int SLOTS = SLOTS_;  // steps whose rows are in LDS or on their way
  static constexpr int SCALES = WAVES * 256;  // of a step; one more than SLOTS, as they are read until the step's end
  static constexpr int LDS = SLOTS * SLOT + (SLOTS + 1) * SCALES;
  static_assert(LDS <= 160 * 1024, "LDS");
  static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0 && TN <= 128 && 128 % TN == 0, "tile");
  static_assert((BM + 63) / 64 + (BN + 63) / 64 <= WAVES, "scales: 64 rows a wave");
};

template <class Cfg, bool E5M2, bool ROWS, bool EXACT>
__global__ void __launch_bounds__(Cfg::THREADS, 2) gemm8_tile_kernel(const Gemm8Args p) {
  typedef Block8<E5M2, EXACT> Block;
  __shared__ __align__(1024) char lds[Cfg::LDS];
  constexpr int FM = Cfg::FM, FN = Cfg::FN;
  constexpr int GF = EXACT || FN % 2 ? 1 : 2;  // instructions whose columns lie side by side
  // row of B's tile (column of C's), from a wave's first on, that instruction f takes as its first
  auto col_of = [](int f) { return 16 * GF * (f / GF) + 4 * (f % GF); };
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;

  // The arguments that only a change of tiles needs are read again there: kept in
  // scalar registers through the steps they pushed others out of them.
  auto args = []() __attribute__((always_inline)) -> const Gemm8Args& {
    auto q = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(q));
    return *(const Gemm8Args*)q;
  };

  // Work item -> (split, tile): the XCDs, which take workgroups in turn, get runs of
  // neighbouring tiles, in groups of 8 tile rows, so that those in flight share
  // panels in L2.  A workgroup takes every gridDim-th item; with a split K there are
  // as many workgroups as items, so that a workgroup has one split.
  struct Place {
    int m0, n0;
  };
  auto item_of = [](const Gemm8Args& a, uint32_t raw) __attribute__((always_inline)) {
    const uint32_t xcd = raw & 7, more = (uint32_t)a.total & 7;
    return xcd * ((uint32_t)a.total >> 3) + min(xcd, more) + (raw >> 3);
  };
  const int split = p.splits > 1 ? item_of(p, blockIdx.x) / (uint32_t)(p.tiles_m * p.tiles_n) : 0;
  const int kb0 = split * p.per_split, kb1 = min(p.blocks, kb0 + p.per_split);
  auto place = [&](const Gemm8Args& a, int raw) __attribute__((always_inline)) {
    const uint32_t tile = item_of(a, raw) - split * a.tiles_m * a.tiles_n;
    const uint32_t group = (uint32_t)((uint64_t)tile * a.by_group.magic >> a.by_group.shift);
    const uint32_t in_group = tile - group * 8 * a.tiles_n;
    const bool full = group < (uint32_t)a.tiles_m >> 3;
    const uint32_t n = full ? in_group >> 3 : (uint32_t)((uint64_t)in_group * a.by_last.magic >> a.by_last.shift);
    const uint32_t height = full ? 8 : a.tiles_m & 7;
    return Place{(int)(group * 8 + in_group - n * height) * Cfg::BM, (int)n * Cfg::BN};
  };
  if (p.blocks == 0) {  // sums of nothing
    for (int raw = blockIdx.x; raw < p.total; raw += gridDim.x) {
      const Place t = place(p, raw);
      for (int e = threadIdx.x; e < Cfg::BM * Cfg::BN / 4; e += Cfg::THREADS)
        store_c8<4>(p, 0, t.m0 + e / (Cfg::BN / 4), t.n0 + e % (Cfg::BN / 4) * 4, {0.f, 0.f, 0.f, 0.f});
    }
    return;
  }

  // loads: instruction q = wave + i WAVES takes rows 8q .. 8q+7 of the tile, lane
  // l row l / 8 of them, position l % 8.  The offset of a lane outside the
  // matrices is beyond every range, which reads zeros; the descriptors' own range
  // is not used.
  const int lrow = wave * 8 + (lane >> 3);
  auto chunk_b = [&](int i) { return ((lane & 7) ^ swz8_b<GF>(lrow + i * Cfg::WAVES * 8)) << 4; };
  const int la = ((lane & 7) ^ swz8_a(lrow)) << 4;
  static_assert(Cfg::WAVES * 8 % 16 == 0, "A's rows of a lane have one permutation");
  const uint32_t va = (uint32_t)((lane >> 3) * (int)p.lda + la);
  const int a_step = Cfg::WAVES * 8 * (int)p.lda, b_step = Cfg::WAVES * 8 * (int)p.ldb;
  // scales: a wave takes 64 rows, of A's or (behind them) of B's; what nobody
  // reads (B's without ROWS) is zeros
  constexpr int SA_WAVES = (Cfg::BM + 63) / 64;
  const bool of_a = wave < SA_WAVES;
  const int srow = (of_a ? wave : wave - SA_WAVES) * 64 + lane;
  const int64_t s_step = of_a ? p.sab : p.sbb;
  // The step that is loaded next, of a tile that may be ahead of the one being formed.
  const int k_stop = kb1 * 128;
  int l_raw = (int)blockIdx.x - (int)gridDim.x, m_left = 0, n_left = 0;  // rows of A and B from the tile's first on
  int k_next = k_stop, k_end = 0;                                        // k_end 0: there is no such step
  i32x4 rsrc_a = make_rsrc(p.a, 0x7FFFFFF0u), rsrc_b = make_rsrc(p.b, 0x7FFFFFF0u);
  uint32_t vs = kOOB;
  const float* ps = p.sa;
  auto enter = [&]() __attribute__((always_inline)) {  // the next tile
    const Gemm8Args& a = args();
    l_raw = min(l_raw + (int)gridDim.x, a.total);
    const Place t = place(a, min(l_raw, a.total - 1));
    m_left = a.M - t.m0;
    n_left = a.N - t.n0;
    k_next = kb0 * 128;
    k_end = l_raw < a.total ? a.K : 0;
    rsrc_a = make_rsrc(a.a + (uint64_t)(uint32_t)(t.m0 + wave * 8) * (uint32_t)a.lda, 0x7FFFFFF0u);
    rsrc_b = make_rsrc(a.b + (uint64_t)(uint32_t)(t.n0 + wave * 8) * (uint32_t)a.ldb, 0x7FFFFFF0u);
    const uint32_t stride = of_a ? (uint32_t)a.sam : (uint32_t)a.sbn;
    const bool live = of_a ? srow < Cfg::BM && srow < m_left : ROWS && srow < Cfg::BN && srow < n_left;
    vs = live ? (uint32_t)srow * stride * 4u : kOOB;
    ps = (of_a ? a.sa : a.sb) + (of_a || ROWS ? (uint64_t)(uint32_t)(of_a ? t.m0 : t.n0) * stride : 0) + kb0 * s_step;
  };

  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_u32((const char LL_LDS*)lds));
  constexpr uint32_t SC = Cfg::SLOTS * Cfg::SLOT;  // scales: per step, A's then B's
  // Load i (of QA + QB + 1) of the next step into its slot; past the last step it
  // reads nothing and writes zeros that nobody reads.
  constexpr int LOADS = Cfg::QA + Cfg::QB + 1;
  auto issue = [&](int i, int slot, int sslot) __attribute__((always_inline)) {
    const uint32_t at = lds0 + slot * Cfg::SLOT + wave * 1024;
    if (i < Cfg::QA) {
      const bool in = lrow + i * Cfg::WAVES * 8 < m_left && la < k_end - k_next;
      dma16s(rsrc_a, at + i * Cfg::WAVES * 1024, in ? va : kOOB, (uint32_t)(k_next + i * a_step));
    } else if (i < Cfg::QA + Cfg::QB) {
      const int q = i - Cfg::QA, lb = chunk_b(q);
      const bool in = lrow + q * Cfg::WAVES * 8 < n_left && lb < k_end - k_next;
      dma16s(rsrc_b, at + Cfg::A_BYTES + q * Cfg::WAVES * 1024,
             in ? (uint32_t)((lane >> 3) * (int)p.ldb + lb) : kOOB, (uint32_t)(k_next + q * b_step));
    } else {
      dma4(make_rsrc(ps, k_end ? 0x7FFFFFF0u : 0u), lds0 + SC + sslot * Cfg::SCALES + wave * 256, vs);
    }
  };
  // fragments: lane l takes row l % 16 and chunks l / 16 and l / 16 + 4
  const int row16 = lane & 15, g = lane >> 4;
  const int arow = wm * Cfg::TM + row16;
  const int brow = wn * Cfg::TN + (row16 >> 2) * 4 * GF + (row16 & 3);
  const int a_off = arow * 128 + ((g ^ swz8_a(arow)) << 4);                            // + 2048 i
  const int b_off = Cfg::A_BYTES + brow * 128 + ((g ^ swz8_b<GF>(brow)) << 4);  // + 128 col_of(f)
  // B's scales of squares: of the step's block row, unless ROWS
  typedef const float __attribute__((address_space(4))) * ScalePtr;
  auto squares_of = [&](const Gemm8Args& a, const Place& t) __attribute__((always_inline)) {
    return (ScalePtr)(a.sb + (int64_t)min((t.n0 + wn * Cfg::TN) / 128, (a.N - 1) / 128) * a.sbn + kb0 * a.sbb);
  };

  f32x4 acc[FM][FN];
  // One type, and pieces known to be whole, at a time: with every choice made at every
  // piece the stores' code was 40 KB, most of it jumped over.
  auto store = [&](const Place& t) __attribute__((always_inline)) {
    const Gemm8Args& a = args();
    const int m = t.m0 + wm * Cfg::TM + row16, n = t.n0 + wn * Cfg::TN + 4 * GF * g;
    auto pieces = [&](auto type, auto whole) __attribute__((always_inline)) {
      constexpr int TYPE = decltype(type)::value;
      typedef typename std::conditional<TYPE == LL_F32, float, uint16_t>::type E;
      E* const base = a.partial ? (E*)(a.partial + ((int64_t)split * a.M + m) * a.N + n) : (E*)a.c + m * a.ldc + n;
      const int64_t ld = 16 * (a.partial ? a.N : a.ldc);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int f = 0; f < FN; f += GF) {
          float v[4 * GF];
#pragma unroll
          for (int q = 0; q < 4 * GF; ++q) v[q] = acc[i][f + q / 4][q % 4];
          const int left = a.N - n - col_of(f);
          if (m + 16 * i < a.M && left > 0)
            store_piece8<TYPE, 4 * GF>(base + i * ld + col_of(f), v, decltype(whole)::value ? 4 * GF : left);
        }
    };
    auto typed = [&](auto whole) __attribute__((always_inline)) {
      if (EXACT || a.partial) pieces(std::integral_constant<int, LL_F32>(), whole);
      else if (a.c_type == LL_BF16) pieces(std::integral_constant<int, LL_BF16>(), whole);
      else pieces(std::integral_constant<int, LL_F16>(), whole);
    };
    if (a.N % (4 * GF) == 0 || t.n0 + Cfg::BN <= a.N) typed(std::true_type());
    else typed(std::false_type());
  };
  const int tail = p.K & 15 ? p.K / 128 : -1;  // the block whose last piece K ends in
  // Clears the bytes past K of the piece that K ends in.
  auto clear_tail = [&](int slot) __attribute__((always_inline)) {
    const int c = (p.K & 127) >> 4;
    for (int row = threadIdx.x; row < Cfg::BM + Cfg::BN; row += Cfg::THREADS) {
      const bool of_a = row < Cfg::BM;
      const int r = of_a ? row : row - Cfg::BM;
      char* q = lds + slot * Cfg::SLOT + row * 128 + ((c ^ (of_a ? swz8_a(r) : swz8_b<GF>(r))) << 4);
      for (int i = p.K & 15; i < 16; ++i) q[i] = 0;
    }
    __syncthreads();
  };
  // The rows of the next step are in their slot, for every wave, and nobody reads
  // those of the step before: the loads of another may begin there.
  auto landed = [&]() __attribute__((always_inline)) {
    static_assert((Cfg::SLOTS - 2) * LOADS < 64, "vmcnt");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((Cfg::SLOTS - 2) * LOADS) : "memory");  // those of later steps stay under way
    lds_barrier();
  };
  auto read_x = [&](const char* st, int i) {
    return frag8(*(const i32x4*)(st + a_off + 2048 * i), *(const i32x4*)(st + (a_off ^ 64) + 2048 * i));
  };
  auto read_w = [&](const char* st, int f) {
    return frag8(*(const i32x4*)(st + b_off + 128 * col_of(f)), *(const i32x4*)(st + (b_off ^ 64) + 128 * col_of(f)));
  };
  const int sa_off = SC + (wm * Cfg::TM + row16) * 4;                              // + 64 i
  const int sb_off = SC + (SA_WAVES * 64 + wn * Cfg::TN + 4 * GF * g) * 4;  // + 4 col_of(f)

  // A step is FM x FN products, in the order below.  A product's fmas follow LAG
  // products later, when its result is there; the fragments of A are read one
  // row of products ahead, those of the next step during the last row, after the
  // barrier that says that its rows have landed and that nobody reads this step's.
  constexpr bool FEW_SB = EXACT;
  constexpr int T = FM * FN, LAG = EXACT ? 1 : FN < 3 ? FN : 3, ND = LAG < 2 ? 2 : 4;
  static_assert(T % ND == 0 && LAG < ND && LAG <= FN && FM % 2 == 0, "ring of results");
  // The loads of a later step begin behind that barrier and go on into the next
  // step, AT_ONCE for every PACE products: in a burst they filled the address
  // unit's queue, and the matrix unit stood still meanwhile (8192^3, 256x256, one or
  // two more at once: 3% and 12% more cycles; at every second product 7% fewer and,
  // with the clock that the card's power then allows, 445 -> 436 us, but with B's
  // scales by rows 504 -> 510, to fp32 824 -> 832, and 2048 x 4096 x 4096, 128x256, 37.5
  // -> 38.8).
  constexpr int PACE = T >= 32 && !EXACT && !ROWS ? 2 : 1, AT_ONCE = (LOADS * PACE + T - 1) / T;
  constexpr int EARLY = FN / PACE * AT_ONCE < LOADS ? FN / PACE * AT_ONCE : LOADS;
  static_assert(FN % PACE == 0 && T % PACE == 0, "loads of a step");
  f32x4 d[ND], sbv[FEW_SB ? 1 : FN];  // sbv (ROWS): of all f, or (EXACT, whose operands take the registers) of the last product
  i32x8 wr[FN], xr[2];
  typename Block::W w[FN];
  typename Block::X x;
  float s = 0.f, sa_next = 0.f, sb = 0.f, sb_next = 0.f;  // s: scale of the last row of products
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int f = 0; f < FN; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ND; ++i) d[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int f = 0; f < (FEW_SB ? 1 : FN); ++f) sbv[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    s = 0.f;
  };
  auto add = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      acc[t / FN][t % FN][r] =
          fmaf(d[t % ND][r], ROWS ? s * sbv[FEW_SB ? 0 : t % FN][r] : s, acc[t / FN][t % FN][r]);
    asm volatile("" : "+v"(acc[t / FN][t % FN]));  // here, not where the compiler would sink them to
  };

#pragma nounroll
  for (int n = 0;; ++n) {
    if (k_next >= k_stop) enter();
    if (n == Cfg::SLOTS - 1) break;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) issue(i, n, n);
    k_next += 128;
    ps += s_step;
  }
  landed();
  if (kb0 == tail) clear_tail(0);
#pragma unroll
  for (int i = 0; i < EARLY; ++i) issue(i, Cfg::SLOTS - 1, Cfg::SLOTS - 1);
  xr[0] = read_x(lds, 0);
  sa_next = *(const float*)(lds + sa_off);
#pragma unroll
  for (int f = 0; f < FN; ++f) wr[f] = read_w(lds, f);
  int slot = 0, s0 = 0;  // of the step's rows and scales
  Place at = place(p, blockIdx.x);
  ScalePtr squares = squares_of(p, at);
  if constexpr (!ROWS) sb = *squares;
  for (int raw = blockIdx.x;;) {
    clear();
    raw += gridDim.x;
    const bool more = raw < p.total;
    ScalePtr squares_then = squares;
    if (!ROWS && more) squares_then = squares_of(args(), place(args(), raw));
    for (int kb = kb0; kb < kb1; ++kb) {
      const bool last = kb + 1 == kb1;
      const int slot1 = slot + 1 < Cfg::SLOTS ? slot + 1 : 0, s1 = s0 < Cfg::SLOTS ? s0 + 1 : 0;  // of the next step
      const int slot_before = slot > 0 ? slot - 1 : Cfg::SLOTS - 1;  // free since the last barrier
      const int s_last2 = s0 >= 2 ? s0 - 2 : s0 + Cfg::SLOTS - 1, s_last1 = s0 >= 1 ? s0 - 1 : Cfg::SLOTS;
      const char* st = lds + slot * Cfg::SLOT;
      const char* next = lds + slot1 * Cfg::SLOT;
      const char* sc = lds + s0 * Cfg::SCALES;
      squares = last ? squares_then : squares + p.sbb;
      if constexpr (!ROWS) sb_next = *squares;
      auto product = [&](int t) __attribute__((always_inline)) {
        const int i = t / FN, f = t % FN;
        if (f == 0) x = Block::x(xr[i & 1]);
        if (i == 0) w[f] = Block::w(wr[f]);
        // (8192 x 8192 x 16384 to fp32 with B's scales by rows 1946 -> 1820 us; by squares
        // 8192^3 824 -> 832, and without EXACT 3% more)
        if (EXACT && ROWS) __builtin_amdgcn_s_setprio(1);
        d[t % ND] = Block::product(w[f], x);
        if (EXACT && ROWS) __builtin_amdgcn_s_setprio(0);
        add((t + T - LAG) % T);
        if (f == LAG - 1) s = ROWS ? sa_next : sa_next * sb;  // of this row of products from here on
        if (ROWS && FEW_SB) sbv[0] = *(const f32x4*)(sc + sb_off + 4 * col_of(f));
        if (ROWS && !FEW_SB && t == LAG - 1) {
#pragma unroll
          for (int q = 0; q < FN; ++q) sbv[q] = *(const f32x4*)(sc + sb_off + 4 * col_of(q));
        }
        if (f == 0) xr[(i + 1) & 1] = i + 1 < FM ? read_x(st, i + 1) : read_x(next, 0);
        // the scales of the next row of products, once those of this one have been taken
        if (LAG == FN && f == 0) sa_next = *(const float*)(sc + sa_off + 64 * i);
        if (LAG < FN && f == LAG)
          sa_next = *(const float*)(i + 1 < FM ? sc + sa_off + 64 * (i + 1) : lds + s1 * Cfg::SCALES + sa_off);
        if (i == FM - 1) wr[f] = read_w(next, f);
        if (t % PACE == 0) {
#pragma unroll
          for (int n = 0; n < AT_ONCE; ++n) {
            const int q = t / PACE * AT_ONCE + n + EARLY;
            if (q < LOADS && i < FM - 1) issue(q, slot_before, s_last2);
          }
#pragma unroll
          for (int n = 0; n < AT_ONCE; ++n) {
            const int q = f / PACE * AT_ONCE + n;
            if (i == FM - 1 && q < EARLY) issue(q, slot, s_last1);
          }
        }
      };
#pragma unroll
      for (int t = 0; t < T - FN; ++t) product(t);
      k_next += 128;
      ps += s_step;
      landed();
      const bool cut = (last ? kb0 : kb + 1) == tail, end = k_next >= k_stop;
      if (cut || end) {
        if (cut) clear_tail(slot1);
        if (end) enter();
      }
#pragma unroll
      for (int t = T - FN; t < T; ++t) product(t);
      sb = sb_next;
      slot = slot1;
      s0 = s1;
    }
#pragma unroll
    for (int t = T - LAG; t < T; ++t) add(t);
    store(at);
    if (!more) break;
    at = place(args(), raw);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the workgroup
}

template <class Cfg, bool EXACT>
hipError_t launch_gemm8_tile(const Gemm8Args& args, bool a_e5m2, bool rows, hipStream_t s) {
  auto kernel = a_e5m2 ? (rows ? gemm8_tile_kernel<Cfg, true, true, EXACT> : gemm8_tile_kernel<Cfg, true, false, EXACT>)
                       : (rows ? gemm8_tile_kernel<Cfg, false, true, EXACT>
                               : gemm8_tile_kernel<Cfg, false, false, EXACT>);
  Gemm8Args a = args;
  a.by_group = quotient8(8u * (uint32_t)a.tiles_n);
  a.by_last = quotient8(std::max(1u, (uint32_t)a.tiles_m & 7));
  const int grid = a.splits > 1 ? a.total : std::min(a.total, a.cus);
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(Cfg::THREADS), 0, s, a);
  return hipGetLastError();
}

}  // namespace ll
