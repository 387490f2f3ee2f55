// The cross entropy of narrow rows (D up to 128): the logits are formed again in
// each of the three steps, and never stored.
//
// With D this small a logit costs less to form (2 D flops) than to write and
// read back as 16 bits in three passes.  One kernel, by what it makes of the
// logits of its own rows against streamed ones:
//
//   kNarrowStats  own x, streamed w: (maximum, sum) of each row's logits
//   kNarrowDx     own x, streamed w: dx[n] = sum_v dz[n][v] w[v]
//   kNarrowDw     own w, streamed x: dw[v] = sum_n dz[n][v] x[n]
//
// with dz = (exp(z - lse) - onehot) * coef.  A wave holds 16 RT own rows in
// registers as the columns of the 16x16x32 matrix instruction; the streamed
// rows pass through LDS, 64 at a time, two buffers.  The instruction leaves in
// each lane the logits of one own row against streamed rows 4 g + e of two tiles
// of 16; rounded, these are already the operand of the second product, if its
// inner index runs 4 g + 0 .. 3 of the first tile and then of the second, and the
// streamed rows are read from LDS (transposed) in that order.  So nothing goes
// from lane to lane.  Column m of the second product's d-tile is column 16 (m / 4)
// + 4 dt + m % 4 of its 64, which leaves 16 consecutive values of an own row in
// a lane.
//
// Bound by the vector ALU: per logit and step a subtraction, a multiplication
// or fma, an exponential (at a fraction of the others' rate), dw's factor and
// half a conversion, 5 or 6 instructions beside 2 (statistics) or 4 D flops of
// the matrix cores.  16384 x 131072 x 64 (2.1e9 logits): statistics 640 us, dx
// and dw 1580 us, 3.6e12 logits a second in all; 8192 x 32768 x 128: 132 and 445
// us.  Two tiles of own rows per wave and three waves per SIMD (D <= 64): four
// tiles and two waves took 2330 us against 2145 for the whole call; both halves
// of a step unrolled spilled (2480).
#include <algorithm>

#include "ops_common.hpp"
#include "xent.hpp"
#include "xent_rows.hpp"

namespace ll {

constexpr int kNarrowBlock = 64;  // streamed rows per step
constexpr int kNarrowTiles = 2;   // own 16-row tiles per wave
// dx of fp16: exp(z - lse) as 16 bits carries this factor, so that it stays a
// normal number down to 2^-29
template <int TY>
constexpr int kNarrowExp = TY == LL_F16 ? 15 : 0;

template <int DP>
constexpr int kNarrowWaves = DP == 64 ? 3 : 2;  // per SIMD
template <int DP>
struct NarrowLds {
  static constexpr int PITCH = DP + 8;
  __attribute__((aligned(16))) uint16_t tile[2][kNarrowBlock * PITCH];
  __attribute__((aligned(16))) float lse[2][kNarrowBlock], coef[2][kNarrowBlock];
  __attribute__((aligned(16))) int column[2][kNarrowBlock];
};

// Elements d .. d + 7 of a row of D, D >= 8: 16 bytes that lie in the row, to be
// moved down once they are there.
struct NarrowRow {
  int at, by;
  __device__ __forceinline__ NarrowRow(int d, int D) : at(min(d, D - 8)), by(d - at) {}
  template <class C>
  __device__ __forceinline__ void place(C& c) const {
    if (by == 0) return;
    if (by >= 8) {
      c.clear();
      return;
    }
    if (by & 4) {
      c.w[0] = c.w[2];
      c.w[1] = c.w[3];
      c.w[2] = c.w[3] = 0;
    }
    if (by & 2) {
      c.w[0] = c.w[1];
      c.w[1] = c.w[2];
      c.w[2] = c.w[3];
      c.w[3] = 0;
    }
    if (by & 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) c.w[i] = c.w[i] >> 16 | (i < 3 ? c.w[i + 1] << 16 : 0);
    }
  }
};

template <int TY, int DP, int MODE>
__device__ __forceinline__ void narrow_body(const XentRows& r, const XentNarrowOut& o, NarrowLds<DP>& lds, int row_block,
                                            int share, int shares) {
  constexpr int RT = kNarrowTiles, KS = DP / 32, PITCH = DP + 8, CHUNKS = DP / 8;
  constexpr int PER = kNarrowBlock * CHUNKS / 256;  // 16-byte loads per thread and step
  typedef Chunk<TY, 8> C;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, c16 = lane & 15;
  // N and V are below 2^30
  const int own_n = (int)(MODE == kNarrowDw ? r.V : r.N), str_n = (int)(MODE == kNarrowDw ? r.N : r.V);
  const int64_t own_ld = MODE == kNarrowDw ? r.ldw : r.ldx, str_ld = MODE == kNarrowDw ? r.ldx : r.ldw;
  const uint16_t* const own_p = (const uint16_t*)(MODE == kNarrowDw ? r.w : r.x);
  const uint16_t* const str_p = (const uint16_t*)(MODE == kNarrowDw ? r.x : r.w);
  const int own0 = row_block * (64 * RT) + wave * 16 * RT;

  C own[RT][KS];
  float lse[RT], coef[RT];
  int column[RT];
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    const int i = own0 + 16 * q + c16;
    lse[q] = coef[q] = 0.f;
    column[q] = -1;
    if (i < own_n) {
      if constexpr (MODE == kNarrowStats) {
        const int64_t t = r.target[i];
        if (has_target(r, t)) column[q] = (int)t;
      } else if constexpr (MODE == kNarrowDx) {
        coef[q] = r.coef[i];
        column[q] = r.column[i];
        // no target: exp(0 - infinity), so that the sums are 0; those of w itself may pass fp32's range
        lse[q] = column[q] >= 0 ? r.lse[i] : __builtin_huge_valf();
      }
    }
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int d = 32 * k + 8 * g;
      own[q][k].clear();
      // a row of x without a target counts as zeros, whatever it holds
      if (i < own_n && d < r.D && (MODE == kNarrowDw || column[q] >= 0))
        own[q][k].template load<true>(own_p + (int64_t)i * own_ld + d, r.D - d);
    }
  }

  C in[PER];
  float in_lse = 0.f, in_coef = 0.f;
  int in_column = -1;
  bool in_live[PER];
  const int d = threadIdx.x % CHUNKS * 8;  // of this thread's chunks
  const bool short_row = r.D < 8;          // uniform
  const NarrowRow at(d, r.D);
  auto load = [&](int b) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = b * kNarrowBlock + threadIdx.x / CHUNKS + 256 / CHUNKS * j;
      in[j].clear();
      in_live[j] = true;
      if (i < str_n && d < r.D) {
        if (MODE == kNarrowDw) in_live[j] = r.column[i] >= 0;
        if (short_row) in[j].template load<true>(str_p + (int64_t)i * str_ld + d, r.D - d);
        else in[j].template load<false>(str_p + (int64_t)i * str_ld + at.at, 8);
      }
    }
    if (MODE == kNarrowDw && threadIdx.x < kNarrowBlock) {
      const int i = b * kNarrowBlock + threadIdx.x;
      in_lse = i < str_n ? r.lse[i] : 0.f;
      in_coef = i < str_n ? r.coef[i] : 0.f;
      in_column = i < str_n ? r.column[i] : -1;
    }
  };
  auto put = [&](int slot) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (MODE == kNarrowDw && !in_live[j]) in[j].clear();
      if (!short_row && (r.D & 7)) at.place(in[j]);
      __builtin_memcpy(&lds.tile[slot][(threadIdx.x / CHUNKS + 256 / CHUNKS * j) * PITCH + d], &in[j], 16);
    }
    if (MODE == kNarrowDw && threadIdx.x < kNarrowBlock) {
      lds.lse[slot][threadIdx.x] = in_lse;
      lds.coef[slot][threadIdx.x] = in_coef;
      lds.column[slot][threadIdx.x] = in_column;
    }
  };

  f32x4 acc[KS / 2][4][RT];
  float m[RT], s[RT];
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    m[q] = kNegInf;
    s[q] = 0.f;
#pragma unroll
    for (int d = 0; d < KS / 2; ++d)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[d][t][q] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // SLOW: a row's target is among these logits, w ends in this step or holds infinities
  auto step = [&](auto slow, int slot, int b, int h) {
    constexpr bool SLOW = decltype(slow)::value;
    const uint16_t* const t0 = &lds.tile[slot][32 * h * PITCH];
    f32x4 z[2][RT];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int q = 0; q < RT; ++q) z[t][q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        C a;
        __builtin_memcpy(&a, t0 + (16 * t + c16) * PITCH + 32 * k + 8 * g, 16);
#pragma unroll
        for (int q = 0; q < RT; ++q) z[t][q] = mfma16(a, own[q][k], z[t][q]);
      }
    }
    const int v0 = b * kNarrowBlock + 32 * h + 4 * g;  // + 16 t + e: the lane's streamed rows
    if constexpr (MODE == kNarrowStats) {
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        float top = m[q];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (SLOW) {
              const int v = v0 + 16 * t + e;
              if (column[q] == v) r.zt[own0 + 16 * q + c16] = z[t][q][e];
              if (v >= str_n) z[t][q][e] = kNegInf;
            }
            top = fmaxf(top, z[t][q][e]);
          }
        const float base = top == kNegInf ? 0.f : top;
        float sum = s[q] * __expf(m[q] - base);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += __expf(z[t][q][e] - base);
        m[q] = top;
        s[q] = sum;
      }
    } else {
      C p[RT];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 l4, c4;
        int k4[4];
        if constexpr (MODE == kNarrowDw) {
          l4 = *(const f32x4*)&lds.lse[slot][32 * h + 16 * t + 4 * g];
          c4 = *(const f32x4*)&lds.coef[slot][32 * h + 16 * t + 4 * g];
          if constexpr (SLOW) __builtin_memcpy(k4, &lds.column[slot][32 * h + 16 * t + 4 * g], 16);
        }
#pragma unroll
        for (int q = 0; q < RT; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // dx: its row's coef, and this factor's inverse, wait for the sum
            constexpr float BIAS = MODE == kNarrowDx ? kNarrowExp<TY> : 0, ONE = 1 << (int)BIAS;
            const float x = z[t][q][e] - (MODE == kNarrowDw ? l4[e] : lse[q]);
            float y = __builtin_amdgcn_exp2f(fmaf(x, 1.44269504f, BIAS));
            if constexpr (SLOW) {
              const int v = v0 + 16 * t + e;
              if (MODE == kNarrowDw ? k4[e] == own0 + 16 * q + c16 : column[q] == v) y -= ONE;
              if (MODE == kNarrowDx ? v >= str_n : k4[e] < 0) y = 0.f;
            }
            z[t][q][e] = MODE == kNarrowDw ? y * c4[e] : y;
          }
        // rounded to 16 bits, as the gradient of a logit is everywhere here
#pragma unroll
        for (int q = 0; q < RT; ++q)
#pragma unroll
          for (int e = 0; e < 4; e += 2) p[q].put2(4 * t + e, z[t][q][e], z[t][q][e + 1]);
      }
#pragma unroll
      for (int d = 0; d < KS / 2; ++d)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint16_t LL_LDS* const at = (const uint16_t LL_LDS*)t0 + (4 * g + (c16 >> 2)) * PITCH + 64 * d +
                                            16 * (c16 & 3) + 4 * t;
          const C a = frag_pair<TY>(at, at + 16 * PITCH);
#pragma unroll
          for (int q = 0; q < RT; ++q) acc[d][t][q] = mfma16(a, p[q], acc[d][t][q]);
        }
    }
  };

  const int blocks = (str_n + kNarrowBlock - 1) / kNarrowBlock, per = blocks / shares, more = blocks % shares;
  const int b0 = share * per + min(share, more), b1 = b0 + per + (share < more ? 1 : 0);
  int slot = 0;
  if (b0 < b1) {
    load(b0);
    put(0);
  }
  // an infinity in w (a masked entry): it meets the zeros of rows without a target as a NaN
  bool endless = false;
  if constexpr (MODE == kNarrowDw) {
    constexpr uint32_t EXP = TY == LL_F16 ? 0x7C00u : 0x7F80u;
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) endless |= (own[q][k].get_raw(i) & EXP) == EXP;
    endless = __any(endless);
  }
  for (int b = b0; b < b1; ++b, slot ^= 1) {
    __syncthreads();  // this block is there, and the other slot is free
    if (b + 1 < b1) load(b + 1);
    bool slow = MODE != kNarrowDw && (b + 1) * kNarrowBlock > str_n;
    if constexpr (MODE != kNarrowDw) {
      bool mine = false;
#pragma unroll
      for (int q = 0; q < RT; ++q) mine |= (unsigned)(column[q] - b * kNarrowBlock) < (unsigned)kNarrowBlock;
      slow |= __any(mine);
    } else {
      slow = endless || __any((unsigned)(lds.column[slot][lane] - own0) < (unsigned)(16 * RT));
    }
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      if (slow) step(std::true_type{}, slot, b, h);
      else step(std::false_type{}, slot, b, h);
    }
    if (b + 1 < b1) put(slot ^ 1);
  }

  if constexpr (MODE == kNarrowStats) {
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      join(m[q], s[q], __shfl_xor(m[q], 16, 64), __shfl_xor(s[q], 16, 64));
      join(m[q], s[q], __shfl_xor(m[q], 32, 64), __shfl_xor(s[q], 32, 64));
      const int i = own0 + 16 * q + c16;
      if (g == 0 && i < own_n) r.parts[(int64_t)share * r.part_ld + i] = float2{m[q], s[q]};
    }
  } else {
    const float unscale = o.scale && !o.partial ? *o.scale : 1.f;
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      const int i = own0 + 16 * q + c16;
      if (i >= own_n) continue;
      const float f = (MODE == kNarrowDx ? coef[q] * (1.f / (1 << kNarrowExp<TY>)) : 1.f) * unscale;
#pragma unroll
      for (int d = 0; d < KS / 2; ++d) {
        const int c = 64 * d + 16 * g;
        if (o.partial) {
#pragma unroll
          for (int t = 0; t < 4; ++t)
            *(f32x4*)(o.partial + ((int64_t)share * own_n + i) * DP + c + 4 * t) = acc[d][t][q] * f;
        } else if (o.type == LL_F32) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            Chunk<LL_F32, 4> v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v.put(e, acc[d][t][q][e] * f);
            if (c + 4 * t < r.D) v.template store<true>((uint32_t*)o.out + (int64_t)i * o.ldo + c + 4 * t, r.D - c - 4 * t);
          }
        } else {
#pragma unroll
          for (int t = 0; t < 4; t += 2) {
            C v;
#pragma unroll
            for (int e = 0; e < 8; e += 2)
              v.put2(e, acc[d][t + (e >> 2)][q][e & 3] * f, acc[d][t + (e >> 2)][q][(e & 3) + 1] * f);
            if (c + 4 * t < r.D) v.template store<true>((uint16_t*)o.out + (int64_t)i * o.ldo + c + 4 * t, r.D - c - 4 * t);
          }
        }
      }
    }
  }
}

template <int TY, int DP>
__global__ void __launch_bounds__(256, kNarrowWaves<DP>) xent_narrow_stats_kernel(const XentRows r, int row_blocks) {
  __shared__ NarrowLds<DP> lds;
  if ((int)blockIdx.x == row_blocks * r.np) {
    scale_block<256>(r, lds.lse[0]);
    return;
  }
  narrow_body<TY, DP, kNarrowStats>(r, XentNarrowOut{}, lds, blockIdx.x % row_blocks, blockIdx.x / row_blocks, r.np);
}

// The first workgroups form dx, the others dw: each alone would leave CUs idle
// at small sizes, and a launch costs 4 us.
template <int TY, int DP>
__global__ void __launch_bounds__(256, kNarrowWaves<DP>)
    xent_narrow_grad_kernel(const XentRows r, const XentNarrowOut dx, const XentNarrowOut dw) {
  __shared__ NarrowLds<DP> lds;
  const int nx = dx.row_blocks * dx.shares;
  if ((int)blockIdx.x < nx) {
    narrow_body<TY, DP, kNarrowDx>(r, dx, lds, blockIdx.x % dx.row_blocks, blockIdx.x / dx.row_blocks, dx.shares);
  } else {
    const int b = blockIdx.x - nx;
    narrow_body<TY, DP, kNarrowDw>(r, dw, lds, b % dw.row_blocks, b / dw.row_blocks, dw.shares);
  }
}

// The shares' sums, in order; four columns per thread.  The first `first`
// workgroups take x, the others y.
__global__ void __launch_bounds__(256) xent_narrow_sum_kernel(const XentNarrowOut x, const XentNarrowOut y, int D,
                                                              int dp, int first) {
  const bool second = (int)blockIdx.x >= first;
  const XentNarrowOut& o = second ? y : x;
  const int64_t q = (int64_t)(blockIdx.x - (second ? first : 0)) * 256 + threadIdx.x;
  const int per = dp / 4, c = (int)(q % per) * 4;
  const int64_t i = q / per;
  if (i >= o.rows || c >= D) return;
  const float* p = o.partial + i * dp + c;
  f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < o.shares; ++k) sum += *(const f32x4*)(p + (int64_t)k * o.rows * dp);
  sum *= o.scale ? *o.scale : 1.f;
  auto out = [&](auto type) {
    constexpr int OT = decltype(type)::value;
    Chunk<OT, 4> v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v.put(e, sum[e]);
    v.template store<true>((typename Elem<OT>::raw*)o.out + i * o.ldo + c, D - c);
  };
  if (o.type == LL_BF16) out(std::integral_constant<int, LL_BF16>{});
  else if (o.type == LL_F16) out(std::integral_constant<int, LL_F16>{});
  else out(std::integral_constant<int, LL_F32>{});
}

constexpr int kNarrowRows = 64 * kNarrowTiles;  // own rows of a workgroup

// Enough shares for `slots` workgroups, each with at least four steps of its own.
int xent_narrow_shares(int64_t own, int64_t streamed, int64_t slots) {
  const int64_t blocks = (own + kNarrowRows - 1) / kNarrowRows;
  const int64_t steps = (streamed + kNarrowBlock - 1) / kNarrowBlock;
  return (int)std::max<int64_t>(1, std::min<int64_t>(slots / blocks, steps / 4));
}

hipError_t launch_xent_narrow_stats(const XentRows& r, bool scaled, int type, hipStream_t s) {
  if (r.N < 1 || r.ldp < r.D || (r.ldp != 64 && r.ldp != 128)) return hipErrorInvalidValue;
  const int row_blocks = (int)((r.N + kNarrowRows - 1) / kNarrowRows);
  const dim3 grid((unsigned)(row_blocks * r.np + scaled));
#define LL_STATS(TY, DP) \
  hipLaunchKernelGGL((xent_narrow_stats_kernel<TY, DP>), grid, dim3(256), 0, s, r, row_blocks)
  if (type == LL_BF16) {
    if (r.ldp == 64) LL_STATS(LL_BF16, 64);
    else LL_STATS(LL_BF16, 128);
  } else {
    if (r.ldp == 64) LL_STATS(LL_F16, 64);
    else LL_STATS(LL_F16, 128);
  }
#undef LL_STATS
  return hipGetLastError();
}

hipError_t launch_xent_narrow_grad(const XentRows& r, XentNarrowOut dx, XentNarrowOut dw, int type, hipStream_t s) {
  if (r.N < 1 || r.ldp < r.D || (r.ldp != 64 && r.ldp != 128)) return hipErrorInvalidValue;
  int sums[2], i = 0;
  for (XentNarrowOut* o : {&dx, &dw}) {
    o->rows = o == &dx ? r.N : r.V;
    o->row_blocks = o->shares ? (int)((o->rows + kNarrowRows - 1) / kNarrowRows) : 0;
    if ((o->shares > 1) != (o->partial != nullptr)) return hipErrorInvalidValue;
    sums[i++] = o->shares > 1 ? (int)((o->rows * (r.ldp / 4) + 255) / 256) : 0;
  }
  const dim3 grid((unsigned)(dx.row_blocks * dx.shares + dw.row_blocks * dw.shares));
#define LL_GRAD(TY, DP) hipLaunchKernelGGL((xent_narrow_grad_kernel<TY, DP>), grid, dim3(256), 0, s, r, dx, dw)
  if (type == LL_BF16) {
    if (r.ldp == 64) LL_GRAD(LL_BF16, 64);
    else LL_GRAD(LL_BF16, 128);
  } else {
    if (r.ldp == 64) LL_GRAD(LL_F16, 64);
    else LL_GRAD(LL_F16, 128);
  }
#undef LL_GRAD
  if (sums[0] + sums[1])
    hipLaunchKernelGGL(xent_narrow_sum_kernel, dim3((unsigned)(sums[0] + sums[1])), dim3(256), 0, s, dx, dw, r.D, r.ldp,
                       sums[0]);
  return hipGetLastError();
}

}  // namespace ll
