// Embedding lookup out[t] = scale * table[ids[t]] and its gradient
// dw[v] = scale * (sum of dout[t] over the tokens t with ids[t] == v).
//
// The lookup reads and writes each row once: HBM bound.  32768 rows of 4096 bf16
// out of 131072: 81 us, 6.6 TB/s of rows in and out (repeated ids come from the
// caches); one row: 1.9 us, the launch.
//
// The gradient sorts the tokens by id, stably (a counting sort by digits of
// the (id, position) pairs, so a row's tokens stay in their order), and sums
// each row's tokens, now neighbours, in that order: no floating-point atomics,
// so the result does not depend on timing.  Most rows of a large table have no
// token.  The sort keeps few CUs busy, so its longer launches also write a
// share of the zeros each, and the sums then overwrite the rows that have tokens.
// A few ids take a large share of the positions in real data: sums over whole
// chunks of kEmbedChunk sorted positions that belong to one row are formed in
// parallel over the chunks, beside the rows that hold none, and a last launch
// joins those of the rows that hold some.
// HBM bound by the zeros and the tokens' rows: 32768 x 4096 bf16 into 65536 rows
// 182 us, 4.4 TB/s (sort and zeros 85 to 90, sums 74, long rows 13); 262144 x 64
// fp32 into 1000003 103 us, 3.1 TB/s (sort and zeros 55 to 60, sums 32, long rows
// 11), there bound by the sort's chain of launches.
//
// Rows start at any element and have any width: a 16-byte access needs no
// alignment here, so the lanes always move 16 bytes and only a row's last
// lane takes single elements.
#include "embed.hpp"

#include <algorithm>

#include "ops_common.hpp"

namespace ll {

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------

// lx lanes move one row; 256 / lx rows per workgroup and step.
template <int TY, bool TAIL>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedArgs a, int lx_log2) {
  constexpr int VEC = kWide<TY>;
  typedef Chunk<TY, VEC> C;
  typedef typename C::raw raw;
  const int lx = 1 << lx_log2;
  const int x = threadIdx.x & (lx - 1), y = threadIdx.x >> lx_log2;
  const int rows = 256 >> lx_log2;
  for (int64_t t = (int64_t)blockIdx.x * rows + y; t < a.T; t += (int64_t)gridDim.x * rows) {
    const int64_t id = a.ids[t];
    const bool inside = id >= 0 && id < a.V;
    raw* dst = (raw*)a.out + t * a.ldo;
    const raw* src = (const raw*)a.table + (inside ? id : 0) * a.ldt;
    for (int d = x * VEC; d < a.D; d += lx * VEC) {
      C v;
      if (inside) v.template load<TAIL>(src + d, a.D - d);
      else v.clear();
#pragma unroll
      for (int i = 0; i < VEC; ++i) v.put(i, v.get(i) * a.scale);
      v.template store<TAIL>(dst + d, a.D - d);
    }
  }
}

// Smallest power of two >= n, at most 2^most_log2, as its logarithm.
static int log2_up(int64_t n, int most_log2) {
  int l = 0;
  while (l < most_log2 && (1ll << l) < n) ++l;
  return l;
}

template <int TY, bool TAIL>
static hipError_t launch_embed_t(const EmbedArgs& a, hipStream_t s) {
  constexpr int VEC = kWide<TY>;
  const int lx = log2_up((a.D + VEC - 1) / VEC, 8);
  const int rows = 256 >> lx;
  const int64_t blocks = std::min<int64_t>((a.T + rows - 1) / rows, 1 << 16);
  hipLaunchKernelGGL((embed_kernel<TY, TAIL>), dim3((unsigned)blocks), dim3(256), 0, s, a, lx);
  return hipGetLastError();
}

hipError_t launch_embed(const EmbedArgs& a, int type, hipStream_t s) {
  switch (type) {
    case LL_BF16: return a.D % 8 ? launch_embed_t<LL_BF16, true>(a, s) : launch_embed_t<LL_BF16, false>(a, s);
    case LL_F16: return a.D % 8 ? launch_embed_t<LL_F16, true>(a, s) : launch_embed_t<LL_F16, false>(a, s);
    case LL_F32: return a.D % 4 ? launch_embed_t<LL_F32, true>(a, s) : launch_embed_t<LL_F32, false>(a, s);
    default: return hipErrorInvalidValue;
  }
}

// ---------------------------------------------------------------------------
// Stable sort of (id, position).  Tokens without a gradient (padding or an id
// outside the table) get the key V and end up behind all others.
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t token_key(const EmbedGradArgs& a, int t) {
  const int64_t id = a.ids[t];
  return (id < 0 || id >= a.V || id == a.padding) ? (uint32_t)a.V : (uint32_t)id;
}

// One wave-step of a stable counting sort: lanes with equal digits find each
// other with one ballot per digit bit and take consecutive places after the
// digit's count so far (cnt, of this wave), which then moves on.
__device__ __forceinline__ uint32_t wave_place(uint32_t* cnt, uint32_t digit, int bits, bool live, uint64_t below) {
  uint64_t peers = __ballot(live);
  for (int k = 0; k < bits; ++k) {
    const uint64_t set = __ballot((digit >> k) & 1);
    peers &= ((digit >> k) & 1) ? set : ~set;
  }
  const uint32_t rank = (uint32_t)__popcll(peers & below);
  const uint32_t at = live ? cnt[digit] + rank : 0;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (live && rank == 0) cnt[digit] += (uint32_t)__popcll(peers);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return at;
}

// Exclusive scan of v over the workgroup's threads; tmp holds one word per wave.
template <int THREADS>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* tmp) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  uint32_t s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t t = __shfl_up(s, d, 64);
    if (lane >= d) s += t;
  }
  if (lane == 63) tmp[wave] = s;
  __syncthreads();
  uint32_t base = 0;
  for (int w = 0; w < wave; ++w) base += tmp[w];
  __syncthreads();
  return base + s - v;
}

// Share `part` of `parts` of the zeros of dw, by the launch's workgroups from
// `first` on (none where the sums are added to dw).  Whole rows per share.
struct FillShare {
  int first, part, parts;
};
template <int THREADS>
__device__ __forceinline__ void fill_share(const EmbedGradArgs& a, int esize, const FillShare f) {
  const int64_t r0 = a.V * f.part / f.parts, r1 = a.V * (f.part + 1) / f.parts;
  const int64_t id = (int64_t)(blockIdx.x - f.first) * THREADS + threadIdx.x;
  const int64_t step = (int64_t)(gridDim.x - f.first) * THREADS;
  typedef uint32_t words __attribute__((ext_vector_type(4)));
  typedef words unaligned_words __attribute__((aligned(2)));
  const words zero = {0, 0, 0, 0};
  char* const base = (char*)a.dw;
  if (a.ldw == a.D) {  // one run of bytes
    const int64_t b0 = r0 * a.D * esize, n = (r1 - r0) * a.D * esize;
    for (int64_t i = id; i < n / 16; i += step) __builtin_nontemporal_store(zero, (unaligned_words*)(base + b0) + i);
    if (id < n % 16 / 2) ((uint16_t*)(base + b0 + n / 16 * 16))[id] = 0;
  } else {
    const int row_words = (int)(((int64_t)a.D * esize + 15) / 16);  // the last perhaps in part
    for (int64_t i = id; i < (r1 - r0) * row_words; i += step) {
      char* const row = base + (r0 + i / row_words) * a.ldw * esize;
      const int64_t b = i % row_words * 16, n = (int64_t)a.D * esize - b;
      if (n >= 16) __builtin_nontemporal_store(zero, (unaligned_words*)(row + b));
      else
        for (int k = 0; k < n / 2; ++k) ((uint16_t*)(row + b))[k] = 0;
    }
  }
}

// Up to kEmbedSmall tokens: all passes in the first workgroup, tokens in
// registers between them.  A wave holds `steps` times 64 consecutive tokens.
__global__ void __launch_bounds__(1024) embed_small_sort_kernel(const EmbedGradArgs a, int esize, const FillShare f) {
  constexpr int I = kEmbedSmall / 1024;
  __shared__ uint32_t skey[kEmbedSmall], spos[kEmbedSmall];
  __shared__ uint32_t cnt[16][256];
  __shared__ uint32_t tmp[16];
  if ((int)blockIdx.x >= f.first) {
    fill_share<1024>(a, esize, f);
    return;
  }
  if (threadIdx.x == 0) *a.long_count = 0;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint64_t below = (1ull << lane) - 1;
  const int steps = (a.T + 1023) / 1024;
  const int t0 = wave * (steps * 64) + lane;
  uint32_t key[I], pos[I];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int t = t0 + i * 64;
    key[i] = i < steps && t < a.T ? token_key(a, t) : 0;
    pos[i] = t;
  }
  for (int p = 0; p < a.passes; ++p) {
    const int shift = 8 * p;
    for (int b = threadIdx.x; b < 16 * 256; b += 1024) cnt[b >> 8][b & 255] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < I; ++i)
      if (i < steps && t0 + i * 64 < a.T) atomicAdd(&cnt[wave][(key[i] >> shift) & 255], 1u);  // whole numbers: any order
    __syncthreads();
    uint32_t sum = 0;
    if (threadIdx.x < 256)
#pragma unroll
      for (int w = 0; w < 16; ++w) sum += cnt[w][threadIdx.x];
    uint32_t at = block_scan<1024>(sum, tmp);
    if (threadIdx.x < 256)
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        const uint32_t n = cnt[w][threadIdx.x];
        cnt[w][threadIdx.x] = at;
        at += n;
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < I; ++i) {
      if (i >= steps) break;
      const bool live = t0 + i * 64 < a.T;
      const uint32_t q = wave_place(cnt[wave], (key[i] >> shift) & 255, 8, live, below);
      if (live) {
        skey[q] = key[i];
        spos[q] = pos[i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int t = t0 + i * 64;
      if (i < steps && t < a.T) {
        key[i] = skey[t];
        pos[i] = spos[t];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int t = t0 + i * 64;
    if (i < steps && t < a.T) {
      a.key[0][t] = key[i];
      a.pos[0][t] = pos[i];
    }
  }
}

// More tokens: per pass the digit counts of each workgroup's tokens, their
// running sums over the workgroups, and the move.  (Counting the next pass's
// digits with global atomics during the move is a launch less but slower: the
// frequent ids meet on a few counters.  16 against 8.5 + 5 us at 32768 tokens.)
template <bool FIRST>
__global__ void __launch_bounds__(256) embed_hist_kernel(const EmbedGradArgs a, int pass, int esize,
                                                         const FillShare f) {
  __shared__ uint32_t cnt[1 << kSortMaxBits];
  const int bins = 1 << a.bits, shift = pass * a.bits, src = pass & 1;
  if ((int)blockIdx.x >= f.first) {
    fill_share<256>(a, esize, f);
    return;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.long_count = 0;
  for (int b = threadIdx.x; b < bins; b += 256) cnt[b] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortItems / 256; ++i) {
    const int t = blockIdx.x * kSortItems + i * 256 + threadIdx.x;
    if (t < a.T) atomicAdd(&cnt[((FIRST ? token_key(a, t) : a.key[src][t]) >> shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += 256) a.hist[(int64_t)blockIdx.x * bins + b] = cnt[b];
}

// hist[k][b] becomes the tokens with digit b in workgroups before k; total[b]
// all of them.  64 digits per workgroup, 16 waves with a sixteenth of the k each.
__global__ void __launch_bounds__(1024) embed_scan_kernel(const EmbedGradArgs a, int nblk) {
  __shared__ uint32_t part[16][64];
  uint32_t* const hist = a.hist;
  const int bins = 1 << a.bits;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int b = blockIdx.x * 64 + lane;
  const int lo = (int)((int64_t)nblk * w / 16), hi = (int)((int64_t)nblk * (w + 1) / 16);
  uint32_t sum = 0;
  if (b < bins) {
#pragma unroll 8
    for (int k = lo; k < hi; ++k) sum += hist[(int64_t)k * bins + b];
  }
  part[w][lane] = sum;
  __syncthreads();
  if (b >= bins) return;
  uint32_t at = 0;
  for (int q = 0; q < w; ++q) at += part[q][lane];
  if (w == 15) a.total[b] = at + sum;
  for (int k0 = lo; k0 < hi; k0 += 8) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k0 + i < hi ? hist[(int64_t)(k0 + i) * bins + b] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k0 + i < hi) {
        hist[(int64_t)(k0 + i) * bins + b] = at;
        at += v[i];
      }
  }
}

// Moves each token to its place by the pass's digit; a wave owns consecutive
// tokens and takes them 64 at a time in order, so equal digits keep theirs.
template <bool FIRST>
__global__ void __launch_bounds__(256) embed_scatter_kernel(const EmbedGradArgs a, int pass, int esize,
                                                            const FillShare f) {
  constexpr int I = kSortItems / 256;
  __shared__ uint32_t cnt[4][1 << kSortMaxBits];
  __shared__ uint32_t tmp[4];
  if ((int)blockIdx.x >= f.first) {
    fill_share<256>(a, esize, f);
    return;
  }
  const int bins = 1 << a.bits, shift = pass * a.bits, src = pass & 1;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t0 = blockIdx.x * kSortItems + wave * (I * 64) + lane;
  for (int b = threadIdx.x; b < 4 * bins; b += 256) cnt[b >> a.bits][b & (bins - 1)] = 0;
  __syncthreads();
  uint32_t key[I];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int t = t0 + i * 64;
    key[i] = t < a.T ? (FIRST ? token_key(a, t) : a.key[src][t]) : 0;
    if (t < a.T) atomicAdd(&cnt[wave][(key[i] >> shift) & (bins - 1)], 1u);
  }
  // thread x: digits [x q, x q + q)
  const int q = (bins + 255) / 256, b0 = threadIdx.x * q;
  uint32_t tot[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tot[i] = i < q && b0 + i < bins ? a.total[b0 + i] : 0;
    sum += tot[i];
  }
  uint32_t base = block_scan<256>(sum, tmp);  // its barriers also order the counts above
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = b0 + i;
    if (i < q && b < bins) {
      uint32_t at = base + a.hist[(int64_t)blockIdx.x * bins + b];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t n = cnt[w][b];
        cnt[w][b] = at;
        at += n;
      }
    }
    base += tot[i];
  }
  __syncthreads();
  const uint64_t below = (1ull << lane) - 1;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int t = t0 + i * 64;
    const bool live = t < a.T;
    const uint32_t at = wave_place(cnt[wave], (key[i] >> shift) & (bins - 1), a.bits, live, below);
    if (live) {
      a.key[src ^ 1][at] = key[i];
      a.pos[src ^ 1][at] = FIRST ? (uint32_t)t : a.pos[src][t];
    }
  }
}

// ---------------------------------------------------------------------------
// Sums.  A group of lx lanes holds lx chunks of VEC columns; 256 / lx groups
// per workgroup.
// ---------------------------------------------------------------------------

template <int TY, int VEC>
__device__ __forceinline__ void add_chunk(float (&acc)[VEC], const Chunk<TY, VEC>& v) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] += v.get(i);
}

// Adds tokens pos(lo) .. pos(hi - 1) (dout rows) at column d, in order, U loads at a time.
template <int TY, bool TAIL, int U, class Pos>
__device__ __forceinline__ void add_tokens(const EmbedGradArgs& a, Pos pos, int lo, int hi, int d,
                                           float (&acc)[kWide<TY>]) {
  typedef Chunk<TY, kWide<TY>> C;
  const typename C::raw* base = (const typename C::raw*)a.dout + d;
  int p = lo;
  for (; p + U <= hi; p += U) {
    C v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) v[i].template load<TAIL>(base + (int64_t)pos(p + i) * a.ldg, a.D - d);
#pragma unroll
    for (int i = 0; i < U; ++i) add_chunk(acc, v[i]);
  }
  for (; p < hi; ++p) {
    C v;
    v.template load<TAIL>(base + (int64_t)pos(p) * a.ldg, a.D - d);
    add_chunk(acc, v);
  }
}

// Adds the sums of whole chunks lo .. hi - 1.
template <int VEC, bool TAIL>
__device__ __forceinline__ void add_partials(const EmbedGradArgs& a, int lo, int hi, int d, float (&acc)[VEC]) {
  typedef Chunk<LL_F32, VEC> F;
  const uint32_t* base = (const uint32_t*)a.partial + d;
  int p = lo;
  for (; p + 4 <= hi; p += 4) {
    F v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i].template load<TAIL>(base + (int64_t)(p + i) * a.D, a.D - d);
#pragma unroll
    for (int i = 0; i < 4; ++i) add_chunk(acc, v[i]);
  }
  for (; p < hi; ++p) {
    F v;
    v.template load<TAIL>(base + (int64_t)p * a.D, a.D - d);
    add_chunk(acc, v);
  }
}

// Sum over the workgroup's groups in group order; the first group gets it.
template <int THREADS, int VEC>
__device__ __forceinline__ void groups_sum(float (&red)[THREADS * VEC], int lx_log2, int x, int g,
                                           float (&acc)[VEC]) {
  const int groups = THREADS >> lx_log2;
  __syncthreads();  // red may still be read for the sum before
#pragma unroll
  for (int i = 0; i < VEC; ++i) red[i * THREADS + threadIdx.x] = acc[i];
  __syncthreads();
  if (g == 0) {
    for (int k = 1; k < groups; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += red[i * THREADS + (k << lx_log2) + x];
  }
}

template <int TY, bool TAIL>
__device__ __forceinline__ void write_row(const EmbedGradArgs& a, int64_t v, int d, const float (&acc)[kWide<TY>]) {
  constexpr int VEC = kWide<TY>;
  typedef Chunk<TY, VEC> C;
  typename C::raw* dst = (typename C::raw*)a.dw + v * a.ldw + d;
  C o;
  if (a.accumulate) {
    C old;
    old.template load<TAIL>(dst, a.D - d);
#pragma unroll
    for (int i = 0; i < VEC; ++i) o.put(i, old.get(i) + acc[i] * a.scale);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) o.put(i, acc[i] * a.scale);
  }
  // the gradient is not read again soon (262144 tokens into 1000003 x 64 fp32: 149 -> 109 us)
  o.template store<TAIL, true>(dst, a.D - d);
}

// The first `chunk_blocks` workgroups, in `chunk_cols` shares of the columns, go
// through the chunks of sorted positions: the sum of a chunk that belongs to one row
// whole, and that row's bounds.  The others: the rows without a whole chunk, a
// group from the row's first sorted position, a block of columns at a time.
template <int TY, bool TAIL>
__global__ void __launch_bounds__(256) embed_sums_kernel(const EmbedGradArgs a, int src, int lx_log2, int chunk_blocks,
                                                         int chunk_cols, int col_blocks, int first_block) {
  constexpr int VEC = kWide<TY>;
  __shared__ float red[256 * VEC];
  const uint32_t* key = a.key[src];
  const uint32_t* order = a.pos[src];
  auto pos = [&](int p) { return order[p]; };
  const int lx = 1 << lx_log2;
  const int x = threadIdx.x & (lx - 1), g = threadIdx.x >> lx_log2;
  const int groups = 256 >> lx_log2;
  const int block = first_block + (int)blockIdx.x;
  if (block < chunk_blocks) {
    const int cb = block % chunk_cols, nch = a.T / kEmbedChunk;
    for (int chunk = block / chunk_cols; chunk < nch; chunk += chunk_blocks / chunk_cols) {
      const int p0 = chunk * kEmbedChunk;
      const uint32_t k0 = key[p0];
      if (key[p0 + kEmbedChunk - 1] != k0 || (int64_t)k0 >= a.V) continue;  // uniform
      // the first whole chunk of its row: sorted keys, so the one before is whole if it starts with the same key
      if (cb == 0 && threadIdx.x == 0 && (p0 == 0 || key[p0 - kEmbedChunk] != k0)) {
        int lo = p0;
        while (lo > 0 && key[lo - 1] == k0) --lo;
        int in = p0 + kEmbedChunk - 1, out = a.T;  // last position known to be the row's, first known not to be
        while (in + 1 < out) {
          const int mid = in + (out - in) / 2;
          if (key[mid] == k0) in = mid;
          else out = mid;
        }
        a.long_rows[atomicAdd(a.long_count, 1u)] = int2{lo, out};
      }
      const int per = (kEmbedChunk + groups - 1) / groups;
      const int lo = p0 + min(g * per, kEmbedChunk), hi = p0 + min((g + 1) * per, kEmbedChunk);
      for (uint32_t d0 = cb * lx * VEC; d0 < (uint32_t)a.D; d0 += chunk_cols * lx * VEC) {
        const int d = (int)d0 + x * VEC;
        float acc[VEC] = {};
        if (d < a.D) add_tokens<TY, TAIL, 4>(a, pos, lo, hi, d, acc);
        groups_sum<256>(red, lx_log2, x, g, acc);
        if (g == 0 && d < a.D) {
          Chunk<LL_F32, VEC> o;
  #pragma unroll
          for (int i = 0; i < VEC; ++i) o.put(i, acc[i]);
          o.template store<TAIL>((uint32_t*)a.partial + (int64_t)chunk * a.D + d, a.D - d);
        }
      }
    }
    return;
  }
  // Everything that depends on the position alone is loaded at once; a row of up
  // to four tokens then needs their rows and nothing else.  (Two positions per
  // group at once: more registers, fewer groups in flight, 206 against 195 us.)
  constexpr uint32_t none = 0xFFFFFFFFu;  // no key
  const int item = block - chunk_blocks, cb = item % col_blocks;
  const int p = item / col_blocks * groups + g;
  if (p >= a.T) return;
  const int whole = (p + kEmbedChunk - 1) / kEmbedChunk * kEmbedChunk + kEmbedChunk - 1;
  const uint32_t k = key[p], before = p > 0 ? key[p - 1] : none, in_whole = whole < a.T ? key[whole] : none;
  uint32_t at[4];
  at[0] = order[p];
  int n = 1;  // tokens of the row that starts here, up to four
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    const uint32_t after = p + i < a.T ? key[p + i] : none;
    at[i] = p + i < a.T ? order[p + i] : 0;
    n += n == i && after == k;
  }
  if ((int64_t)k >= a.V || before == k || in_whole == k) return;  // not a row's first, or it holds a whole chunk
  int end = p + n;
  if (n == 4) {  // without a whole chunk, fewer than two chunks: six halvings
    int out = min(p + 2 * kEmbedChunk, a.T);
    for (int in = p + 3; in + 1 < out;) {
      const int mid = in + (out - in) / 2;
      if (key[mid] == k) in = mid;
      else out = mid;
    }
    end = out;
  }
  for (uint32_t d0 = (cb * lx + x) * VEC; d0 < (uint32_t)a.D; d0 += col_blocks * lx * VEC) {
    const int d = (int)d0;
    const typename Elem<TY>::raw* base = (const typename Elem<TY>::raw*)a.dout + d;
    Chunk<TY, VEC> v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i].template load<TAIL>(base + (int64_t)at[i] * a.ldg, a.D - d);
      else v[i].clear();
    float acc[VEC] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) add_chunk(acc, v[i]);
    add_tokens<TY, TAIL, 4>(a, pos, p + n, end, d, acc);
    write_row<TY, TAIL>(a, k, d, acc);
  }
}

// The rows that hold whole chunks, a block of columns at a time: loose tokens
// in front, whole chunks, loose tokens behind, split over the groups of 16 waves
// and joined in their order.
template <int TY, bool TAIL>
__global__ void __launch_bounds__(1024) embed_long_kernel(const EmbedGradArgs a, int src, int lx_log2) {
  constexpr int VEC = kWide<TY>;
  __shared__ float red[1024 * VEC];
  const uint32_t* order = a.pos[src];
  auto pos = [&](int p) { return order[p]; };
  const int lx = 1 << lx_log2;
  const int x = threadIdx.x & (lx - 1), g = threadIdx.x >> lx_log2;
  const int groups = 1024 >> lx_log2;
  const int all_cols = (a.D + lx * VEC - 1) / (lx * VEC);
  const int64_t items = (int64_t)*a.long_count * all_cols;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int2 s = a.long_rows[it / all_cols];
    const int64_t v = a.key[src][s.x];
    const int d = ((int)(it % all_cols) * lx + x) * VEC;
    const int h0 = (s.x + kEmbedChunk - 1) / kEmbedChunk * kEmbedChunk, h1 = s.y / kEmbedChunk * kEmbedChunk;
    const int nh = h0 - s.x, nc = (h1 - h0) / kEmbedChunk, n = nh + nc + (s.y - h1);
    const int lo = (int)((int64_t)n * g / groups), hi = (int)((int64_t)n * (g + 1) / groups);
    float acc[VEC] = {};
    if (d < a.D) {
      add_tokens<TY, TAIL, 4>(a, pos, s.x + lo, s.x + min(hi, nh), d, acc);
      const int k0 = h0 / kEmbedChunk - nh;  // item i is chunk k0 + i
      add_partials<VEC, TAIL>(a, k0 + max(lo, nh), k0 + min(hi, nh + nc), d, acc);
      const int b0 = h1 - nh - nc;           // item i is sorted position b0 + i
      add_tokens<TY, TAIL, 4>(a, pos, b0 + max(lo, nh + nc), b0 + hi, d, acc);
    }
    groups_sum<1024>(red, lx_log2, x, g, acc);
    if (g == 0 && d < a.D) write_row<TY, TAIL>(a, v, d, acc);
  }
}

// Most rows a group handles one after the other.
constexpr int kRowsPerGroup = 8;

// Few tokens: each workgroup picks its rows' tokens from ids itself, orders
// them by (row, position) in LDS, and sums; rows of more than kEmbedChunk
// tokens with all groups together.
template <int TY, bool TAIL>
__global__ void __launch_bounds__(256) embed_few_kernel(const EmbedGradArgs a, int lx_log2, int group_rows,
                                                        int col_blocks) {
  constexpr int VEC = kWide<TY>;
  __shared__ float red[256 * VEC];
  __shared__ uint32_t list[kEmbedDirect], order[kEmbedDirect];
  __shared__ int wcnt[4];
  __shared__ int2 seg[256 * kRowsPerGroup];
  const int lx = 1 << lx_log2;
  const int x = threadIdx.x & (lx - 1), g = threadIdx.x >> lx_log2;
  const int groups = 256 >> lx_log2;
  const int nrows = groups * group_rows;
  const int64_t v0 = (int64_t)(blockIdx.x / col_blocks) * nrows;
  const int cb = blockIdx.x % col_blocks;
  for (int r = threadIdx.x; r < nrows; r += 256) seg[r] = int2{0, 0};
  int n = 0;  // matching tokens so far: local row << 16 | token
  for (int t0 = 0; t0 < a.T; t0 += 256) {
    const int t = t0 + threadIdx.x;
    const uint32_t k = t < a.T ? token_key(a, t) : (uint32_t)a.V;
    const bool hit = (int64_t)k < a.V && (int64_t)k >= v0 && (int64_t)k < v0 + nrows;
    const uint64_t m = __ballot(hit);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (lane == 0) wcnt[wave] = __popcll(m);
    __syncthreads();
    int at = n;
    for (int w = 0; w < wave; ++w) at += wcnt[w];
    if (hit) list[at + __popcll(m & ((1ull << lane) - 1))] = (uint32_t)((int64_t)k - v0) << 16 | (uint32_t)t;
    n += wcnt[0] + wcnt[1] + wcnt[2] + wcnt[3];
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n; i += 256) {
    const uint32_t e = list[i];
    int rank = 0, first = 0, last = 0;
    for (int j = 0; j < n; ++j) {
      const uint32_t f = list[j];
      rank += f < e;
      first += (f >> 16) < (e >> 16);
      last += (f >> 16) <= (e >> 16);
    }
    order[rank] = e & 0xFFFF;
    if (rank == first) seg[e >> 16] = int2{first, last};
  }
  __syncthreads();
  auto pos = [&](int p) { return order[p]; };
  for (uint32_t d0 = cb * lx * VEC; d0 < (uint32_t)a.D; d0 += col_blocks * lx * VEC) {
    const int d = (int)d0 + x * VEC;
    for (int i = 0; i < group_rows; ++i) {
      const int r = i * groups + g;
      const int2 s = seg[r];
      if (v0 + r >= a.V || d >= a.D || s.y - s.x > kEmbedChunk || (a.accumulate && s.y == s.x)) continue;
      float acc[VEC] = {};
      add_tokens<TY, TAIL, 4>(a, pos, s.x, s.y, d, acc);
      write_row<TY, TAIL>(a, v0 + r, d, acc);
    }
    if (n <= kEmbedChunk) continue;
    for (int r = 0; r < nrows; ++r) {  // uniform
      const int2 s = seg[r];
      const int len = s.y - s.x;
      if (len <= kEmbedChunk) continue;
      float acc[VEC] = {};
      if (d < a.D) add_tokens<TY, TAIL, 4>(a, pos, s.x + len * g / groups, s.x + len * (g + 1) / groups, d, acc);
      groups_sum<256>(red, lx_log2, x, g, acc);
      if (g == 0 && d < a.D) write_row<TY, TAIL>(a, v0 + r, d, acc);
    }
  }
}

// Most workgroups of 256 in a launch: a grid of 2^32 threads or more is not supported.
constexpr int64_t kMaxBlocks = (1ll << 32) / 256 - 1;

template <int TY, bool TAIL>
static hipError_t launch_embed_grad_t(const EmbedGradArgs& a, int cus, hipStream_t s) {
  constexpr int VEC = kWide<TY>, ESIZE = (int)sizeof(typename Elem<TY>::raw);
  const int chunks = (a.D + VEC - 1) / VEC;
  const int lx = log2_up(chunks, 6);
  const int groups = 256 >> lx;
  const int all_cols = (chunks + (1 << lx) - 1) >> lx;  // blocks of columns
  if (a.direct) {
    // Fewer rows per group, then workgroups along the columns, until there are
    // 16 workgroups per CU (each scans all ids, so no more than that).
    const int64_t want = 16 * (int64_t)cus;
    const int rows = (int)std::max<int64_t>(1, std::min<int64_t>(kRowsPerGroup, a.V / (groups * want)));
    const int64_t rb = (a.V + groups * rows - 1) / (groups * rows);
    const int cb = (int)std::min<int64_t>(all_cols, std::max<int64_t>(1, want / rb));
    if (rb * cb > kMaxBlocks) return hipErrorInvalidValue;
    hipLaunchKernelGGL((embed_few_kernel<TY, TAIL>), dim3((unsigned)(rb * cb)), dim3(256), 0, s, a, lx, rows, cb);
    return hipGetLastError();
  }
  const int nch = a.T / kEmbedChunk;  // whole chunks
  const int ccb = nch ? (int)std::min<int64_t>(all_cols, std::max<int64_t>(1, 16 * (int64_t)cus / nch)) : 1;
  const int cwg = (int)std::min<int64_t>(nch, std::max<int64_t>(1, 16 * (int64_t)cus / ccb)) * ccb;
  const int64_t sums = cwg + (int64_t)(a.T + groups - 1) / groups * all_cols;
  if (sums > 0x7FFFFFFF) return hipErrorInvalidValue;  // before anything is written
  // 8 KB of zeros per workgroup of 256: two stores per lane (64 KB took 28 us for
  // a share of 134 MB instead of 22, 4 KB 29)
  const int shares = a.T <= kEmbedSmall ? 1 : 2 * a.passes;
  const int64_t share_bytes = a.V * (int64_t)a.D * ESIZE / shares + 1;
  const int fill = a.accumulate ? 0 : (int)std::min<int64_t>((share_bytes + 8191) / 8192, 256 * cus);
  int src = 0;
  if (a.T <= kEmbedSmall) {
    hipLaunchKernelGGL(embed_small_sort_kernel, dim3(1 + (fill + 3) / 4), dim3(1024), 0, s, a, ESIZE,
                       FillShare{1, 0, 1});
  } else {
    const int nblk = (a.T + kSortItems - 1) / kSortItems;
    for (int p = 0; p < a.passes; ++p) {
      const FillShare h = {nblk, 2 * p, shares}, m = {nblk, 2 * p + 1, shares};
      if (p == 0)
        hipLaunchKernelGGL((embed_hist_kernel<true>), dim3(nblk + fill), dim3(256), 0, s, a, p, ESIZE, h);
      else
        hipLaunchKernelGGL((embed_hist_kernel<false>), dim3(nblk + fill), dim3(256), 0, s, a, p, ESIZE, h);
      hipLaunchKernelGGL(embed_scan_kernel, dim3(((1 << a.bits) + 63) / 64), dim3(1024), 0, s, a, nblk);
      if (p == 0)
        hipLaunchKernelGGL((embed_scatter_kernel<true>), dim3(nblk + fill), dim3(256), 0, s, a, p, ESIZE, m);
      else
        hipLaunchKernelGGL((embed_scatter_kernel<false>), dim3(nblk + fill), dim3(256), 0, s, a, p, ESIZE, m);
      src ^= 1;
    }
  }
  for (int64_t first = 0; first < sums; first += kMaxBlocks)
    hipLaunchKernelGGL((embed_sums_kernel<TY, TAIL>), dim3((unsigned)std::min(sums - first, kMaxBlocks)), dim3(256), 0, s,
                       a, src, lx, cwg, ccb, all_cols, (int)first);
  if (nch == 0) return hipGetLastError();
  const int lb = (int)std::min<int64_t>((int64_t)nch * all_cols, 2 * cus);
  hipLaunchKernelGGL((embed_long_kernel<TY, TAIL>), dim3(lb), dim3(1024), 0, s, a, src, lx);
  return hipGetLastError();
}

hipError_t launch_embed_grad(const EmbedGradArgs& a, int type, int cus, hipStream_t s) {
  switch (type) {
    case LL_BF16:
      return a.D % 8 ? launch_embed_grad_t<LL_BF16, true>(a, cus, s) : launch_embed_grad_t<LL_BF16, false>(a, cus, s);
    case LL_F16:
      return a.D % 8 ? launch_embed_grad_t<LL_F16, true>(a, cus, s) : launch_embed_grad_t<LL_F16, false>(a, cus, s);
    case LL_F32:
      return a.D % 4 ? launch_embed_grad_t<LL_F32, true>(a, cus, s) : launch_embed_grad_t<LL_F32, false>(a, cus, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ll
