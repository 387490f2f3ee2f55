// Embedding lookup out[t] = scale * table[ids[t]] and its gradient
// dw[v] = scale * (sum of dout[t] over the tokens t with ids[t] == v).
//
// The lookup reads and writes each row once: HBM bound.
//
// The gradient sorts the tokens by id (a stable radix sort of (id, position)
// pairs, so a row's tokens stay in their order) and then every row of dw is
// written once, by the lanes that own it, as the sum of its tokens in that
// order: no floating-point atomics, so the result does not depend on timing.
// A few ids take a large share of the positions in real data.  A row's tokens
// are consecutive after the sort, so sums over whole chunks of kEmbedChunk
// sorted positions are formed ahead (in parallel over the chunks), and a long
// row is then the sum of its chunks and the loose tokens at both ends, split
// over the groups of a workgroup.
#include "embed.hpp"

#include <algorithm>

#include "ops_common.hpp"

namespace ll {

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------

// lx lanes move one row; 256 / lx rows per workgroup and step.
template <int TY, int VEC>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedArgs a, int lx_log2) {
  typedef Chunk<TY, VEC> C;
  const int lx = 1 << lx_log2;
  const int x = threadIdx.x & (lx - 1), y = threadIdx.x >> lx_log2;
  const int rows = 256 >> lx_log2;
  const int chunks = a.D / VEC;
  for (int64_t t = (int64_t)blockIdx.x * rows + y; t < a.T; t += (int64_t)gridDim.x * rows) {
    const int64_t id = a.ids[t];
    C* dst = (C*)((typename Elem<TY>::raw*)a.out + t * a.ldo);
    if (id < 0 || id >= a.V) {
      C z;
#pragma unroll
      for (int i = 0; i < VEC; ++i) z.put(i, 0.f);
      for (int c = x; c < chunks; c += lx) dst[c] = z;
      continue;
    }
    const C* src = (const C*)((const typename Elem<TY>::raw*)a.table + id * a.ldt);
    for (int c = x; c < chunks; c += lx) {
      C v = src[c];
#pragma unroll
      for (int i = 0; i < VEC; ++i) v.put(i, v.get(i) * a.scale);
      dst[c] = v;
    }
  }
}

// Smallest power of two >= n, at most `most`, as its logarithm.
static int log2_up(int64_t n, int most_log2) {
  int l = 0;
  while (l < most_log2 && (1ll << l) < n) ++l;
  return l;
}

template <int TY, int VEC>
static hipError_t launch_embed_t(const EmbedArgs& a, hipStream_t s) {
  const int lx = log2_up(a.D / VEC, 8);
  const int rows = 256 >> lx;
  const int64_t blocks = std::min<int64_t>((a.T + rows - 1) / rows, 1 << 16);
  hipLaunchKernelGGL((embed_kernel<TY, VEC>), dim3((unsigned)blocks), dim3(256), 0, s, a, lx);
  return hipGetLastError();
}

hipError_t launch_embed(const EmbedArgs& a, int type, hipStream_t s) {
  const bool wide = wide_rows(a.table, a.ldt, a.D, type) && wide_rows(a.out, a.ldo, a.D, type);
  switch (type) {
    case LL_BF16: return wide ? launch_embed_t<LL_BF16, 8>(a, s) : launch_embed_t<LL_BF16, 1>(a, s);
    case LL_F16: return wide ? launch_embed_t<LL_F16, 8>(a, s) : launch_embed_t<LL_F16, 1>(a, s);
    case LL_F32: return wide ? launch_embed_t<LL_F32, 4>(a, s) : launch_embed_t<LL_F32, 1>(a, s);
    default: return hipErrorInvalidValue;
  }
}

// ---------------------------------------------------------------------------
// Stable radix sort of (id, position).  Tokens without a gradient (padding or
// an id outside the table) get the key V and end up behind all others.
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t token_key(const EmbedGradArgs& a, int t) {
  const int64_t id = a.ids[t];
  return (id < 0 || id >= a.V || id == a.padding) ? (uint32_t)a.V : (uint32_t)id;
}

template <bool FIRST>
__device__ __forceinline__ uint32_t sort_key(const EmbedGradArgs& a, int src, int t) {
  return FIRST ? token_key(a, t) : a.key[src][t];
}

// Digit counts of each sort workgroup's tokens; the workgroups beyond them
// clear seg (first pass only).
template <bool FIRST>
__global__ void __launch_bounds__(256) embed_hist_kernel(const EmbedGradArgs a, int src, int shift, int nblk) {
  __shared__ uint32_t cnt[1 << kSortMaxBits];
  const int bins = 1 << a.bits;
  if (FIRST && (int)blockIdx.x >= nblk) {
    const int64_t n = a.V;
    for (int64_t i = (int64_t)(blockIdx.x - nblk) * 256 + threadIdx.x; i < n; i += (int64_t)(gridDim.x - nblk) * 256)
      a.seg[i] = int2{0, 0};
    return;
  }
  for (int b = threadIdx.x; b < bins; b += 256) cnt[b] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * kSortItems;
#pragma unroll
  for (int i = 0; i < kSortItems / 256; ++i) {
    const int t = t0 + i * 256 + threadIdx.x;
    if (t < a.T) atomicAdd(&cnt[(sort_key<FIRST>(a, src, t) >> shift) & (bins - 1)], 1u);  // whole numbers: any order
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += 256) a.hist[(int64_t)blockIdx.x * bins + b] = cnt[b];
}

// hist[k][b] becomes the first sorted position of workgroup k's tokens with
// digit b.  One workgroup, thread b for digit b.
__global__ void __launch_bounds__(1024) embed_scan_kernel(uint32_t* hist, int nblk, int bins) {
  __shared__ uint32_t tot[1024];
  const int b = threadIdx.x;
  uint32_t sum = 0;
  if (b < bins) {
#pragma unroll 8
    for (int k = 0; k < nblk; ++k) sum += hist[(int64_t)k * bins + b];
  }
  tot[b] = sum;
  __syncthreads();
  for (int d = 1; d < 1024; d <<= 1) {
    const uint32_t v = b >= d ? tot[b - d] : 0;
    __syncthreads();
    tot[b] += v;
    __syncthreads();
  }
  if (b >= bins) return;
  uint32_t at = tot[b] - sum;
  for (int k0 = 0; k0 < nblk; k0 += 8) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k0 + i < nblk ? hist[(int64_t)(k0 + i) * bins + b] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k0 + i < nblk) {
        hist[(int64_t)(k0 + i) * bins + b] = at;
        at += v[i];
      }
  }
}

// Moves each token to its sorted position.  A wave owns 512 consecutive
// tokens and takes them 64 at a time in order, so equal digits keep their
// order: lanes with the same digit find each other with one ballot per digit
// bit, and the count of that digit so far is kept per wave in LDS.
template <bool FIRST>
__global__ void __launch_bounds__(256) embed_scatter_kernel(const EmbedGradArgs a, int src, int shift) {
  __shared__ uint32_t cnt[4][1 << kSortMaxBits];
  const int bins = 1 << a.bits;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t0 = blockIdx.x * kSortItems + wave * (kSortItems / 4);
  for (int b = threadIdx.x; b < 4 * bins; b += 256) cnt[b >> a.bits][b & (bins - 1)] = 0;
  __syncthreads();
  uint32_t key[kSortItems / 256];
#pragma unroll
  for (int i = 0; i < kSortItems / 256; ++i) {
    const int t = t0 + i * 64 + lane;
    key[i] = t < a.T ? sort_key<FIRST>(a, src, t) : 0;
    if (t < a.T) atomicAdd(&cnt[wave][(key[i] >> shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += 256) {
    uint32_t at = a.hist[(int64_t)blockIdx.x * bins + b];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t n = cnt[w][b];
      cnt[w][b] = at;
      at += n;
    }
  }
  __syncthreads();
  const uint64_t below = (1ull << lane) - 1;
#pragma unroll
  for (int i = 0; i < kSortItems / 256; ++i) {
    const int t = t0 + i * 64 + lane;
    const bool live = t < a.T;
    const uint32_t d = (key[i] >> shift) & (bins - 1);
    uint64_t peers = __ballot(live);
    for (int k = 0; k < a.bits; ++k) {
      const uint64_t set = __ballot((d >> k) & 1);
      peers &= ((d >> k) & 1) ? set : ~set;
    }
    const uint32_t rank = (uint32_t)__popcll(peers & below);
    uint32_t at = 0;
    if (live) {
      at = cnt[wave][d] + rank;
      a.key[src ^ 1][at] = key[i];
      a.pos[src ^ 1][at] = FIRST ? (uint32_t)t : a.pos[src][t];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (live && rank == 0) cnt[wave][d] += (uint32_t)__popcll(peers);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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

// Adds tokens pos[lo .. hi) (dout rows) at column chunk c, in order, four loads at a time.
template <int TY, int VEC, class Pos>
__device__ __forceinline__ void add_tokens(const EmbedGradArgs& a, Pos pos, int lo, int hi, int c,
                                           float (&acc)[VEC]) {
  typedef Chunk<TY, VEC> C;
  const typename Elem<TY>::raw* base = (const typename Elem<TY>::raw*)a.dout;
  int p = lo;
  for (; p + 4 <= hi; p += 4) {
    C v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ((const C*)(base + (int64_t)pos[p + i] * a.ldg))[c];
#pragma unroll
    for (int i = 0; i < 4; ++i) add_chunk<TY, VEC>(acc, v[i]);
  }
  for (; p < hi; ++p) add_chunk<TY, VEC>(acc, ((const C*)(base + (int64_t)pos[p] * a.ldg))[c]);
}

// Adds the sums of whole chunks lo .. hi.
template <int VEC>
__device__ __forceinline__ void add_partials(const EmbedGradArgs& a, int lo, int hi, int c, float (&acc)[VEC]) {
  typedef Chunk<LL_F32, VEC> F;
  int p = lo;
  for (; p + 4 <= hi; p += 4) {
    F v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ((const F*)(a.partial + (int64_t)(p + i) * a.D))[c];
#pragma unroll
    for (int i = 0; i < 4; ++i) add_chunk<LL_F32, VEC>(acc, v[i]);
  }
  for (; p < hi; ++p) add_chunk<LL_F32, VEC>(acc, ((const F*)(a.partial + (int64_t)p * a.D))[c]);
}

// Sum over the workgroup's groups in group order; the first group gets it.
// red holds 256 * VEC floats.
template <int VEC>
__device__ __forceinline__ void groups_sum(float* red, int lx_log2, int x, int g, float (&acc)[VEC]) {
  const int groups = 256 >> lx_log2;
  __syncthreads();  // red may still be read for the sum before
#pragma unroll
  for (int i = 0; i < VEC; ++i) red[i * 256 + threadIdx.x] = acc[i];
  __syncthreads();
  if (g == 0) {
    for (int k = 1; k < groups; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += red[i * 256 + (k << lx_log2) + x];
  }
}

// Row bounds in the sorted order, and the sums of the chunks of sorted
// positions that belong to one row whole.
template <int TY, int VEC>
__global__ void __launch_bounds__(256) embed_chunk_kernel(const EmbedGradArgs a, int src, int lx_log2) {
  __shared__ float red[256 * VEC];
  const uint32_t* key = a.key[src];
  const int p0 = blockIdx.x * kEmbedChunk;
  if (blockIdx.y == 0 && threadIdx.x < kEmbedChunk) {
    const int p = p0 + threadIdx.x;
    if (p < a.T) {
      const uint32_t k = key[p];
      if ((int64_t)k < a.V) {
        if (p == 0 || key[p - 1] != k) a.seg[k].x = p;
        if (p == a.T - 1 || key[p + 1] != k) a.seg[k].y = p + 1;
      }
    }
  }
  if (p0 + kEmbedChunk > a.T) return;
  const uint32_t k0 = key[p0];
  if (key[p0 + kEmbedChunk - 1] != k0 || (int64_t)k0 >= a.V) return;  // uniform
  const int lx = 1 << lx_log2;
  const int x = threadIdx.x & (lx - 1), g = threadIdx.x >> lx_log2;
  const int groups = 256 >> lx_log2;
  const int chunks = a.D / VEC;
  const int per = (kEmbedChunk + groups - 1) / groups;
  for (int c0 = blockIdx.y * lx; c0 < chunks; c0 += gridDim.y * lx) {
    const int c = c0 + x;
    float acc[VEC] = {};
    if (c < chunks)
      add_tokens<TY, VEC>(a, a.pos[src], p0 + min(g * per, kEmbedChunk), p0 + min((g + 1) * per, kEmbedChunk), c, acc);
    groups_sum<VEC>(red, lx_log2, x, g, acc);
    if (g == 0 && c < chunks) {
      Chunk<LL_F32, VEC> o;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o.put(i, acc[i]);
      ((Chunk<LL_F32, VEC>*)(a.partial + (int64_t)blockIdx.x * a.D))[c] = o;
    }
  }
}

template <int TY, int VEC>
__device__ __forceinline__ void write_row(const EmbedGradArgs& a, int64_t v, int c, const float (&acc)[VEC]) {
  typedef Chunk<TY, VEC> C;
  C* dst = (C*)((typename Elem<TY>::raw*)a.dw + v * a.ldw) + c;
  C o;
  if (a.accumulate) {
    const C old = *dst;
#pragma unroll
    for (int i = 0; i < VEC; ++i) o.put(i, old.get(i) + acc[i] * a.scale);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) o.put(i, acc[i] * a.scale);
  }
  *dst = o;
}

// Rows a group handles one after the other.
constexpr int kRowsPerGroup = 8;

// The rows of dw: a group sums a row of up to kEmbedChunk tokens by itself;
// the groups share the longer ones.  DIRECT (few tokens): the workgroup first
// picks its rows' tokens from ids and orders them by (row, position) in LDS.
template <int TY, int VEC, bool DIRECT>
__global__ void __launch_bounds__(256) embed_rows_kernel(const EmbedGradArgs a, int src, int lx_log2) {
  __shared__ float red[256 * VEC];
  __shared__ uint32_t list[DIRECT ? kEmbedDirect : 1], order[DIRECT ? kEmbedDirect : 1];
  __shared__ int wcnt[4];
  __shared__ int2 seg[256 * kRowsPerGroup];
  const int lx = 1 << lx_log2;
  const int x = threadIdx.x & (lx - 1), g = threadIdx.x >> lx_log2;
  const int groups = 256 >> lx_log2;
  const int nrows = groups * kRowsPerGroup;
  const int64_t v0 = (int64_t)blockIdx.x * nrows;
  const int chunks = a.D / VEC;
  if constexpr (DIRECT) {
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
  } else {
    for (int r = threadIdx.x; r < nrows; r += 256) seg[r] = v0 + r < a.V ? a.seg[v0 + r] : int2{0, 0};
  }
  __syncthreads();
  auto pos = [&](int p) { return DIRECT ? order[p] : a.pos[src][p]; };
  struct PosOf {
    decltype(pos)& f;
    __device__ uint32_t operator[](int p) const { return f(p); }
  } posof{pos};
  for (int c0 = blockIdx.y * lx; c0 < chunks; c0 += gridDim.y * lx) {
    const int c = c0 + x;
    for (int i = 0; i < kRowsPerGroup; ++i) {
      const int r = i * groups + g;
      const int64_t v = v0 + r;
      const int2 s = seg[r];
      if (v >= a.V || c >= chunks || s.y - s.x > kEmbedChunk || (a.accumulate && s.y == s.x)) continue;
      float acc[VEC] = {};
      add_tokens<TY, VEC>(a, posof, s.x, s.y, c, acc);
      write_row<TY, VEC>(a, v, c, acc);
    }
    for (int r = 0; r < nrows; ++r) {  // long rows, all groups together (uniform)
      const int2 s = seg[r];
      if (s.y - s.x <= kEmbedChunk) continue;
      // loose tokens in front, whole chunks, loose tokens behind
      int h0 = s.y, h1 = s.y;
      if (!DIRECT) {
        h0 = (s.x + kEmbedChunk - 1) / kEmbedChunk * kEmbedChunk;
        h1 = s.y / kEmbedChunk * kEmbedChunk;
        if (h0 >= h1) h0 = h1 = s.y;
      }
      const int nh = h0 - s.x, nc = (h1 - h0) / kEmbedChunk, n = nh + nc + (s.y - h1);
      const int lo = (int)((int64_t)n * g / groups), hi = (int)((int64_t)n * (g + 1) / groups);
      float acc[VEC] = {};
      if (c < chunks) {
        add_tokens<TY, VEC>(a, posof, s.x + lo, s.x + min(hi, nh), c, acc);
        if (nc > 0) {
          const int k0 = h0 / kEmbedChunk - nh;  // item i is chunk k0 + i
          add_partials<VEC>(a, k0 + max(lo, nh), k0 + min(hi, nh + nc), c, acc);
        }
        const int b0 = h1 - nh - nc;             // item i is sorted position b0 + i
        add_tokens<TY, VEC>(a, posof, b0 + max(lo, nh + nc), b0 + hi, c, acc);
      }
      groups_sum<VEC>(red, lx_log2, x, g, acc);
      if (g == 0 && c < chunks) write_row<TY, VEC>(a, v0 + r, c, acc);
    }
  }
}

template <int TY, int VEC>
static hipError_t launch_embed_grad_t(const EmbedGradArgs& a, int cus, hipStream_t s) {
  const int chunks = a.D / VEC;
  const int lx = log2_up(chunks, 6);
  const int nrows = (256 >> lx) * kRowsPerGroup;
  const int64_t rb = (a.V + nrows - 1) / nrows;
  if (rb > 0x7FFFFFFF) return hipErrorInvalidValue;
  // workgroups along the columns only where the rows alone are few
  const int cb_all = (chunks + (1 << lx) - 1) >> lx;
  const int cb = (int)std::min<int64_t>(cb_all, std::max<int64_t>(1, 16 * (int64_t)cus / rb));
  int src = 0;
  if (a.T > kEmbedDirect) {
    const int nblk = (a.T + kSortItems - 1) / kSortItems;
    const int clear = (int)std::min<int64_t>((a.V + 1023) / 1024, 4 * cus);
    for (int p = 0; p < a.passes; ++p) {
      const int shift = p * a.bits;
      if (p == 0)
        hipLaunchKernelGGL((embed_hist_kernel<true>), dim3(nblk + clear), dim3(256), 0, s, a, src, shift, nblk);
      else
        hipLaunchKernelGGL((embed_hist_kernel<false>), dim3(nblk), dim3(256), 0, s, a, src, shift, nblk);
      hipLaunchKernelGGL(embed_scan_kernel, dim3(1), dim3(1024), 0, s, a.hist, nblk, 1 << a.bits);
      if (p == 0)
        hipLaunchKernelGGL((embed_scatter_kernel<true>), dim3(nblk), dim3(256), 0, s, a, src, shift);
      else
        hipLaunchKernelGGL((embed_scatter_kernel<false>), dim3(nblk), dim3(256), 0, s, a, src, shift);
      src ^= 1;
    }
    const int nch = (a.T + kEmbedChunk - 1) / kEmbedChunk;
    const int ccb = (int)std::min<int64_t>(cb_all, std::max<int64_t>(1, 16 * (int64_t)cus / nch));
    hipLaunchKernelGGL((embed_chunk_kernel<TY, VEC>), dim3(nch, ccb), dim3(256), 0, s, a, src, lx);
    hipLaunchKernelGGL((embed_rows_kernel<TY, VEC, false>), dim3((unsigned)rb, cb), dim3(256), 0, s, a, src, lx);
  } else {
    hipLaunchKernelGGL((embed_rows_kernel<TY, VEC, true>), dim3((unsigned)rb, cb), dim3(256), 0, s, a, 0, lx);
  }
  return hipGetLastError();
}

hipError_t launch_embed_grad(const EmbedGradArgs& a, int type, int cus, hipStream_t s) {
  const bool wide = wide_rows(a.dout, a.ldg, a.D, type) && wide_rows(a.dw, a.ldw, a.D, type);
  switch (type) {
    case LL_BF16: return wide ? launch_embed_grad_t<LL_BF16, 8>(a, cus, s) : launch_embed_grad_t<LL_BF16, 1>(a, cus, s);
    case LL_F16: return wide ? launch_embed_grad_t<LL_F16, 8>(a, cus, s) : launch_embed_grad_t<LL_F16, 1>(a, cus, s);
    case LL_F32: return wide ? launch_embed_grad_t<LL_F32, 4>(a, cus, s) : launch_embed_grad_t<LL_F32, 1>(a, cus, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ll
