// Embedding lookup and its gradient: arguments and launches (embed.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ll {

struct EmbedArgs {
  const void* table;
  const int64_t* ids;
  void* out;
  int64_t V, ldt, ldo;
  int32_t T, D;
  float scale;
};

// Sorted positions per chunk; a chunk that belongs to one row whole is summed
// once, ahead of the rows.
constexpr int kEmbedChunk = 16;
// Tokens up to which the rows find their tokens by themselves, without a sort,
constexpr int kEmbedDirect = 512;
// as long as the zeros are not most of the work (they go out faster as one run:
// us direct / sorted, 19 tokens into 116319 x 1302 fp32 189 / 110, 300 into
// 50000 x 4096 bf16 80 / 68, one into 131072 x 512 bf16 25.3 / 26.0, 100 into
// 20000 x 512 fp32 10.9 / 15.8),
constexpr int64_t kEmbedDirectBytes = 128ll << 20;
// and up to which one workgroup sorts them in LDS.
constexpr int kEmbedSmall = 8192;
// Tokens per workgroup of the sort beyond that, and its most digit bits per pass.
constexpr int kSortItems = 1024;
constexpr int kSortMaxBits = 10;

struct EmbedGradArgs {
  const int64_t* ids;
  const void* dout;
  void* dw;
  int64_t V, ldg, ldw;
  int64_t padding;  // id without a gradient, or -1
  int32_t T, D;
  int32_t accumulate;
  float scale;
  int32_t direct;   // the rows find their tokens by themselves, no workspace
  // workspace (null when direct)
  uint32_t* key[2];
  uint32_t* pos[2];
  uint32_t* hist;       // [sort workgroups][1 << bits]
  uint32_t* total;      // [1 << bits]
  float* partial;       // [T / kEmbedChunk][D] sums of whole chunks
  uint32_t* long_count; // rows that hold a whole chunk, in any order:
  int2* long_rows;      // their sorted positions first, last + 1
  int32_t bits, passes; // digits; 8 bits where one workgroup sorts
};

hipError_t launch_embed(const EmbedArgs& a, int type, hipStream_t s);
hipError_t launch_embed_grad(const EmbedGradArgs& a, int type, int cus, hipStream_t s);

}  // namespace ll
