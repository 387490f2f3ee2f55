// Device helpers of the cross entropy's row kernels.
#pragma once

#include "ops_common.hpp"
#include "xent.hpp"

namespace ll {

constexpr float kNegInf = -__builtin_huge_valf();

// (m, s) joined with (m2, s2).  An empty or all -inf piece is (-inf, 0).
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float M = fmaxf(m, m2);
  s = (m == M ? s : s * __expf(m - M)) + (m2 == M ? s2 : s2 * __expf(m2 - M));
  m = M;
}

__device__ __forceinline__ bool has_target(const XentRows& r, int64_t t) { return t >= 0 && t < r.V && t != r.ignore; }

}  // namespace ll
