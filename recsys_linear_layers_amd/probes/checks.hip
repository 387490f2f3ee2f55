// Checks of the kernels' own steps (include/llchecks.h).
#include "../../include/llchecks.h"

#include <algorithm>

#include "../csrc/quant8.hpp"

namespace {

template <int Q>
__global__ void __launch_bounds__(256) scale8_kernel(uint32_t first, int64_t n, float* scale, float* inv) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const ll::Scale8 s = ll::scale8<Q>(first + (uint32_t)i);
    scale[i] = s.scale;
    inv[i] = s.inv;
  }
}

}  // namespace

extern "C" int ll_check_scale8(int q_type, uint32_t first, int64_t n, float* scale, float* inv, void* stream) {
  if ((q_type != LL_E4M3 && q_type != LL_E5M2) || n < 0 || n > (1ll << 31) || (int64_t)first + n > (1ll << 31)) return -1;
  if (n == 0) return 0;
  if (!scale || !inv || ((uintptr_t)scale & 3) || ((uintptr_t)inv & 3)) return -1;
  const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, 1 << 16);
  if (q_type == LL_E4M3)
    scale8_kernel<LL_E4M3><<<grid, 256, 0, (hipStream_t)stream>>>(first, n, scale, inv);
  else
    scale8_kernel<LL_E5M2><<<grid, 256, 0, (hipStream_t)stream>>>(first, n, scale, inv);
  return (int)hipGetLastError();
}
