// 128x128 tiles of the 8-bit product: four waves of 64x64, two workgroups per CU.
#include "gemm8_tile.hpp"

namespace ll {

hipError_t launch_gemm8_tile128(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  return a.c_type == LL_F32 ? launch_gemm8_tile<G8Cfg<128, 128, 2, 2>, true>(a, a_e5m2, rows, s)
                            : launch_gemm8_tile<G8Cfg<128, 128, 2, 2>, false>(a, a_e5m2, rows, s);
}

}  // namespace ll
