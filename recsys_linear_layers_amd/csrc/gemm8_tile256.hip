// 256x256 tiles of the 8-bit product: eight waves of 128x64, two per SIMD.
#include "gemm8_tile.hpp"

namespace ll {

hipError_t launch_gemm8_tile256(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  return a.c_type == LL_F32 ? launch_gemm8_tile256_exact(a, a_e5m2, rows, s)
                            : launch_gemm8_tile<G8Cfg<256, 256, 2, 4>, false>(a, a_e5m2, rows, s);
}

}  // namespace ll
