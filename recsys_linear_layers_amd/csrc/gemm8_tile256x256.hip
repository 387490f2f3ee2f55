// 256x256 tiles of the 8-bit product: eight waves of 128x64, two per SIMD, two steps
// in LDS.
#include "gemm8_tile.hpp"

namespace ll {

hipError_t launch_gemm8_tile256x256(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  return launch_gemm8_tile<G8Cfg<256, 256, 2, 4, 2>, false>(a, a_e5m2, rows, s);
}

}  // namespace ll
