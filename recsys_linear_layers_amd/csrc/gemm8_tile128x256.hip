// 128x256 tiles of the 8-bit product: eight waves of 64x64, three steps in LDS.
#include "gemm8_tile.hpp"

namespace ll {

hipError_t launch_gemm8_tile128x256(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  return launch_gemm8_tile<G8Cfg<128, 256, 2, 4, 3>, false>(a, a_e5m2, rows, s);
}

}  // namespace ll
