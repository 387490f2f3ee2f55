// 256x256 tiles of the 8-bit product with a 16-bit C: eight waves of 128x64, two
// per SIMD.
#include "gemm8_tile.hpp"

namespace ll {

hipError_t launch_gemm8_tile256(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  return launch_gemm8_tile<G8Cfg<256, 256, 2, 4>, false>(a, a_e5m2, rows, s);
}

}  // namespace ll
