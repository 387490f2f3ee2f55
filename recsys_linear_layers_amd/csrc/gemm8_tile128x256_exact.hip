// 128x256 tiles of the 8-bit product with C in fp32.
#include "gemm8_tile.hpp"

namespace ll {

hipError_t launch_gemm8_tile128x256_exact(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  return launch_gemm8_tile<G8Cfg<128, 256, 2, 4, 3>, true>(a, a_e5m2, rows, s);
}

}  // namespace ll
