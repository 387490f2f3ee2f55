// 64x128 tiles of the 8-bit product: eight waves of 32x32, six steps in LDS, for up
// to 64 rows, where the bytes of B bound it.
#include "gemm8_tile.hpp"

namespace ll {

hipError_t launch_gemm8_tile64x128(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  return launch_gemm8_tile<G8Cfg<64, 128, 2, 4, 6>, false>(a, a_e5m2, rows, s);
}

}  // namespace ll
