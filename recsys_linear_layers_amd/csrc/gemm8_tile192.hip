// 192x256 tiles of the 8-bit product with C in fp32: eight waves of 96x64, two per
// SIMD.  The widened operands take the registers that 256x256 tiles would need
// for their accumulators (they spilled: 8192 x 8192 x 16384 with row scales 3445 us).
#include "gemm8_tile.hpp"

namespace ll {

hipError_t launch_gemm8_tile192(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  return launch_gemm8_tile<G8Cfg<192, 256, 2, 4>, true>(a, a_e5m2, rows, s);
}

}  // namespace ll
