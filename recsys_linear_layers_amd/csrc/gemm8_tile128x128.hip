// 128x128 tiles of the 8-bit product: eight waves of 64x32, four steps in LDS, one
// workgroup per CU.  (Four waves of 64x64, two steps and two workgroups per CU took
// 31 us where these take 25, at 1024 x 4096 x 4096.)
#include "gemm8_tile.hpp"

namespace ll {

hipError_t launch_gemm8_tile128x128(const Gemm8Args& a, bool a_e5m2, bool rows, hipStream_t s) {
  return launch_gemm8_tile<G8Cfg<128, 128, 2, 4, 4>, false>(a, a_e5m2, rows, s);
}

}  // namespace ll
