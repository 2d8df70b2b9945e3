// The tensor-core products for 4-bit codes.
#include "gemv_mma.cuh"
#include "gemv_wide.cuh"

namespace qwha {
cudaError_t launch_gemv_b4(const GemvArgs &a, cudaStream_t s) {
  return a.npad ? wide::launch_bits<4>(a, s) : gemv::launch_bits<4>(a, s);
}
}  // namespace qwha
