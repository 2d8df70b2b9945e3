// The tensor-core products for 2-bit codes.
#include "gemv_mma.cuh"
#include "gemv_wide.cuh"

namespace qwha {
cudaError_t launch_gemv_b2(const GemvArgs &a, cudaStream_t s) {
  return a.npad ? wide::launch_bits<2>(a, s) : gemv::launch_bits<2>(a, s);
}
}  // namespace qwha
