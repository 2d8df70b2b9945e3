// The tensor-core products for 3-bit codes.
#include "gemv_mma.cuh"
#include "gemv_wide.cuh"

namespace qwha {
cudaError_t launch_gemv_b3(const GemvArgs &a, cudaStream_t s) {
  return a.npad ? wide::launch_bits<3>(a, s) : gemv::launch_bits<3>(a, s);
}
}  // namespace qwha
