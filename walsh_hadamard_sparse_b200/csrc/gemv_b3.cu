// The tensor-core matrix-vector product for 3-bit codes.
#include "gemv_mma.cuh"

namespace qwha {
cudaError_t launch_gemv_b3(const GemvArgs &a, cudaStream_t s) { return gemv::launch_bits<3>(a, s); }
}  // namespace qwha
