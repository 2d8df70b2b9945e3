// The tensor-core matrix-vector product for 2-bit codes.
#include "gemv_mma.cuh"

namespace qwha {
cudaError_t launch_gemv_b2(const GemvArgs &a, cudaStream_t s) { return gemv::launch_bits<2>(a, s); }
}  // namespace qwha
