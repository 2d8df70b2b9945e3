// The tensor-core matrix-vector product for 4-bit codes.
#include "gemv_mma.cuh"

namespace qwha {
cudaError_t launch_gemv_b4(const GemvArgs &a, cudaStream_t s) { return gemv::launch_bits<4>(a, s); }
}  // namespace qwha
