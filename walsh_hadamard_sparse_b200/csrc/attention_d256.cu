// Attention over the quantized cache: heads of up to 256 channels.
#include "attention_mma.cuh"

namespace qwha {

cudaError_t launch_attention_d256(const AttnArgs &a, const MmaLaunch &l, cudaStream_t s) {
  if (l.nt == 1) return attn::launch_mma_nt<256, 1>(a, l, s);
  return attn::launch_mma_nt<256, 2>(a, l, s);
}

}  // namespace qwha
