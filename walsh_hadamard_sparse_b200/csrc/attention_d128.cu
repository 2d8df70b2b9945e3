// Attention over the quantized cache: heads of up to 128 channels.
#include "attention_mma.cuh"

namespace qwha {

cudaError_t launch_attention_d128(const AttnArgs &a, const MmaLaunch &l, cudaStream_t s) {
  if (l.nt == 1) return attn::launch_mma_nt<128, 1>(a, l, s);
  if (l.nt == 2) return attn::launch_mma_nt<128, 2>(a, l, s);
  return attn::launch_mma_nt<128, 4>(a, l, s);
}

}  // namespace qwha
