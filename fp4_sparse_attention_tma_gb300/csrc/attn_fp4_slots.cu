// Instantiations of the attention kernel over lists of slots of a 4-bit cache (attn_fp4.cuh).
#include "attn_fp4.cuh"

namespace idxk {

cudaError_t launch_attn_fp4_slots(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream) {
  return bf16 ? attn::fp4::pick<true, true>(p, sm_count, stream) : attn::fp4::pick<false, true>(p, sm_count, stream);
}

}  // namespace idxk
