// Instantiations of the tensor-core attention kernel (attn_tc.cuh).
#include "attn_tc.cuh"

namespace idxk {

template <bool BF16>
static cudaError_t pick(const AttnParams& p, int sm_count, cudaStream_t stream) {
  using namespace attn;
  if (p.slots) return tc::launch<BF16, 1, true>(p, sm_count, stream);
  if (p.tile == 2 * tc::kCols) return tc::launch<BF16, 2, false>(p, sm_count, stream);
  return tc::launch<BF16, 1, false>(p, sm_count, stream);
}

cudaError_t launch_attn_tc(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream) {
  return bf16 ? pick<true>(p, sm_count, stream) : pick<false>(p, sm_count, stream);
}

}  // namespace idxk
