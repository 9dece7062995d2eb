// Instantiations of the attention kernel over pages (attn.cuh).
#include "attn.cuh"

namespace idxk {

template <bool BF16>
static cudaError_t pick(const AttnParams& p, int sm_count, cudaStream_t stream) {
  using namespace attn;
  if (p.dim == 64 && p.tile == 16) return launch_one<BF16, 64, 16, 16, 3, false>(p, sm_count, stream);
  if (p.dim == 64 && p.tile == 32) return launch_one<BF16, 64, 32, 12, 3, false>(p, sm_count, stream);
  if (p.dim == 128 && p.tile == 16) return launch_one<BF16, 128, 16, 8, 3, false>(p, sm_count, stream);
  if (p.dim == 128 && p.tile == 32) return launch_one<BF16, 128, 32, 8, 3, false>(p, sm_count, stream);
  if (p.dim == 256 && p.tile == 16) return launch_one<BF16, 256, 16, 4, 3, false>(p, sm_count, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_attn_pages(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream) {
  return bf16 ? pick<true>(p, sm_count, stream) : pick<false>(p, sm_count, stream);
}

}  // namespace idxk
