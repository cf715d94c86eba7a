// Paged attention, head_dim 64, BF16 cache (kernels in paged_attn.cuh).
#include "paged_attn.cuh"

namespace dsa {

cudaError_t launch_paged_attention_64(const AttnParams& p, int grid, int sm_count, cudaStream_t stream) {
  return p.plan.pair ? attn::launch<64, false, true>(p, grid, sm_count, stream)
                     : attn::launch<64, false, false>(p, grid, sm_count, stream);
}

}  // namespace dsa
