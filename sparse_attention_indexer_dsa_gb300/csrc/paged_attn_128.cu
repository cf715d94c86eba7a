// Paged attention, head_dim 128, BF16 cache (kernels in paged_attn.cuh).
#include "paged_attn.cuh"

namespace dsa {

cudaError_t launch_paged_attention_128(const AttnParams& p, int grid, int sm_count, cudaStream_t stream) {
  return p.plan.pair ? attn::launch<128, false, true>(p, grid, sm_count, stream)
                     : attn::launch<128, false, false>(p, grid, sm_count, stream);
}

}  // namespace dsa
