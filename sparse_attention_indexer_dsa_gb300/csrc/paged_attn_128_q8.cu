// Paged attention, head_dim 128, 8-bit cache (kernels in paged_attn.cuh).
#include "paged_attn.cuh"

namespace dsa {

cudaError_t launch_paged_attention_128_q8(const AttnParams& p, int grid, int sm_count, cudaStream_t stream) {
  return p.plan.pair ? attn::launch<128, true, true>(p, grid, sm_count, stream)
                     : attn::launch<128, true, false>(p, grid, sm_count, stream);
}

}  // namespace dsa
