// Paged attention, head_dim 128, BF16 cache (kernels in paged_attn.cuh).
#include "paged_attn.cuh"

namespace dsa {

cudaError_t launch_paged_attention_128(const AttnParams& p, int grid, int sm_count, cudaStream_t stream) {
  if (p.plan.pair) return attn::launch<128, false, attn::PAIR>(p, grid, sm_count, stream);
  if (p.plan.narrow) return attn::launch<128, false, attn::GATHER, true>(p, grid, sm_count, stream);
  if (p.plan.gather) return attn::launch<128, false, attn::GATHER>(p, grid, sm_count, stream);
  return attn::launch<128, false, attn::SOLO>(p, grid, sm_count, stream);
}

}  // namespace dsa
