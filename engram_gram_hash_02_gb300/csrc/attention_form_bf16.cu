// The paged attention over a bf16 cache with a form of scores, or joined with the part of a shared prefix (see attention.cuh).
#include "attention.cuh"

namespace engram {

cudaError_t launch_attention_form_bf16(const AttnParams& p, const AttnPlan& plan, int64_t max_tiles, cudaStream_t stream, bool pdl) {
  return attn::launch_any<false, true>(p, plan, max_tiles, stream, pdl);
}

}  // namespace engram
