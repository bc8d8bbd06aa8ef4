// The paged attention over an FP8 cache with a form of scores, or joined with the part of a shared prefix (see attention.cuh).
#include "attention.cuh"

namespace engram {

cudaError_t launch_attention_form_fp8(const AttnParams& p, const AttnPlan& plan, int64_t max_tiles, cudaStream_t stream, bool pdl) {
  return attn::launch_any<true, true>(p, plan, max_tiles, stream, pdl);
}

}  // namespace engram
