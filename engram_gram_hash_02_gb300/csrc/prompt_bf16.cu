// Attention of prompts over a bf16 cache (see prompt.cuh).
#include "prompt.cuh"

namespace engram {
namespace prompt {

cudaError_t launch_bf16(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_q, const Args& a, cudaStream_t stream) {
  return launch_any<false>(tm_k, tm_v, tm_q, a, stream);
}

}  // namespace prompt
}  // namespace engram
