// Attention of prompts over an FP8 cache (see prompt.cuh).
#include "prompt.cuh"

namespace engram {
namespace prompt {

cudaError_t launch_fp8(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_q, const Args& a, cudaStream_t stream) {
  return launch_any<true>(tm_k, tm_v, tm_q, a, stream);
}

}  // namespace prompt
}  // namespace engram
