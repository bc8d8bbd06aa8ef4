// Attention of prompts over a bf16 cache (see prompt.cuh).
#include "prompt.cuh"

namespace engram {
namespace prompt {

cudaError_t launch_bf16(const Args& a, cudaStream_t stream) { return launch_any<false>(a, stream); }

}  // namespace prompt
}  // namespace engram
