// Attention of prompts over an FP8 cache (see prompt.cuh).
#include "prompt.cuh"

namespace engram {
namespace prompt {

cudaError_t launch_fp8(const Args& a, cudaStream_t stream) { return launch_any<true>(a, stream); }

}  // namespace prompt
}  // namespace engram
