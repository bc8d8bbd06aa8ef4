// The paged attention over a bf16 cache (see attention.cuh), and the plan both formats share.
#include "attention.cuh"

namespace engram {

AttnPlan attn_plan(int32_t G, int32_t D, bool fp8, int sms) {
  AttnPlan a;
  a.nq = G <= 8 ? 1 : 2;                              // 9 and more heads: 16 per CTA share a row's read
  a.chunks = (G + 8 * a.nq - 1) / (8 * a.nq);
  const int dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  const int ctas = sms * attn::resident_ctas(fp8, dp, a.nq);
  a.tile = attn::kRings * attn::step_keys(fp8, dp, a.nq);
  a.grid_max = ctas < kMaxAttnCtas ? ctas : kMaxAttnCtas;
  a.slot_floats = 8 * a.nq * (dp + 2);
  return a;
}

size_t attn_workspace_bytes(int32_t G, int32_t D, bool fp8, int sms) {
  const AttnPlan a = attn_plan(G, D, fp8, sms);
  return kAttnZeroBytes + (size_t)2 * a.grid_max * a.slot_floats * sizeof(float);
}

cudaError_t launch_attention_bf16(const AttnParams& p, const AttnPlan& plan, int64_t max_tiles, cudaStream_t stream, bool pdl) {
  return attn::launch_any<false>(p, plan, max_tiles, stream, pdl);
}

}  // namespace engram
