// Attention of all new tokens of ragged sequences over the paged cache: a warp per row and head, key after key.
#include "attn.cuh"

namespace engram {
namespace {

__global__ void __launch_bounds__(256) prompt_kernel(const PromptParams p) {
  const int lane = threadIdx.x & 31;
  const int Hq = p.Hk * p.G;
  pdl_wait();
  if (blockIdx.x == 0 && p.err != nullptr)
    for (int b = threadIdx.x; b < p.B; b += 256) {
      const int s0 = __ldcg(p.cu + b), s1 = __ldcg(p.cu + b + 1), len = __ldcg(p.lens + b);
      if (s0 < 0 || s0 > p.T || s1 > p.T || s1 < s0 || len < 0 || len > p.cap) atomicOr(p.err, ENGRAM_ERR_SEQ_LEN);
    }
  const int64_t warps = (int64_t)gridDim.x * 8;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < p.T * Hq; w += warps) {
    const int64_t t = w / Hq;
    const int h = (int)(w % Hq), kh = h / p.G;
    int lo_b = 0, hi_b = p.B;                          // the last sequence that starts at t or before
    while (hi_b - lo_b > 1) {
      const int mid = (lo_b + hi_b) / 2;
      (__ldcg(p.cu + mid) <= t ? lo_b : hi_b) = mid;
    }
    const int b = lo_b;
    const int64_t s0 = p.B > 0 ? max(__ldcg(p.cu + b), 0) : 0, s1 = p.B > 0 ? min((int64_t)__ldcg(p.cu + b + 1), p.T) : 0;
    const bool mine = p.B > 0 && t >= s0 && t < s1;
    if (!mine && p.out != nullptr) continue;
    int lo = 0, hi = 0, pos = 0;
    if (mine) {
      int len = __ldcg(p.lens + b);
      len = min(max(len, 0), p.cap);
      if (p.own_lens != nullptr) {
        pos = len + min(max(__ldcg(p.own_lens + t), 0), p.own_cap) - 1;
        hi = len;
      } else {
        pos = len - (int)(s1 - t);
        if (len < s1 - s0 && p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_SEQ_LEN);
        hi = p.causal ? min(len, max(pos + 1, p.prefix_ends != nullptr ? __ldcg(p.prefix_ends + t) : 0)) : len;
        if (p.window > 0) lo = max(lo, pos + 1 - p.window);
        if (p.doc_starts != nullptr) lo = max(lo, __ldcg(p.doc_starts + t));
      }
    }
    const float slope = p.form.slopes != nullptr ? p.form.slopes[h] * 1.44269504f : 0.f;
    const uint16_t* q = static_cast<const uint16_t*>(p.q.data) + t * p.q.ts + (int64_t)h * p.q.hs;
    float x[8], o[8], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = lane + 32 * i < p.D ? __uint_as_float((uint32_t)q[lane + 32 * i] << 16) : 0.f;
      o[i] = 0.f;
    }
    for (int j = lo; j < hi; ++j) {
      const int n = (int)fast_div((uint32_t)j, p.cache.div_page), at = j - n * p.cache.page_size;
      const int page = p.table[(int64_t)b * p.table_stride + n];
      if (page < 0 || page >= p.cache.num_pages) {
        if (p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_PAGE);
        continue;
      }
      const int64_t row = page * p.cache.page_b + kh * p.cache.head_b + at * p.cache.tok_b;
      const int64_t srow = page * p.cache.spage_b + kh * p.cache.shead_b + at * p.cache.stok_b;
      auto value = [&](const uint8_t* base, const uint8_t* scales, int d) {
        if (!p.cache.fp8) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base + row)[d] << 16);
        uint32_t a, c;
        e4m3x4_to_f16x2(base[row + d], a, c);
        return __low2float(*reinterpret_cast<const __half2*>(&a)) * __uint_as_float((uint32_t)scales[srow + d / 32] << 23);
      };
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (lane + 32 * i < p.D) s += x[i] * value(p.cache.k, p.cache.ks, lane + 32 * i);
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
      s *= p.scale_log2;
      if (p.form.cap2 > 0.f) s = capped(s, p.form.cap2, p.form.cap_inv);
      s -= slope * (float)abs(pos - j);
      const float mn = fmaxf(m, s);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float f = ex2(m - base), e = ex2(s - base);
      m = mn;
      l = l * f + e;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (lane + 32 * i < p.D) o[i] = o[i] * f + e * value(p.cache.v, p.cache.vs, lane + 32 * i);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l, sum = l == 0.f ? -INFINITY : m + log2f(l);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = lane + 32 * i;
      if (d >= p.D) continue;
      if (p.out != nullptr)
        p.out[t * p.out_ts + (int64_t)h * p.out_hs + d] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] * inv));
      else
        p.prior_o[(t * Hq + h) * p.D + d] = o[i] * inv;
    }
    if (lane == 0) {
      if (p.out == nullptr) p.prior_lse[t * Hq + h] = sum;
      else if (p.lse != nullptr) p.lse[t * Hq + h] = 0.6931471805599453f * sum;
    }
  }
}

}  // namespace

size_t prompt_workspace_bytes(int32_t Hk, int32_t G, int32_t D, bool fp8, int64_t T, int32_t B, int sms) { return kAttnZeroBytes; }

cudaError_t launch_prompt(const PromptParams& p, cudaStream_t stream) {
  const int64_t blocks = (p.T * p.Hk * p.G + 7) / 8;
  const int64_t most = (int64_t)num_sms() * 8;
  return launch_k(prompt_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, stream, true, p);
}

}  // namespace engram
