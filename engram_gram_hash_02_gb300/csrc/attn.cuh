// Declarations shared by the attention side of libengram (heads.cu, attention.cuh, attn_abi.cu): the
// layer's attention over a paged key-value cache, next to its Engram residual.
#pragma once

#include "internal.cuh"

namespace engram {

constexpr int kMaxHeadDim = 256;

// rows of heads: value (t, h, d) at data + t * ts + h * hs + d (strides in values); data == NULL: absent
struct HeadRows {
  void* data;
  int64_t ts, hs;
  int32_t heads;
  int32_t f32;                 // 1: fp32, 0: bf16
};

// the paged cache with byte strides; row (page, head, place) of k or v at page * page_b + head * head_b + place * tok_b
struct CacheRef {
  uint8_t *k, *v;
  uint8_t *ks, *vs;            // scale words (FP8 only)
  int64_t page_b, head_b, tok_b;
  int64_t spage_b, shead_b, stok_b;
  uint32_t page_u, tok_u;      // page_b and tok_b in units of 16 bytes
  uint32_t spage_u, stok_u;    // spage_b and stok_b in units of 4 bytes
  int64_t slots;               // num_pages * page_size
  int64_t num_pages;
  int32_t page_size, fp8;
  FastDiv div_page;
};

struct NormRope {
  const uint16_t *qw, *kw;     // bf16 [D]; NULL: no norm
  float eps;
  const float* table;          // [rows, R]: cos, then sin; R == 0: no rotation
  int64_t rows;
  int32_t R, start, interleaved;
};

// one launch over a batch's query, key and value rows (see heads.cu)
struct QkvParams {
  int64_t T;
  int32_t D;
  HeadRows q, k, v, q_out, k_out;
  NormRope nr;
  const int32_t* positions;    // [T]
  const int64_t* slots;        // [T] (with a cache)
  CacheRef cache;              // cache.k == NULL: nothing is written to a cache
  int32_t* err;
  // filled by the launcher: the first blocks of keys and values, division by a token's row groups, 1 / D
  uint32_t first_k, first_v;
  FastDiv div_q, div_kv;
  float inv_d;
};
cudaError_t launch_qkv(const QkvParams& p, cudaStream_t stream);

struct KvReadParams {
  int64_t T;
  int32_t D, heads;
  CacheRef cache;
  const int64_t* slots;
  HeadRows k_out, v_out;
  int32_t* err;
  FastDiv div_token;
};
cudaError_t launch_kv_read(const KvReadParams& p, cudaStream_t stream);

// The form of scores, in units of log 2: cap2 * tanh(x * cap_inv) (cap2 0: x itself), less slopes[head] log2(e) per token
// of distance (NULL: none)
struct ScoreForm {
  float cap2, cap_inv;
  const float* slopes;
};

struct AttnParams {
  HeadRows q;                  // [B, Hq, D]
  CacheRef cache;
  const int32_t* table;        // [B, width] page numbers
  int64_t table_stride;
  const int32_t* lens;         // [B]
  int32_t lens_ready;          // 1: read before the wait: the preceding kernel does not write lens, and lets this one
                               // start only after its own wait (what wrote them has finished)
  int32_t B, Hk, G, chunks;    // G query heads per key head, in `chunks` groups of at most 8 * NQ
  int32_t D;
  int32_t cap;                 // longest length the table holds (width * page_size, below 2^31)
  int32_t window;              // 0: none
  float scale_log2;            // softmax scale * log2(e)
  uint16_t* out;               // bf16
  int64_t out_ts, out_hs;
  float* lse;                  // [B, Hq] or NULL
  uint32_t* counters;          // 3 * kMaxAttnCtas words, zero between calls
  float* part;                 // partial results, two slots per CTA
  int32_t* err;
  // with a form (kernels of their own; see ScoreForm), or joined with the keys that were attended before
  ScoreForm form;
  const float* prior_o;        // fp32 [B, Hq, D], or NULL: attended values over those keys
  const float* prior_lse;      // fp32 [B, Hq]: log2 of their exponentials' sum
};
constexpr int kMaxAttnCtas = 1024;
constexpr size_t kAttnZeroBytes = ENGRAM_ATTENTION_ZERO_BYTES;
static_assert(3 * kMaxAttnCtas * sizeof(uint32_t) <= kAttnZeroBytes, "the counters lie in the zeroed part");
// how a shape runs: its kernel's query tiles per CTA, CTAs, partial floats per slot, keys per tile
struct AttnPlan {
  int32_t nq, chunks, grid_max, slot_floats, tile;
};
AttnPlan attn_plan(int32_t G, int32_t D, bool fp8, int sms);
size_t attn_workspace_bytes(int32_t G, int32_t D, bool fp8, int sms);
cudaError_t launch_attention_bf16(const AttnParams& p, const AttnPlan& plan, int64_t max_tiles, cudaStream_t stream, bool pdl);
cudaError_t launch_attention_fp8(const AttnParams& p, const AttnPlan& plan, int64_t max_tiles, cudaStream_t stream, bool pdl);
// the same with a form of scores or a prior part
cudaError_t launch_attention_form_bf16(const AttnParams& p, const AttnPlan& plan, int64_t max_tiles, cudaStream_t stream, bool pdl);
cudaError_t launch_attention_form_fp8(const AttnParams& p, const AttnPlan& plan, int64_t max_tiles, cudaStream_t stream, bool pdl);

// Attention of all new tokens of ragged sequences (prompt.cu), or of one token for each row of a group that shares its
// keys (a prefix): rows [T, Hq, D], those of sequence b are [cu[b], cu[b + 1])
struct PromptParams {
  HeadRows q;                  // bf16
  int64_t T;
  const int32_t* cu;           // [B + 1]
  CacheRef cache;
  const int32_t* table;        // [B, width]
  int64_t table_stride;
  const int32_t* lens;         // [B]
  int32_t B, Hk, G, D;
  int32_t cap;                 // longest length the table holds
  int32_t causal, window;
  const int32_t *doc_starts, *prefix_ends;   // [T] or NULL
  const int32_t* own_lens;     // [T], or NULL. Shared prefix: a row's own tokens, which its position counts behind the prefix
  int32_t own_cap;             // and their longest length
  float scale_log2;
  ScoreForm form;
  uint16_t* out;               // bf16 rows, or (NULL) the prior part of an attention over the rows' own keys:
  int64_t out_ts, out_hs;
  float* lse;                  // [T, Hq] or NULL
  float *prior_o, *prior_lse;  // fp32 [T, Hq, D], [T, Hq] (see AttnParams)
  uint8_t* workspace;
  int32_t* err;
};
size_t prompt_workspace_bytes(int32_t Hk, int32_t G, int32_t D, bool fp8, int64_t T, int32_t B, int sms);
cudaError_t launch_prompt(const PromptParams& p, cudaStream_t stream);

// ---- exponentials and scores ----------------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// cap tanh(x / cap) with cap and x in one unit, inv = 1 / cap. With y = x / cap: 1 - 2 / (1 + exp(2 y)), and below 1/4, where
// that difference loses bits, y - y^3/3 + 2 y^5/15 - 17 y^7/315 (the next term is 3e-7 of it). Off by 2^-19 of itself at most:
// 2^-22 of exp, of the reciprocal and of the difference, against a value of 0.245 and more.
__device__ __forceinline__ float capped(float x, float cap, float inv) {
  const float y = x * inv, t = y * y;
  const float near = y * fmaf(t, fmaf(t, fmaf(t, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  const float far = fmaf(-2.f, __fdividef(1.f, 1.f + ex2(y * 2.88539008f)), 1.f);
  return cap * (fabsf(y) < 0.25f ? near : far);
}

// ---- asynchronous copies of 16 bytes to shared memory --------------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---- rows of 8 values per thread -----------------------------------------------------------
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// four e4m3 codes as two pairs of halves: exact
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
      : "=r"(lo), "=r"(hi) : "r"(codes));
}

}  // namespace engram
