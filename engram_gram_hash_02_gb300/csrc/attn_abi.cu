// The extern "C" entry points of the attention side of libengram: argument checks and launches.
#include <math.h>

#include "attn.cuh"

namespace engram {
namespace {

int64_t value_bytes(int32_t type) { return type == ENGRAM_F32 ? 4 : 2; }

int check_dim(const char* fn, int32_t D) {
  ENGRAM_CHECK_ARG(D >= 8 && D <= kMaxHeadDim && D % 8 == 0, "%s: head_dim must be a multiple of 8 in [8, %d] (got %d)",
                   fn, kMaxHeadDim, D);
  return ENGRAM_OK;
}

// rows [T, heads, D] as input; `out`: as an output, whose rows must not overlap
int check_heads(const char* fn, const char* name, const EngramHeads* r, int64_t T, int32_t D, bool out, HeadRows* to) {
  ENGRAM_CHECK_ARG(r != nullptr && (r->data != nullptr || T == 0), "%s: %s must be non-NULL", fn, name);
  ENGRAM_CHECK_ARG(r->type == ENGRAM_BF16 || r->type == ENGRAM_F32, "%s: %s has unknown type %d", fn, name, r->type);
  ENGRAM_CHECK_ARG(r->heads >= 1 && r->heads <= 65536, "%s: %s must have 1 to 65536 heads (got %d)", fn, name, r->heads);
  const int64_t unit = 16 / value_bytes(r->type);
  ENGRAM_CHECK_ARG(aligned(r->data, 16) && r->token_stride % unit == 0 && r->head_stride % unit == 0,
                   "%s: %s and its strides must be multiples of 16 bytes", fn, name);
  ENGRAM_CHECK_ARG(r->token_stride >= 0 && r->head_stride >= 0, "%s: %s must have strides >= 0", fn, name);
  if (out) {
    const int64_t t = r->token_stride, h = r->head_stride;
    // head inside token, or token inside head: the inner rows fit one outer stride (128-bit: no overflow)
    const bool inner_h = (r->heads == 1 || h >= D) && (T <= 1 || (__int128)(r->heads - 1) * h + D <= t);
    const bool inner_t = (T <= 1 || t >= D) && (r->heads == 1 || (__int128)(T > 0 ? T - 1 : 0) * t + D <= h);
    ENGRAM_CHECK_ARG(inner_h || inner_t, "%s: rows of %s overlap (token stride %lld, head stride %lld)", fn, name,
                     (long long)t, (long long)h);
  }
  to->data = r->data;
  to->ts = r->token_stride;
  to->hs = r->head_stride;
  to->heads = r->heads;
  to->f32 = r->type == ENGRAM_F32;
  return ENGRAM_OK;
}

int check_tokens(const char* fn, int64_t T) {
  ENGRAM_CHECK_ARG(T >= 0 && T < (int64_t)1 << 31, "%s: T must be in [0, 2^31) (got %lld)", fn, (long long)T);
  return ENGRAM_OK;
}

int check_nr(const char* fn, const EngramNormRope* nr, int64_t T, int32_t D, const int32_t* positions, NormRope* to) {
  ENGRAM_CHECK_ARG(nr != nullptr, "%s: nr is NULL", fn);
  ENGRAM_CHECK_ARG((nr->q_weight == nullptr) == (nr->k_weight == nullptr),
                   "%s: q_weight and k_weight must both be given, or neither", fn);
  ENGRAM_CHECK_ARG(aligned(nr->q_weight, 16) && aligned(nr->k_weight, 16), "%s: q_weight and k_weight must be 16-byte aligned", fn);
  ENGRAM_CHECK_ARG(nr->eps >= 0.f && isfinite(nr->eps), "%s: eps must be finite and >= 0", fn);
  const int32_t R = nr->rope_dim;
  ENGRAM_CHECK_ARG(R >= 0 && R <= D && nr->rope_start >= 0 && nr->rope_start <= D - R,
                   "%s: the rotated part [%d, %d + %d) must lie in [0, %d)", fn, nr->rope_start, nr->rope_start, R, D);
  ENGRAM_CHECK_ARG(nr->rope_start % 8 == 0, "%s: rope_start must be a multiple of 8 (got %d)", fn, nr->rope_start);
  ENGRAM_CHECK_ARG(R % (nr->interleaved ? 8 : 16) == 0, "%s: rope_dim must be a multiple of %d (got %d)", fn,
                   nr->interleaved ? 8 : 16, R);
  if (R > 0) {
    ENGRAM_CHECK_ARG(nr->table != nullptr && aligned(nr->table, 16), "%s: the rotation table must be non-NULL and 16-byte aligned", fn);
    ENGRAM_CHECK_ARG(nr->table_rows >= 1, "%s: the rotation table must have a row", fn);
    ENGRAM_CHECK_ARG((positions != nullptr || T == 0) && aligned(positions, 4), "%s: positions must be a non-NULL, aligned int32 array", fn);
  }
  to->qw = nr->q_weight;
  to->kw = nr->k_weight;
  to->eps = nr->eps;
  to->table = nr->table;
  to->rows = nr->table_rows;
  to->R = R;
  to->start = nr->rope_start;
  to->interleaved = nr->interleaved != 0;
  return ENGRAM_OK;
}

int check_cache(const char* fn, const EngramKVCache* c, CacheRef* to) {
  ENGRAM_CHECK_ARG(c != nullptr, "%s: cache is NULL", fn);
  const bool fp8 = c->format == ENGRAM_CACHE_FP8_E8M0;
  ENGRAM_CHECK_ARG(fp8 || c->format == ENGRAM_CACHE_BF16, "%s: unknown cache format %d", fn, c->format);
  const int32_t unit = fp8 ? 32 : 16;
  ENGRAM_CHECK_ARG(c->head_dim >= unit && c->head_dim <= kMaxHeadDim && c->head_dim % unit == 0,
                   "%s: the cache's head_dim must be a multiple of %d in [%d, %d] (got %d)", fn, unit, unit, kMaxHeadDim, c->head_dim);
  ENGRAM_CHECK_ARG(c->kv_heads >= 1 && c->kv_heads <= 65536, "%s: kv_heads must be in [1, 65536] (got %d)", fn, c->kv_heads);
  ENGRAM_CHECK_ARG(c->page_size >= 1, "%s: page_size must be >= 1 (got %d)", fn, c->page_size);
  ENGRAM_CHECK_ARG(c->num_pages >= 0 && c->num_pages <= (int64_t)1 << 31, "%s: num_pages must be in [0, 2^31]", fn);
  ENGRAM_CHECK_ARG(c->k != nullptr && c->v != nullptr && aligned(c->k, 16) && aligned(c->v, 16),
                   "%s: the cache's k and v must be non-NULL and 16-byte aligned", fn);
  const int64_t bytes = fp8 ? 1 : 2;
  ENGRAM_CHECK_ARG(c->page_stride >= 0 && c->head_stride >= 0 && c->token_stride >= 0, "%s: the cache's strides must be >= 0", fn);
  ENGRAM_CHECK_ARG(c->page_stride * bytes % 16 == 0 && c->head_stride * bytes % 16 == 0 && c->token_stride * bytes % 16 == 0,
                   "%s: the cache's strides must be multiples of 16 bytes", fn);
  to->k = static_cast<uint8_t*>(c->k);
  to->v = static_cast<uint8_t*>(c->v);
  to->page_b = c->page_stride * bytes;
  to->head_b = c->head_stride * bytes;
  to->tok_b = c->token_stride * bytes;
  ENGRAM_CHECK_ARG(to->page_b / 16 < (int64_t)1 << 32 && to->tok_b / 16 < (int64_t)1 << 32,
                   "%s: the cache's page and token strides must be below 2^36 bytes", fn);
  to->page_u = (uint32_t)(to->page_b / 16);
  to->tok_u = (uint32_t)(to->tok_b / 16);
  to->spage_u = to->stok_u = 0;
  to->ks = to->vs = nullptr;
  to->spage_b = to->shead_b = to->stok_b = 0;
  if (fp8) {
    ENGRAM_CHECK_ARG(c->k_scales != nullptr && c->v_scales != nullptr && aligned(c->k_scales, 4) && aligned(c->v_scales, 4),
                     "%s: an FP8 cache's scales must be non-NULL and 4-byte aligned", fn);
    ENGRAM_CHECK_ARG(c->scale_page_stride >= 0 && c->scale_head_stride >= 0 && c->scale_token_stride >= 0 &&
                         c->scale_page_stride % 4 == 0 && c->scale_head_stride % 4 == 0 && c->scale_token_stride % 4 == 0,
                     "%s: the scale strides must be multiples of 4 bytes and >= 0", fn);
    to->ks = c->k_scales;
    to->vs = c->v_scales;
    to->spage_b = c->scale_page_stride;
    to->shead_b = c->scale_head_stride;
    to->stok_b = c->scale_token_stride;
    ENGRAM_CHECK_ARG(to->spage_b / 4 < (int64_t)1 << 32 && to->stok_b / 4 < (int64_t)1 << 32,
                     "%s: the scale page and token strides must be below 2^34 bytes", fn);
    to->spage_u = (uint32_t)(to->spage_b / 4);
    to->stok_u = (uint32_t)(to->stok_b / 4);
  }
  to->num_pages = c->num_pages;
  to->page_size = c->page_size;
  to->slots = c->num_pages * c->page_size;
  to->fp8 = fp8;
  to->div_page = make_fastdiv((uint32_t)c->page_size);
  return ENGRAM_OK;
}

int check_slots(const char* fn, const int64_t* slots, int64_t T) {
  ENGRAM_CHECK_ARG((slots != nullptr || T == 0) && aligned(slots, 8), "%s: slots must be a non-NULL, aligned int64 array", fn);
  return ENGRAM_OK;
}

// one type and kv_heads heads for the rows that go to a cache
int check_kv(const char* fn, const EngramKVCache* c, const HeadRows& k, const HeadRows& v) {
  ENGRAM_CHECK_ARG(k.heads == c->kv_heads && v.heads == c->kv_heads, "%s: k and v must have the cache's %d heads (got %d and %d)",
                   fn, c->kv_heads, k.heads, v.heads);
  ENGRAM_CHECK_ARG(k.f32 == v.f32, "%s: k and v must have one type", fn);
  return ENGRAM_OK;
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Attn {
  AttnParams p;
  AttnPlan plan;
  int64_t max_tiles;
};

// everything but q, err and the stream
int check_attention(const char* fn, const EngramKVCache* cache, const EngramPagedSeqs* s, int32_t q_heads, float scale,
                    int32_t window, const EngramHeads* out, float* lse, void* workspace, size_t ws_bytes, size_t ws_need, Attn* a) {
  AttnParams& p = a->p;
  int rc = check_cache(fn, cache, &p.cache);
  if (rc) return rc;
  ENGRAM_CHECK_ARG(s != nullptr, "%s: seqs is NULL", fn);
  ENGRAM_CHECK_ARG(s->batch >= 0, "%s: batch must be >= 0 (got %d)", fn, s->batch);
  ENGRAM_CHECK_ARG(q_heads >= 1 && q_heads % cache->kv_heads == 0, "%s: q_heads (%d) must be a multiple of kv_heads (%d)", fn,
                   q_heads, cache->kv_heads);
  ENGRAM_CHECK_ARG(s->table_width >= 0 && s->table_stride >= s->table_width, "%s: the page table's stride (%lld) must be >= its width (%d >= 0)",
                   fn, (long long)s->table_stride, s->table_width);
  ENGRAM_CHECK_ARG((s->seq_lens != nullptr || s->batch == 0) && aligned(s->seq_lens, 4) &&
                       (s->block_table != nullptr || s->table_width == 0 || s->batch == 0) &&
                       aligned(s->block_table, 4),
                   "%s: block_table and seq_lens must be non-NULL, aligned int32 arrays", fn);
  ENGRAM_CHECK_ARG(isfinite(scale), "%s: scale must be finite", fn);
  ENGRAM_CHECK_ARG(window >= 0, "%s: window must be >= 0 (got %d)", fn, window);
  HeadRows o;
  rc = check_heads(fn, "out", out, s->batch, cache->head_dim, true, &o);
  if (rc) return rc;
  ENGRAM_CHECK_ARG(!o.f32 && o.heads == q_heads, "%s: out must be bf16 with %d heads", fn, q_heads);
  ENGRAM_CHECK_ARG(aligned(lse, 4), "%s: lse must be 4-byte aligned", fn);
  ENGRAM_CHECK_ARG(workspace != nullptr && aligned(workspace, 256), "%s: workspace must be non-NULL and 256-byte aligned", fn);
  ENGRAM_CHECK_ARG(ws_bytes >= ws_need, "%s: workspace holds %zu bytes, needs %zu", fn, ws_bytes, ws_need);

  p.table = s->block_table;
  p.table_stride = s->table_stride;
  p.lens = s->seq_lens;
  p.B = s->batch;
  p.Hk = cache->kv_heads;
  p.G = q_heads / cache->kv_heads;
  p.D = cache->head_dim;
  const int64_t cap = (int64_t)s->table_width * cache->page_size;
  p.cap = (int32_t)(cap < 0x7FFFFF00 ? cap : 0x7FFFFF00);
  p.window = window;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.out = static_cast<uint16_t*>(o.data);
  p.out_ts = o.ts;
  p.out_hs = o.hs;
  p.lse = lse;
  a->plan = attn_plan(p.G, p.D, p.cache.fp8, num_sms());
  p.chunks = a->plan.chunks;
  p.counters = static_cast<uint32_t*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kAttnZeroBytes);
  const int64_t longest = window > 0 && window < p.cap ? window : p.cap;
  const int64_t tile = a->plan.tile;
  const __int128 tiles = (__int128)p.B * p.Hk * p.chunks * ((longest + tile - 1) / tile);
  ENGRAM_CHECK_ARG(tiles < (__int128)1 << 28, "%s: batch * kv_heads * page table capacity is too large", fn);
  a->max_tiles = tiles < 1 ? 1 : (int64_t)tiles;
  return ENGRAM_OK;
}

int run_attention(const char* fn, const Attn& a, cudaStream_t stream, bool pdl) {
  const cudaError_t e = a.p.cache.fp8 ? launch_attention_fp8(a.p, a.plan, a.max_tiles, stream, pdl)
                                      : launch_attention_bf16(a.p, a.plan, a.max_tiles, stream, pdl);
  return e == cudaSuccess ? ENGRAM_OK : fail_cuda(e, fn);
}

// the join's scratch, then the step's turned queries (fp32 [batch, q_heads, head_dim])
size_t join_bytes(const EngramKVCache* c, int32_t q_heads) {
  return round256(attn_workspace_bytes(q_heads / c->kv_heads, c->head_dim, c->format == ENGRAM_CACHE_FP8_E8M0, num_sms()));
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" {

int engram_qk_norm_rope(const EngramNormRope* nr, int64_t T, int32_t head_dim, const EngramHeads* q, const EngramHeads* k,
                        const int32_t* positions, const EngramHeads* q_out, const EngramHeads* k_out, int32_t* err_flag,
                        engram_stream_t stream) {
  const char* fn = "engram_qk_norm_rope";
  QkvParams p{};
  int rc = check_dim(fn, head_dim);
  if (!rc) rc = check_tokens(fn, T);
  if (!rc) rc = check_nr(fn, nr, T, head_dim, positions, &p.nr);
  if (rc) return rc;
  ENGRAM_CHECK_ARG((q == nullptr) == (q_out == nullptr) && (k == nullptr) == (k_out == nullptr) && (q != nullptr || k != nullptr),
                   "%s: q with q_out, k with k_out, or both", fn);
  if (q != nullptr) {
    rc = check_heads(fn, "q", q, T, head_dim, false, &p.q);
    if (!rc) rc = check_heads(fn, "q_out", q_out, T, head_dim, true, &p.q_out);
    if (rc) return rc;
    ENGRAM_CHECK_ARG(p.q.heads == p.q_out.heads, "%s: q has %d heads but q_out %d", fn, p.q.heads, p.q_out.heads);
  }
  if (k != nullptr) {
    rc = check_heads(fn, "k", k, T, head_dim, false, &p.k);
    if (!rc) rc = check_heads(fn, "k_out", k_out, T, head_dim, true, &p.k_out);
    if (rc) return rc;
    ENGRAM_CHECK_ARG(p.k.heads == p.k_out.heads, "%s: k has %d heads but k_out %d", fn, p.k.heads, p.k_out.heads);
  }
  ENGRAM_CHECK_ARG(q == nullptr || k == nullptr || p.q.f32 == p.k.f32, "%s: q and k must have one type", fn);
  if (T == 0) return ENGRAM_OK;
  p.T = T;
  p.D = head_dim;
  p.positions = positions;
  p.err = err_flag;
  const cudaError_t e = launch_qkv(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ENGRAM_OK : fail_cuda(e, fn);
}

int engram_kv_write(const EngramKVCache* cache, int64_t T, const EngramHeads* k, const EngramHeads* v, const int64_t* slots,
                    int32_t* err_flag, engram_stream_t stream) {
  const char* fn = "engram_kv_write";
  QkvParams p{};
  int rc = check_cache(fn, cache, &p.cache);
  if (!rc) rc = check_tokens(fn, T);
  if (!rc) rc = check_heads(fn, "k", k, T, cache->head_dim, false, &p.k);
  if (!rc) rc = check_heads(fn, "v", v, T, cache->head_dim, false, &p.v);
  if (!rc) rc = check_kv(fn, cache, p.k, p.v);
  if (!rc) rc = check_slots(fn, slots, T);
  if (rc) return rc;
  if (T == 0) return ENGRAM_OK;
  p.T = T;
  p.D = cache->head_dim;
  p.slots = slots;
  p.err = err_flag;
  const cudaError_t e = launch_qkv(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ENGRAM_OK : fail_cuda(e, fn);
}

int engram_kv_read(const EngramKVCache* cache, int64_t T, const int64_t* slots, const EngramHeads* k_out,
                   const EngramHeads* v_out, int32_t* err_flag, engram_stream_t stream) {
  const char* fn = "engram_kv_read";
  KvReadParams p{};
  int rc = check_cache(fn, cache, &p.cache);
  if (!rc) rc = check_tokens(fn, T);
  if (!rc) rc = check_slots(fn, slots, T);
  if (!rc) rc = check_heads(fn, "k_out", k_out, T, cache->head_dim, true, &p.k_out);
  if (!rc) rc = check_heads(fn, "v_out", v_out, T, cache->head_dim, true, &p.v_out);
  if (!rc) rc = check_kv(fn, cache, p.k_out, p.v_out);
  if (rc) return rc;
  if (T == 0) return ENGRAM_OK;
  p.T = T;
  p.D = cache->head_dim;
  p.heads = cache->kv_heads;
  p.slots = slots;
  p.err = err_flag;
  const cudaError_t e = launch_kv_read(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ENGRAM_OK : fail_cuda(e, fn);
}

size_t engram_attention_workspace_bytes(const EngramKVCache* cache, int32_t q_heads, int32_t batch) {
  if (cache == nullptr || cache->kv_heads < 1 || q_heads < 1 || q_heads % cache->kv_heads != 0 || cache->head_dim < 1 ||
      cache->head_dim > kMaxHeadDim || batch < 0)
    return 0;
  return join_bytes(cache, q_heads) + round256((size_t)batch * q_heads * cache->head_dim * sizeof(float));
}

int engram_paged_attention(const EngramKVCache* cache, const EngramPagedSeqs* seqs, const EngramHeads* q, float scale,
                           int32_t window, const EngramHeads* out, float* lse, void* workspace, size_t ws_bytes,
                           int32_t* err_flag, engram_stream_t stream) {
  const char* fn = "engram_paged_attention";
  Attn a{};
  CacheRef c;
  int rc = check_cache(fn, cache, &c);
  if (rc) return rc;
  ENGRAM_CHECK_ARG(seqs != nullptr, "%s: seqs is NULL", fn);
  rc = check_heads(fn, "q", q, seqs->batch, cache->head_dim, false, &a.p.q);
  if (rc) return rc;
  ENGRAM_CHECK_ARG(q->heads % cache->kv_heads == 0, "%s: q_heads (%d) must be a multiple of kv_heads (%d)", fn, q->heads,
                   cache->kv_heads);
  rc = check_attention(fn, cache, seqs, q->heads, scale, window, out, lse, workspace, ws_bytes, join_bytes(cache, q->heads), &a);
  if (rc) return rc;
  if (seqs->batch == 0) return ENGRAM_OK;
  a.p.err = err_flag;
  return run_attention(fn, a, static_cast<cudaStream_t>(stream), true);
}

int engram_attention_step(const EngramNormRope* nr, const EngramKVCache* cache, const EngramPagedSeqs* seqs, const EngramHeads* q,
                          const EngramHeads* k, const EngramHeads* v, const int32_t* positions, const int64_t* slots, float scale,
                          int32_t window, const EngramHeads* out, float* lse, void* workspace, size_t ws_bytes, int32_t* err_flag,
                          engram_stream_t stream) {
  const char* fn = "engram_attention_step";
  Attn a{};
  QkvParams p{};
  int rc = check_cache(fn, cache, &p.cache);
  if (rc) return rc;
  ENGRAM_CHECK_ARG(seqs != nullptr, "%s: seqs is NULL", fn);
  const int32_t B = seqs->batch, D = cache->head_dim;
  rc = check_nr(fn, nr, B, D, positions, &p.nr);
  if (!rc) rc = check_heads(fn, "q", q, B, D, false, &p.q);
  if (!rc) rc = check_heads(fn, "k", k, B, D, false, &p.k);
  if (!rc) rc = check_heads(fn, "v", v, B, D, false, &p.v);
  if (!rc) rc = check_kv(fn, cache, p.k, p.v);
  if (!rc) rc = check_slots(fn, slots, B);
  if (rc) return rc;
  ENGRAM_CHECK_ARG(p.q.f32 == p.k.f32, "%s: q, k and v must have one type", fn);
  ENGRAM_CHECK_ARG(q->heads % cache->kv_heads == 0, "%s: q_heads (%d) must be a multiple of kv_heads (%d)", fn, q->heads,
                   cache->kv_heads);
  const size_t join = join_bytes(cache, q->heads);
  rc = check_attention(fn, cache, seqs, q->heads, scale, window, out, lse, workspace, ws_bytes,
                       engram_attention_workspace_bytes(cache, q->heads, B), &a);
  if (rc) return rc;
  if (B == 0) return ENGRAM_OK;
  p.T = B;
  p.D = D;
  p.q_out.data = static_cast<uint8_t*>(workspace) + join;
  p.q_out.hs = D;
  p.q_out.ts = (int64_t)q->heads * D;
  p.q_out.heads = q->heads;
  p.q_out.f32 = 1;
  p.positions = positions;
  p.slots = slots;
  p.err = err_flag;
  const cudaError_t e = launch_qkv(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda(e, fn);
  a.p.q = p.q_out;
  a.p.lens_ready = 1;
  a.p.err = err_flag;
  return run_attention(fn, a, static_cast<cudaStream_t>(stream), true);
}

}  // extern "C"
