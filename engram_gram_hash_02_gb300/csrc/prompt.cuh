// Attention of all new tokens of ragged sequences over a paged cache, on the tensor cores (tcgen05).
//
// For a token's query head h and the keys [lo, hi) that it sees:
//   s_j = form(scale q_h . k_j),   o_h = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse_h = log sum_j exp(s_j)
// with a running maximum m (units of log 2, every exponential one ex2). Rows are tokens times the G query heads of a key
// head, so that a key row is used by all of them; 128 rows make a tile (the MMA's M), two tiles share every key and value
// tile that is brought in (heads of up to 128; one tile for wider heads, whose sums fill tensor memory).
//
// One CTA per SM, 16 warps (FP8: 20) with roles of their own, joined by mbarriers only:
//   warps 0..3, 4..7   softmax of tile 0 and 1: a thread has a row. S (fp32) comes from tensor memory, P goes back there
//                      as bf16, in S's place; o is multiplied there only when the maximum grows by more than 2^30
//   warp 8             issues the MMAs:  S = Q K^T (both from shared memory),  O += P V (P from tensor memory, V as it
//                      lies, by rows of keys: an MN-major operand)
//   warp 9             walks the CTA's share of the work and hands segments (a run of key tiles of one pair of tiles) out
//   warps 12, 13       look pages up and request K and V tiles in the order in which they are used: TMA boxes of
//                      the cache's own layout, up to 64 tokens of a page at once. bf16 goes to a ring of 32 KB slots
//                      that the MMAs read, FP8 to stages
//   warps 10, 11, 14, 15 (FP8: ..19)   bring Q in, look through values (below); FP8: convert a stage's rows to bf16 into the
//                      ring (exact), half of them a slot in turn. Pages that are no multiple of 8 tokens do not divide
//                      into boxes: these warps, and all loaders but one, then fetch the rows themselves
// While the softmax of one tile runs, the tensor cores work on the other; with one tile, on the next key tile.
//
// Work is cut at key tiles: a first kernel (one CTA) lists the pairs of tiles with the hull of their keys, and every CTA
// takes an equal run of the list. A pair that is cut leaves (o, m, sum) per CTA; the last warp to arrive joins them, or a
// kernel behind this one where pairs are few and their parts many (prompt.cu says when).
//
// Keys outside of a row's interval are masked in S. P is zero there, but 0 * inf is not: in a value tile that some row sees
// only in part, infinities and NaN are replaced by zeros, and the softmax warps add their products to the rows that see
// them. A row that sees nothing is left out of that, and is zero by a select.
//
// A barrier tells its phases apart by parity alone, so nobody may wait for a phase that lies two away from where the barrier is:
// whoever waits for a slot has a part in filling it, and whoever waits for scores or sums in what comes next. (A model of all
// waits and arrivals is among the tests.)
//
// Roundings below 32 bits: P to bf16, once (2^-8 of itself at most): it is an operand of the tensor cores beside V, which is bf16,
// and two bf16 for it would be a second P V. The sums take P before that.
//
// Measured (one GB300, 8192 tokens of one prompt, 32 / 8 heads of 128): bf16 462 us, 1.19 PFLOP/s, the tensor pipe 56 % busy; a
// cap 817 us, slopes 647, FP8 717. Heads of 256 (16 / 2): 606 us, bound by key and value tiles from L2 for every 128 rows
// (without softmax and MMAs 425). Without the softmax heads of 128 take 363 us: its latency per tile is what bounds them, and over FP8 the
// codes' conversion beside it. (What stands elsewhere in the kernel moves the hot loops' code: up to 4 % between builds that differ
// in nothing that runs.)
#pragma once

#include "attn.cuh"
#include "ring.h"
#include "tc_common.cuh"

namespace engram {
namespace prompt {

constexpr int kKeys = 128;                            // of a tile
constexpr int kSlotBytes = 32768;                     // 128 keys of up to 128 values, as two blocks of 128-byte rows
constexpr int kBlockBytes = 16384;
__host__ __device__ constexpr int slots_of(bool fp8) { return fp8 ? 3 : 4; }
// of a softmax warp: 32 rows of 32 values (FP8: 16, its stages leave no room for more) on their way out, in pieces of 16 bytes
__host__ __device__ constexpr int staging_pieces(bool fp8) { return fp8 ? 2 : 4; }
__host__ __device__ constexpr int staging_bytes(bool fp8) { return 32 * 16 * staging_pieces(fp8); }
constexpr int kStages = 3;                            // FP8: of 128 codes and their scale word for each of 128 keys
constexpr int kStageBytes = kBlockBytes + 512;
constexpr int kQBytes = 65536;
// Warps that convert FP8 rows are what bounds it: four more of them, with fewer registers each
__host__ __device__ constexpr int threads_of(bool fp8) { return fp8 ? 640 : 512; }
// Behind the softmax, MMA and dividing warps: those that request boxes (one requests a box in about 200 cycles, and a page of
// 16 tokens is a box), and helpers. Where rows are fetched one by one only the first loader is one.
__host__ __device__ constexpr int loaders_of(bool fp8) { return 2; }
__host__ __device__ constexpr int helpers_of(bool fp8) { return fp8 ? 8 : 4; }
constexpr int kMaxHelpers = 9;
constexpr int kMeta = 8;                              // key tiles whose masks are kept
constexpr int kRunCost = 1;                           // a pair's fixed cost in key tiles, when work is divided
// How far a row's maximum may run ahead of the one its sums are in units of, log 2. fp32 and bf16 keep their bits there;
// what it takes is range: sums come to 2^30 times what they stand for at most, so values may be as large as 2^85 or so over
// a few thousand keys. (With 8, rows whose scores spread by 2^14 had o multiplied in most of their tiles: 8192 tokens of 32 / 8
// heads of 128, scores capped at 30, took three times as long.)
constexpr float kLag = 30.f;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 256;                       // S of buffer b at column 128 b, O of tile t at 256 + 128 t

// one pair of tiles of a sequence, equal for all key heads
struct Entry {
  int32_t b, row0, rows;                              // sequence; rows [row0, rows) of its n * G, at most a pair's
  int32_t s0, n, len;
  int32_t hi;                                         // past the last key that any of its rows sees
  int32_t max_lo, min_hi;                             // keys from max_lo to min_hi are seen by every row that sees any
  int32_t key0, units;                                // first key and number of its key tiles
  int64_t place;                                      // in the row of a head's work
};
struct Header {
  int64_t entries, places, per_cta;                   // places per head, places per CTA
};
struct Start {                                        // a CTA's first entry
  int32_t head, entry;
};
// workspace behind its zeroed start, which is the one-token calls' and stays as it is
struct Layout {
  size_t header, counters, starts, offsets, entries, parts, all;
  int64_t max_entries;
  int32_t slot_floats;
};
__host__ __device__ constexpr int pair_rows(int D) { return D > 128 ? 128 : 256; }

struct Args {
  PromptParams p;
  Header* header;
  Start* starts;
  int32_t* offsets;                                   // [B + 1] first entries of the sequences
  Entry* entries;
  uint32_t* counters;                                 // [CTA][8 warps], zeroed by the list kernel: a call that gave up leaves any
  float* parts;
  int64_t max_entries;
  int32_t slot_floats;
  int32_t join;                                       // 1: the last warp to arrive joins a cut pair's rows
  int32_t ctas;
  int32_t box;                                        // tokens per TMA box, a power of two that divides a page (0: rows one by one)
  int32_t q_box;                                      // 1: a tile is whole tokens, and Q comes as TMA boxes
  FastDiv div_g;
};

struct Row {                                          // what a row is and sees
  int64_t token;
  int32_t head, lo, hi, pos;                          // head among its key head's
};
__device__ __forceinline__ int clamp_len(int len, int cap) { return len < 0 ? 0 : len > cap ? cap : len; }

// token i (row0 .. of sequence rows) of an entry's sequence
__device__ __forceinline__ void visible(const PromptParams& p, int s0, int n, int len, int i, int& lo, int& hi, int& pos) {
  const int64_t t = (int64_t)s0 + i;
  lo = 0;
  if (p.own_lens != nullptr) {
    pos = len + clamp_len(__ldcg(p.own_lens + t), p.own_cap) - 1;
    hi = len;
    return;
  }
  pos = len - n + i;
  hi = len;
  if (p.causal) hi = min(len, max(pos + 1, p.prefix_ends != nullptr ? __ldcg(p.prefix_ends + t) : 0));
  if (p.window > 0 && pos + 1 > p.window) lo = pos + 1 - p.window;
  // (no further than the keys: any number may stand there, and what follows adds a tile's keys to it)
  if (p.doc_starts != nullptr) lo = max(lo, min(__ldcg(p.doc_starts + t), len));
}

// ---- parts of cut pairs: o [D / 4][rows of a pair] of 4 floats, then (m, sum) [rows] ------------------------------
__device__ __forceinline__ float4* part_o(float* slot, int R, int d4, int r) { return reinterpret_cast<float4*>(slot) + (int64_t)d4 * R + r; }
__device__ __forceinline__ float2* part_ml(float* slot, int R, int D, int r) {
  return reinterpret_cast<float2*>(reinterpret_cast<float4*>(slot) + (int64_t)(D / 4) * R) + r;
}
__device__ __forceinline__ float ex2_rel(float x, float m) { return ex2(x - (m == -INFINITY ? 0.f : m)); }

// 16 values of a row from value d on, and (with d 0) its log-sum-exp. A row without a weight is zero by a select, not by a
// product: the MMAs have multiplied its weights of zero with values that may be infinite, and its sums are NaN then
__device__ __forceinline__ void emit16(const PromptParams& p, int64_t token, int h, int d, const float (&sums)[16], float m, float l) {
  const float inv = 1.f / l;
  float o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = l == 0.f ? 0.f : sums[i] * inv;
  const int64_t row = token * (p.Hk * p.G) + h;
  if (p.out != nullptr) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
    uint4* dst = reinterpret_cast<uint4*>(p.out + token * p.out_ts + (int64_t)h * p.out_hs + d);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    float4* dst = reinterpret_cast<float4*>(p.prior_o + row * p.D + d);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  }
  if (d == 0) {
    const float sum = l == 0.f ? -INFINITY : m + log2f(l);
    if (p.out == nullptr)
      p.prior_lse[row] = sum;
    else if (p.lse != nullptr)
      p.lse[row] = 0.6931471805599453f * sum;
  }
}

// joins 16 values of a pair's row r from the parts of CTAs first .. last, in the order of their keys
__device__ __forceinline__ void join16(const Args& a, int first, int last, int R, int r, int64_t token, int h, int d) {
  auto slot = [&](int c) { return a.parts + (int64_t)(2 * c + (c == first ? 1 : 0)) * a.slot_floats; };
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  constexpr int kBatch = 4;
  for (int c0 = first; c0 <= last; c0 += kBatch) {
    float2 ml[kBatch];
    float4 y[kBatch][4];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c0 + k <= last) {
        float* s = slot(c0 + k);
        ml[k] = __ldcg(part_ml(s, R, a.p.D, r));
#pragma unroll
        for (int i = 0; i < 4; ++i) y[k][i] = __ldcg(part_o(s, R, d / 4 + i, r));
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, ml[k].x);
    const float f0 = ex2_rel(m, mn);
    m = mn;
    l *= f0;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= f0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float f = ex2_rel(ml[k].x, mn);
      l += ml[k].y * f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[4 * i] += y[k][i].x * f;
        o[4 * i + 1] += y[k][i].y * f;
        o[4 * i + 2] += y[k][i].z * f;
        o[4 * i + 3] += y[k][i].w * f;
      }
    }
  }
  emit16(a.p, token, h, d, o, m, l);
}

// ---- tensor memory -------------------------------------------------------------------------------------------
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]), "=f"(x[9]),
        "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15]), "=f"(x[16]), "=f"(x[17]), "=f"(x[18]),
        "=f"(x[19]), "=f"(x[20]), "=f"(x[21]), "=f"(x[22]), "=f"(x[23]), "=f"(x[24]), "=f"(x[25]), "=f"(x[26]), "=f"(x[27]),
        "=f"(x[28]), "=f"(x[29]), "=f"(x[30]), "=f"(x[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  return r;
}
// nothing moves what uses x before the wait that this stands behind
template <int N>
__device__ __forceinline__ void hold(float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(x[i]));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// S = Q K^T: both operands K-major from shared memory (tc_mma). O += P V: A from tensor memory
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// V as it lies: rows of keys (the products' K), 64 values to a 128-byte row (N), 128B swizzle; the next 8 keys are 1024
// bytes on (stride offset), the next 64 values a block of 128 rows (leading offset)
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kBlockBytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// bf16 operands, fp32 sums, M = 128
__device__ __forceinline__ uint32_t idesc_of(int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// one lane of a warp that is together
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(is));
  return is != 0;
}
// (the warpgroups' shares come to what the block is launched with: 2 * 168 + 2 * 88 = 4 * 128 a thread; FP8 2 * 144 + 3 * 64 = 5 * 96)
template <int kRegs>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
               : "memory");
}
// mbar_wait without a call, which would cost the softmax warps their registers
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, volatile int32_t* abort_flag, int32_t* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0) {
      if (*abort_flag) return false;
      if ((uint64_t)clock64() - t0 > kWaitLimitCycles) {
        *abort_flag = 1;
        if (err != nullptr) atomicOr(err, ENGRAM_ERR_PIPE_TIMEOUT);
        return false;
      }
    }
  }
}

// ---- shared memory behind the ring -----------------------------------------------------------------------------
struct Segment {
  int32_t tiles;                                      // key tiles (0: no more work)
  int32_t nt;                                         // tiles of rows: 1 or 2
  int32_t b, head;
  int32_t row0, rows, s0, n, len;
  int32_t key0;                                       // first key of the segment
  int32_t hull_hi, max_lo, min_hi;                    // see Entry
  int32_t whole;                                      // all of its pair's keys
  int32_t c_first, c_last;                            // CTAs of a cut pair
};
struct Ctl {
  uint64_t full[4], empty[4];
  uint64_t st_full[kStages], st_empty[kStages];
  uint64_t q_full, q_empty;
  uint64_t k_meta[kMeta];                             // of key tiles, in turn: `live` is there
  uint64_t v_go[kMeta], v_meta[kMeta];                // of value tiles that some row sees partly: requested; looked through
  uint64_t s_full[2], p_full[2], o_done;
  uint64_t o_final[2][2];                             // [tile][segments in turn]: the segment's sums are
  uint64_t seg_full[2], seg_empty[2];
  uint64_t drained;
  int32_t asked[2], asked_q;                          // what loaders request next, on their way out (place | parity << 8); Q's last phase
  Segment seg[2];
  alignas(16) uint32_t live[kMeta][4];                // which keys of a tile are there
  uint32_t v_bad[kMeta][kMaxHelpers][4];              // keys whose values are not all finite (in tiles that some row sees partly)
  uint32_t tmem_base;
  int32_t abort_flag;
};
constexpr int smem_bytes(bool fp8) { return 1024 + kQBytes + slots_of(fp8) * kSlotBytes + (fp8 ? kStages * kStageBytes : 0) + 8 * staging_bytes(fp8) + (int)sizeof(Ctl); }
static_assert(smem_bytes(false) <= kSmemBudget && smem_bytes(true) <= kSmemBudget, "one CTA's shared memory");

// A block that leaves because a wait has run out: what it has issued may still run, and boxes may be on their way to shared memory
// that is another block's next. A commit behind the MMAs and everyone's last requests are waited for, with a limit
template <bool kFp8>
__device__ __noinline__ void drain(Ctl* ctl, int loaders, bool q_box) {
  volatile int32_t never = 0;
  mbar_init(smem_u32(&ctl->drained), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  tc_commit(smem_u32(&ctl->drained));
  wait_inline(smem_u32(&ctl->drained), 0, &never, nullptr);
  if (q_box) wait_inline(smem_u32(&ctl->q_full), ctl->asked_q & 1u, &never, nullptr);
  for (int k = 0; k < loaders; ++k)
    for (int i = 0; i < (kFp8 ? kStages : slots_of(kFp8)); ++i)
      wait_inline(smem_u32(kFp8 ? &ctl->st_full[i] : &ctl->full[i]), last_request(i, ctl->asked[k] & 0xFF, (uint32_t)ctl->asked[k] >> 8), &never, nullptr);
}

__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }
// ---- two values at once; the largest of three ------------------------------------------------------------------
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7}; fma.rn.f32x2 x, x, y, z; mov.b64 {%0, %1}, x; }"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// cap tanh(x y1) for two scores, as `capped` forms it
__device__ __forceinline__ float2 capped2(float2 x, float y1, float cap) {
  const float2 y = mul2(x, {y1, y1}), t = mul2(y, y), z = mul2(y, {2.88539008f, 2.88539008f});
  float2 near = fma2(t, {-17.f / 315.f, -17.f / 315.f}, {2.f / 15.f, 2.f / 15.f});
  near = fma2(t, near, {-1.f / 3.f, -1.f / 3.f});
  near = mul2(y, fma2(t, near, {1.f, 1.f}));
  const float2 e = add2({ex2(z.x), ex2(z.y)}, {1.f, 1.f});
  const float2 far = fma2({rcp(e.x), rcp(e.y)}, {-2.f, -2.f}, {1.f, 1.f});
  return mul2({fabsf(y.x) < 0.25f ? near.x : far.x, fabsf(y.y) < 0.25f ? near.y : far.y}, {cap, cap});
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 16-byte piece c of row r in blocks of 128-byte rows, 128B swizzle
__device__ __forceinline__ uint32_t piece(int r, int c) { return (uint32_t)((c >> 3) * kBlockBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4)); }

// kWide: heads of more than 128 values (one tile of rows, two slots per key or value tile). kForm: scores with a form, or a
// scale that is not positive
template <bool kWide, bool kFp8, bool kForm>
__global__ void __launch_bounds__(threads_of(kFp8), 1) prompt_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                                                             const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Args a) {
  const PromptParams& p = a.p;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t q_smem = (raw + 1023u) & ~1023u;
  const uint32_t ring = q_smem + kQBytes;
  constexpr int kSlots = slots_of(kFp8);
  const int loaders = a.box > 0 ? loaders_of(kFp8) : 1, helpers = helpers_of(kFp8) + loaders_of(kFp8) - loaders;
  const uint32_t stages = ring + kSlots * kSlotBytes;
  const uint32_t staging = stages + (kFp8 ? kStages * kStageBytes : 0);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem_raw + (staging + 8 * staging_bytes(kFp8) - raw));
  volatile int32_t* abort_flag = &ctl->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D = p.D, G = p.G;
  constexpr int kSlotsPerTile = kWide ? 2 : 1;
  constexpr int kPair = kWide ? 128 : 256;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), a.box == 0 ? helpers + loaders : kFp8 ? helpers / 2 : loaders);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&ctl->st_full[s]), loaders + 32);  // the boxes, and every lane's scale words
      mbar_init(smem_u32(&ctl->st_empty[s]), helpers);
    }
    mbar_init(smem_u32(&ctl->q_full), a.q_box ? 1 : helpers);
    mbar_init(smem_u32(&ctl->q_empty), 1);
    for (int i = 0; i < kMeta; ++i) {
      mbar_init(smem_u32(&ctl->k_meta[i]), 1);
      mbar_init(smem_u32(&ctl->v_go[i]), 1);
      mbar_init(smem_u32(&ctl->v_meta[i]), helpers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl->s_full[i]), 1);
      mbar_init(smem_u32(&ctl->p_full[i]), 4);
      mbar_init(smem_u32(&ctl->o_final[0][i]), 1);
      mbar_init(smem_u32(&ctl->o_final[1][i]), 1);
      mbar_init(smem_u32(&ctl->seg_full[i]), 1);
      mbar_init(smem_u32(&ctl->seg_empty[i]), 8 + 1 + loaders + helpers);
    }
    mbar_init(smem_u32(&ctl->o_done), 1);
    ctl->abort_flag = 0;
    ctl->asked_q = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 12 && lane == 0 && a.box > 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl->tmem_base)), "n"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  pdl_wait();

  auto wait = [&](uint64_t& bar, uint32_t parity) { return wait_inline(smem_u32(&bar), parity & 1u, abort_flag, p.err); };
  // the same for a whole warp, with one answer for all of it
  auto wait_warp = [&](uint64_t& bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };
  // A segment's key tiles are taken from the last to the first: where a bias falls with distance, the largest scores come
  // first, and the maximum stays
  auto first_of = [&](const Segment& s, int n) { return s.key0 + (s.tiles - 1 - n) * kKeys; };
  // whether some row that sees keys at all does not see all of the tile's (none sees those past its ends), and whether
  // values there were not finite
  auto partly_seen = [&](const Segment& s, int n) {
    const int first = first_of(s, n);
    return first < s.max_lo || first + kKeys > s.min_hi;
  };
  // (of the pc-th such tile. Barriers tell their phases apart by parity alone, so nobody may wait for one that lies two
  // behind or ahead of where it is: these are counted in tiles that all who meet there wait for.)
  auto bad_keys = [&](uint32_t pc, int w) {
    uint32_t y = 0;
    for (int h = 0; h < helpers; ++h) y |= *(volatile uint32_t*)&ctl->v_bad[pc % kMeta][h][w];
    return y;
  };
  auto not_finite = [&](uint32_t pc) { return (bad_keys(pc, 0) | bad_keys(pc, 1) | bad_keys(pc, 2) | bad_keys(pc, 3)) != 0; };
  auto arrive = [&](uint64_t& bar) { mbar_arrive(smem_u32(&bar)); };
  uint32_t seg_n = 0;                                 // segments read so far
  auto next_segment = [&](bool whole_warp) {
    uint64_t& bar = ctl->seg_full[seg_n & 1];
    if (!(whole_warp ? wait_warp(bar, seg_n >> 1) : wait(bar, seg_n >> 1))) return false;
    return ctl->seg[seg_n & 1].tiles > 0;
  };

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    more_registers<kFp8 ? 144 : 168>();
    const int tile = warp >> 2, wl = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(wl * 32) << 16);
    const uint32_t o_t = lanes + kOCol + (uint32_t)(tile * 128);
    uint32_t used[2] = {0, 0};                        // tiles that went through the S buffers
    uint32_t dones = 0, keys_n = 0, pc = 0;           // o_done phases; key tiles; those some row sees partly
    bool ok = true;
    while (ok && next_segment(true)) {
      const Segment& s = ctl->seg[seg_n & 1];         // read where it lies: registers are for the scores
      const bool mine = tile < s.nt;
      if (mine) {
        const int r_in = tile * 128 + wl * 32 + lane;             // row of the pair
        const int r = s.row0 + r_in;
        const bool valid = r < s.rows;
        int lo = 0, hi = 0x7FFFFFFF, pos = 0, g = 0;
        if (valid) {
          const int i = (int)fast_div((uint32_t)r, a.div_g);
          g = r - i * G;
          visible(p, s.s0, s.n, s.len, i, lo, hi, pos);
        }
        const float slope = kForm && p.form.slopes != nullptr && valid ? p.form.slopes[s.head * G + g] * 1.44269504f : 0.f;
        float m = -INFINITY, l = 0.f;
        // A score is x times + plus of what the loop below makes of a product: the product itself; with a form its score; or
        // capped alone, by up to 128, the reciprocal in the tanh (see `only_cap`): off by 2^-22 cap, where `capped2`, for any
        // cap, keeps a score's own bits at twice the price (8192 tokens capped at 30: 1143 us)
        const bool only_cap = kForm && p.form.slopes == nullptr && p.form.cap2 > 0.f && p.form.cap2 <= 128.f * 1.4427f;
        const float times = !kForm ? p.scale_log2 : only_cap ? 2.f * p.form.cap2 : 1.f, plus = only_cap ? p.form.cap2 : 0.f;
        const float to_exp = p.scale_log2 * p.form.cap_inv * 2.88539008f;
        // Tiles [whole_from, whole_to) are seen whole by every row of the warp, tiles [plain_from, plain_to) by every row of
        // the pair that sees any
        const int T = s.tiles, nt = s.nt, first_key = s.key0;
        const int whole_from = __reduce_max_sync(0xFFFFFFFFu, lo > first_key ? (lo - first_key + kKeys - 1) / kKeys : 0);
        const int whole_to = __reduce_min_sync(0xFFFFFFFFu, hi > first_key ? (hi - first_key) / kKeys : 0);
        const int plain_from = s.max_lo > first_key ? (s.max_lo - first_key + kKeys - 1) / kKeys : 0;
        const int plain_to = s.min_hi > first_key ? (s.min_hi - first_key) / kKeys : 0;
        uint32_t nth = used[nt == 2 ? tile : 0], other = used[1];
        for (int n = 0; n < T; ++n) {
          const int buf = nt == 2 ? tile : n & 1;
          const uint32_t s_t = lanes + (uint32_t)(buf * 128);
          const uint32_t kn = keys_n + n;
          const int place = T - 1 - n, key0 = first_of(s, n);
          // what can be done before the scores are there: the softmax's latency is what the tensor cores wait for
          if (!wait_warp(ctl->k_meta[kn % kMeta], kn / kMeta)) { ok = false; break; }
          const uint4 live = *reinterpret_cast<const uint4*>(ctl->live[kn % kMeta]);
          const bool full = __all_sync(0xFFFFFFFFu, place >= whole_from && place < whole_to && (live.x & live.y & live.z & live.w) == 0xFFFFFFFFu);
          if (nt == 2 || buf == 0 ? !wait_warp(ctl->s_full[buf], nth++) : !wait_warp(ctl->s_full[1], other++)) { ok = false; break; }
          tc_fence_after();
          if (!kForm && !full) {
            // masked before: hardly any tile is, and the loop below stays small
#pragma unroll 1
            for (int c = 0; c < kKeys; c += 32) {
              float y[32];
              tmem_ld32(s_t + c, y);
              const uint32_t sees = ctl->live[kn % kMeta][c >> 5] & bits_below(hi - key0 - c) & ~bits_below(lo - key0 - c);
              tmem_ld_wait();
              hold(y);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((sees >> e) & 1u)) y[e] = -INFINITY;
              tmem_st16(s_t + c, reinterpret_cast<const uint32_t*>(y));
              tmem_st16(s_t + c + 16, reinterpret_cast<const uint32_t*>(y + 16));
            }
            tmem_st_wait();
          }
          // Scores at a time: half a tile; a quarter over FP8 where 144 registers do not hold the form or the wide loop beside
          // half a tile's (8192 tokens capped at 30: 1000 us against 1086; heads of 256: 1035 against 1100; elsewhere halves are
          // better, bf16 462 against 499)
          constexpr int kCols = kFp8 && (kWide || kForm) ? 32 : 64;
          // In a loop: unrolled over a whole tile, instruction fetches took a third of the time. The
          // exponentials are formed with the maximum so far, while the half's own is found: o, the sum and P are in units of
          // 2^m, and m follows the true maximum only when that is kLag beyond it, which hardly ever happens after the first
          // tile; then the half is done again. At first m is that maximum and no whole number, so that the largest weight (a row's
          // only one, where it sees one key) is 1 and loses nothing as bf16: rows of documents of a few tokens were off by up to 2^-8 for it.
#pragma unroll 1
          for (int c = 0; c < kKeys; c += kCols) {
            float x[kCols];
            tmem_ld32(s_t + c, x);
            if constexpr (kCols == 64) tmem_ld32(s_t + c + 32, x + 32);
            tmem_ld_wait();
            hold(x);
            if (kForm) {
              // the form, two scores at a time
              if (only_cap) {
                // cap tanh(y) = cap - 2 cap / (1 + exp(2 y)): x becomes the negative reciprocal
#pragma unroll
                for (int j = 0; j < kCols; j += 2) {
                  const float2 z = mul2({x[j], x[j + 1]}, {to_exp, to_exp});
                  const float2 e = fma2({ex2(z.x), ex2(z.y)}, {-1.f, -1.f}, {-1.f, -1.f});
                  x[j] = rcp(e.x);
                  x[j + 1] = rcp(e.y);
                }
              } else if (p.form.cap2 > 0.f) {
                const float y1 = p.scale_log2 * p.form.cap_inv;
#pragma unroll
                for (int j = 0; j < kCols; j += 2) {
                  const float2 y = capped2({x[j], x[j + 1]}, y1, p.form.cap2);
                  x[j] = y.x;
                  x[j + 1] = y.y;
                }
              } else {
#pragma unroll
                for (int j = 0; j < kCols; ++j) x[j] *= p.scale_log2;
              }
              if (p.form.slopes != nullptr) {
                const float back = (float)(pos - key0 - c);
#pragma unroll
                for (int j = 0; j < kCols; ++j) x[j] = fmaf(-slope, fabsf(back - (float)j), x[j]);
              }
              if (!full) {
#pragma unroll
                for (int w = 0; w < kCols / 32; ++w) {
                  const uint32_t sees = ctl->live[kn % kMeta][c / 32 + w] & bits_below(hi - key0 - c - 32 * w) & ~bits_below(lo - key0 - c - 32 * w);
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (!((sees >> j) & 1u)) x[32 * w + j] = -INFINITY;
                }
              }
            }
            float mx[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = max3(x[e], x[4 + e], x[8 + e]);
#pragma unroll
            for (int j = 12; j < kCols - 4; j += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[j + e], x[j + 4 + e]);
            float top = fmaxf(max3(mx[0], mx[1], mx[2]), max3(mx[3], x[kCols - 4], max3(x[kCols - 3], x[kCols - 2], x[kCols - 1])));
            top = fmaf(top, times, plus);
            if (n == 0 && c == 0) m = top;            // (nothing is summed yet)
            const bool grown = top > m + kLag;
            const float base = m == -INFINITY ? 0.f : m;
            const float2 times2 = {times, times}, plus2 = {plus - base, plus - base};
            float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
            uint32_t w[kCols / 2];
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) {
              const float2 xx = {x[2 * j], x[2 * j + 1]};
              const float2 y = fma2(xx, times2, plus2);
              const float2 e = {ex2(y.x), ex2(y.y)};
              sum[j & 1] = add2(sum[j & 1], e);
              w[j] = pack_bf16(e.x, e.y);
            }
            if (__any_sync(0xFFFFFFFFu, grown)) {
              // m moves by a whole number, so that what there is so far is multiplied by a power of two: this tile's P, whose
              // weights may be 2^30 and come to as much as 1 now, keeps the one rounding it has had, and O and the sum theirs
              // (by the maximum's own growth, P was rounded three times and off by 2.3 * 2^-8). Over 2^126 and from a maximum
              // of -inf nothing is left of it, and m is the maximum
              const float by = ceilf(top - m);
              const float alpha = !grown ? 1.f : by < 127.f ? __uint_as_float((uint32_t)(127 - (int)by) << 23) : 0.f;
              if (grown) m = by < 127.f ? m + by : top;
              l *= alpha;
              if (n > 0) {
                if (nt == 1 && !wait_warp(ctl->o_done, dones + n - 1)) { ok = false; break; }
                tc_fence_after();
#pragma unroll 1
                for (int d = 0; d < D; d += 16) {
                  float y[16];
                  tmem_ld16(o_t + d, reinterpret_cast<uint32_t*>(y));
                  tmem_ld_wait();
                  hold(y);
#pragma unroll
                  for (int e = 0; e < 16; ++e) y[e] *= alpha;
                  tmem_st16(o_t + d, reinterpret_cast<const uint32_t*>(y));
                }
              }
              if (c > 0) {
                tmem_st_wait();                       // this tile's P so far
                const __nv_bfloat162 alpha2 = __float2bfloat162_rn(alpha);   // exact
#pragma unroll 1
                for (int d = 0; d < c / 2; d += 16) {
                  float y[16];
                  tmem_ld16(s_t + d, reinterpret_cast<uint32_t*>(y));
                  tmem_ld_wait();
                  hold(y);
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    __nv_bfloat162 z = *reinterpret_cast<__nv_bfloat162*>(&y[e]);
                    z = __hmul2(z, alpha2);
                    y[e] = *reinterpret_cast<float*>(&z);
                  }
                  tmem_st16(s_t + d, reinterpret_cast<const uint32_t*>(y));
                }
              }
              c -= kCols;
              continue;
            }
            tmem_st16(s_t + c / 2, w);                // over scores that have been read
            if constexpr (kCols == 64) tmem_st16(s_t + c / 2 + 16, w + 16);
            const float2 sums = add2(sum[0], sum[1]);
            l += sums.x + sums.y;
          }
          if (!ok) break;
          tmem_st_wait();
          if (place < plain_from || place >= plain_to) {
            // some row does not see all of the tile's keys: values that are not finite must not reach it
            const uint32_t now = pc++;
            if (!wait_warp(ctl->v_meta[now % kMeta], now / kMeta)) { ok = false; break; }
            if (not_finite(now)) {
              if (nt == 1 && n > 0 && !wait_warp(ctl->o_done, dones + n - 1)) { ok = false; break; }
              tc_fence_after();
#pragma unroll 1
              for (int d = 0; d < D; d += 16) {
                float y[16];
                if (n > 0) {
                  tmem_ld16(o_t + d, reinterpret_cast<uint32_t*>(y));
                  tmem_ld_wait();
                  hold(y);
                } else {                              // (the products of a first tile are then added, too)
#pragma unroll
                  for (int e = 0; e < 16; ++e) y[e] = 0.f;
                }
                for (int w = 0; w < 4; ++w) {
                  const uint32_t sees = ctl->live[kn % kMeta][w] & bits_below(hi - key0 - 32 * w) & ~bits_below(lo - key0 - 32 * w);
                  for (uint32_t left = bad_keys(now, w); left != 0; left &= left - 1) {
                    const int j = 32 * w + __ffs(left) - 1;
                    if (!__any_sync(0xFFFFFFFFu, (sees >> (j & 31)) & 1u)) continue;   // (past the sequence, maybe: no page)
                    uint32_t pw = tmem_ld1(s_t + (j >> 1));
                    tmem_ld_wait();
                    asm volatile("" : "+r"(pw));
                    const float pj = (j & 1) ? engram::bf16_hi(pw) : engram::bf16_lo(pw);
                    const int at = (int)fast_div((uint32_t)(key0 + j), p.cache.div_page), in_page = key0 + j - at * p.cache.page_size;
                    const int64_t page = p.table[(int64_t)s.b * p.table_stride + at];
                    const uint8_t* row = p.cache.v + page * p.cache.page_b + s.head * p.cache.head_b + in_page * p.cache.tok_b;
                    const uint8_t* scales = p.cache.vs + page * p.cache.spage_b + s.head * p.cache.shead_b + in_page * p.cache.stok_b;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                      float v;
                      if (kFp8) {
                        uint32_t f0, f1;
                        e4m3x4_to_f16x2(row[d + e], f0, f1);
                        v = __low2float(*reinterpret_cast<const __half2*>(&f0)) * __uint_as_float((uint32_t)scales[(d + e) / 32] << 23);
                      } else {
                        v = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[d + e] << 16);
                      }
                      if (((sees >> (j & 31)) & 1u) && !(fabsf(v) <= 3.3895314e38f)) y[e] = fmaf(pj, v, y[e]);
                    }
                  }
                }
                tmem_st16(o_t + d, reinterpret_cast<const uint32_t*>(y));
              }
              tmem_st_wait();
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive(ctl->p_full[buf]);
        }
        if (!ok) break;
        // ---- the segment's result
        if (!wait_warp(ctl->o_final[tile][seg_n & 1], seg_n >> 1)) { ok = false; break; }
        tc_fence_after();
        const int64_t token = (int64_t)s.s0 + (valid ? (int)fast_div((uint32_t)r, a.div_g) : 0);
        const int h = s.head * G + g;
        if (s.whole && p.out != nullptr) {
          // through shared memory, so that rows leave in longer pieces than a thread's 16 bytes
          constexpr int kPieces = staging_pieces(kFp8), kStaged = 8 * kPieces;
          const float inv = 1.f / l;
          const int64_t row = token * p.out_ts + (int64_t)h * p.out_hs;
          const uint32_t stage = staging + (uint32_t)(warp * staging_bytes(kFp8));
          auto place = [&](int r, int c) { return stage + (uint32_t)(r * 16 * kPieces + ((c ^ ((r * kPieces >> 3) & (kPieces - 1))) << 4)); };
#pragma unroll 1
          for (int d = 0; d < D; d += kStaged) {
            float y[kStaged];
            if (kStaged == 32) tmem_ld32(o_t + d, y); else tmem_ld16(o_t + d, reinterpret_cast<uint32_t*>(y));
            tmem_ld_wait();
            hold(y);
#pragma unroll
            for (int e = 0; e < kStaged; ++e) y[e] = l == 0.f ? 0.f : y[e] * inv;   // (see emit16)
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
              uint32_t v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = pack_bf16(y[8 * c + 2 * e], y[8 * c + 2 * e + 1]);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(place(lane, c)), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
              const int from = 32 / kPieces * k + lane / kPieces, c = lane % kPieces;
              const int64_t to = __shfl_sync(0xFFFFFFFFu, row, from);
              uint4 v;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(place(from, c)) : "memory");
              if (s.row0 + tile * 128 + wl * 32 + from < s.rows && d + 8 * c < D) *reinterpret_cast<uint4*>(p.out + to + d + 8 * c) = v;
            }
            __syncwarp();
          }
          if (valid && p.lse != nullptr) p.lse[token * (p.Hk * G) + h] = l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
        } else if (s.whole) {
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            float y[16];
            tmem_ld16(o_t + d, reinterpret_cast<uint32_t*>(y));
            tmem_ld_wait();
            hold(y);
            if (valid) emit16(p, token, h, d, y, m, l);
          }
        } else {
          float* slot = a.parts + (int64_t)(2 * blockIdx.x + ((int)blockIdx.x == s.c_first ? 1 : 0)) * a.slot_floats;
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            float y[16];
            tmem_ld16(o_t + d, reinterpret_cast<uint32_t*>(y));
            tmem_ld_wait();
            hold(y);
            if (valid) {
#pragma unroll
              for (int e = 0; e < 4; ++e) __stcg(part_o(slot, kPair, d / 4 + e, r_in), make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]));
            }
          }
          if (valid) __stcg(part_ml(slot, kPair, D, r_in), make_float2(m, l));
          if (a.join) {
            __syncwarp();
            uint32_t last = 0;
            if (lane == 0) {
              uint32_t* counter = a.counters + s.c_first * 8 + warp;
              __threadfence();
              asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(last) : "l"(counter) : "memory");
              last = last == (uint32_t)(s.c_last - s.c_first);
              __threadfence();
            }
            if (__shfl_sync(0xFFFFFFFFu, last, 0) && valid)
#pragma unroll 1
              for (int d = 0; d < D; d += 16) join16(a, s.c_first, s.c_last, kPair, r_in, token, h, d);
          }
        }
        tc_fence_before();
      }
      // The second tile's warps stay with a segment of one tile until its sums are final, so that every barrier is at the phase that
      // they have counted when they go on: one's phases are told apart by parity alone. (Not by its scores, tile by tile: nobody
      // waits for these warps there, and while they still join the last segment's rows the scores may be many phases ahead.
      // The segment after next is not handed out without them, so that of two barriers for sums neither is.)
      if (!kWide && !mine) {
        ok = wait_warp(ctl->o_final[1][seg_n & 1], seg_n >> 1);
        for (int n = 0; n < s.tiles; ++n) pc += partly_seen(s, n);
      }
      if (s.nt == 2) {
        used[0] += s.tiles;
        used[1] += s.tiles;
      } else {
        used[0] += (s.tiles + 1) >> 1;
        used[1] += s.tiles >> 1;
        dones += s.tiles;
      }
      keys_n += s.tiles;
      __syncwarp();
      if (lane == 0) arrive(ctl->seg_empty[seg_n & 1]);
      ++seg_n;
    }
  } else {
    fewer_registers<kFp8 ? 64 : 88>();
    if (warp == 8) {
      // -------------------------------------------------------------- MMA
      // The warp stays together: every lane waits, one issues. (Uniform registers hold the descriptors.)
      {
        const bool leader = elect_one();
        uint32_t used[2] = {0, 0}, pc = 0, q_n = 0;
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t id_s = idesc_of(kKeys, false), id_o = idesc_of(min(128, D), true), id_o2 = idesc_of(kWide ? D - 128 : 16, true);
        const uint64_t ring_k = smem_desc_sw128(ring), ring_v = smem_desc_mn(ring);
        while (ok && next_segment(true)) {
          const Segment s = ctl->seg[seg_n & 1];
          const int T = s.tiles;
          auto next_slot = [&] {
            if (++slot == kSlots) { slot = 0; phase ^= 1u; }
          };
          // S(buf) (+)= Q(t) K^T over the part of the heads that lies in a slot. (One thread issues all of it: descriptors
          // are sums with constants, 16 MMAs without a loop.)
          auto qk = [&](int t, int buf, int at, int part) {
            const uint64_t q0 = smem_desc_sw128(q_smem) + (uint64_t)((t + part) * (2 * kBlockBytes >> 4));
            const uint64_t k0 = ring_k + (uint64_t)(at * (kSlotBytes >> 4));
            const uint32_t to = tmem + buf * 128;
            const int steps = kWide && part == 0 ? 8 : (kWide ? D - 128 : D) / 16;
            if (leader) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint64_t off = (uint64_t)(((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4);
                if (k < steps) tc_mma(to, q0 + off, k0 + off, id_s, part > 0 || k > 0 ? 1u : 0u);
              }
            }
            __syncwarp();
          };
          // O(t) (+)= P(buf) V for the values that lie in a slot
          auto pv = [&](int t, int buf, int at, int part, bool add) {
            const uint64_t v0 = ring_v + (uint64_t)(at * (kSlotBytes >> 4));
            const uint32_t to = tmem + kOCol + t * 128 + part * 128, from = tmem + buf * 128, id = part == 0 ? id_o : id_o2;
            if (leader) {
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k) tc_mma_ts(to, from + k * 8, v0 + (uint64_t)(k * (2048 >> 4)), id, add || k > 0 ? 1u : 0u);
            }
            __syncwarp();
          };
          auto commit = [&](uint64_t& bar) {
            if (leader) tc_commit(smem_u32(&bar));
            __syncwarp();
          };
          if (!wait_warp(ctl->q_full, q_n)) break;
          if (!kWide && s.nt == 2) {
            if (!wait_warp(ctl->full[slot], phase)) break;
            tc_fence_after();
            for (int t = 0; t < 2; ++t) {
              qk(t, t, slot, 0);
              commit(ctl->s_full[t]);
            }
            commit(ctl->empty[slot]);
            if (T == 1) commit(ctl->q_empty);
            next_slot();
            for (int n = 0; n < T; ++n) {
              const int v = slot;
              if (!wait_warp(ctl->full[slot], phase)) { ok = false; break; }
              next_slot();
              const bool partly = partly_seen(s, n);
              if (partly && !wait_warp(ctl->v_meta[pc % kMeta], pc / kMeta)) { ok = false; break; }
              const bool add = n > 0 || (partly && not_finite(pc));
              pc += partly;
              for (int t = 0; t < 2; ++t) {
                if (!wait_warp(ctl->p_full[t], used[t] + n)) { ok = false; break; }
                tc_fence_after();
                pv(t, t, v, 0, add);
                if (t == 1) commit(ctl->empty[v]);
                if (n + 1 < T) {
                  if (t == 0) {                       // (not before these products: they need no keys)
                    if (!wait_warp(ctl->full[slot], phase)) { ok = false; break; }
                    tc_fence_after();
                  }
                  qk(t, t, slot, 0);
                  commit(ctl->s_full[t]);
                } else {
                  commit(ctl->o_final[t][seg_n & 1]);
                }
              }
              if (!ok) break;
              if (n + 1 < T) {
                commit(ctl->empty[slot]);
                if (n + 2 == T) commit(ctl->q_empty);
                next_slot();
              }
            }
            used[0] += T;
            used[1] += T;
          } else {
            auto keys = [&](int n) {                  // the scores of key tile n, into its buffer
              for (int part = 0; part < kSlotsPerTile; ++part) {
                if (!wait_warp(ctl->full[slot], phase)) return false;
                tc_fence_after();
                qk(0, n & 1, slot, part);
                commit(ctl->empty[slot]);
                next_slot();
              }
              commit(ctl->s_full[n & 1]);
              if (n + 1 == T) commit(ctl->q_empty);
              return true;
            };
            ok = keys(0) && (T < 2 || keys(1));
            for (int n = 0; ok && n < T; ++n) {
              if (!wait_warp(ctl->p_full[n & 1], used[n & 1] + (n >> 1))) { ok = false; break; }
              const bool partly = partly_seen(s, n);
              if (partly && !wait_warp(ctl->v_meta[pc % kMeta], pc / kMeta)) { ok = false; break; }
              const bool add = n > 0 || (partly && not_finite(pc));
              pc += partly;
              for (int part = 0; part < kSlotsPerTile; ++part) {
                if (!wait_warp(ctl->full[slot], phase)) { ok = false; break; }
                tc_fence_after();
                pv(0, n & 1, slot, part, add);
                commit(ctl->empty[slot]);
                next_slot();
              }
              if (!ok) break;
              commit(ctl->o_done);
              if (n + 1 == T) {
                commit(ctl->o_final[0][seg_n & 1]);
                if (!kWide) commit(ctl->o_final[1][seg_n & 1]);
              }
              if (n + 2 < T) ok = keys(n + 2);
            }
            used[0] += (T + 1) >> 1;
            used[1] += T >> 1;
          }
          if (!ok) break;
          ++q_n;
          if (leader) arrive(ctl->seg_empty[seg_n & 1]);
          ++seg_n;
        }
      }
    } else if (warp == 9) {
      // -------------------------------------------------------------- the CTA's share
      const int64_t U = a.header->places, per = a.header->per_cta;
      const int64_t total = U * p.Hk, at0 = per * blockIdx.x, at1 = min(total, at0 + per);
      if (lane == 0) {
        bool ok = true;
        auto put = [&](const Segment& s) {
          if (seg_n >= 2 && !wait(ctl->seg_empty[seg_n & 1], (seg_n >> 1) - 1)) return false;
          ctl->seg[seg_n & 1] = s;
          arrive(ctl->seg_full[seg_n & 1]);
          ++seg_n;
          return true;
        };
        if (at0 < at1) {
          Start st = a.starts[blockIdx.x];
          int64_t base = st.head * U;
          const int E = (int)a.header->entries;
          while (ok && st.head < p.Hk) {
            const Entry e = a.entries[st.entry];
            const int64_t run0 = base + e.place + kRunCost;       // its first tile's place
            if (e.units > 0) {
              if (base + e.place >= at1) break;
              const int64_t from = max(run0, at0), to = min(run0 + e.units, at1);
              if (from < to) {
                Segment s;
                s.tiles = (int)(to - from);
                s.nt = !kWide && e.rows - e.row0 > 128 ? 2 : 1;
                s.b = e.b;
                s.head = st.head;
                s.row0 = e.row0;
                s.rows = e.rows;
                s.s0 = e.s0;
                s.n = e.n;
                s.len = e.len;
                s.key0 = e.key0 + (int)(from - run0) * kKeys;
                s.hull_hi = e.hi;
                s.max_lo = e.max_lo;
                s.min_hi = e.min_hi;
                s.c_first = (int)(run0 / per);
                s.c_last = (int)((run0 + e.units - 1) / per);
                s.whole = s.c_first == s.c_last;
                ok = put(s);
              }
            }
            if (++st.entry == E) {
              st.entry = 0;
              ++st.head;
              base += U;
            }
          }
        }
        Segment end;
        end.tiles = 0;
        if (ok) put(end);
      }
      __syncwarp();
    } else if (warp >= 12 && warp < 12 + loaders) {
      // -------------------------------------------------------------- pages, and boxes of K and V
      const bool leader = elect_one();
      const int loader = warp - 12;
      int slot = 0, stage = 0;
      uint32_t phase = 0, st_phase = 0, kn = 0, pc = 0;
      bool ok = true;
      while (ok && next_segment(true)) {
        const Segment& s = ctl->seg[seg_n & 1];
        // keys run `lead` tiles ahead of values
        const int T = s.tiles, lead = min(T, !kWide && s.nt == 2 ? 1 : 2);
        const int head = s.head, b = s.b, first_key = s.key0, hull_hi = s.hull_hi;
        // Pages and places of 32 boxes at a time, a lane each: this loop feeds the tensor cores, so looking up and dividing
        // is done once for many tiles. Values are in the older batch, keys in that or the next (a batch is two tiles or more).
        // Rows one by one: the pages are only looked at, key by key; a "box" is a key then, a batch a quarter of a tile.
        const int box_log = a.box > 0 ? 31 - __clz(a.box) : 0, batch_log = 5 + box_log - 7;   // tiles in a batch, log 2
        int pg[2] = {-1, -1}, pl[2] = {0, 0};
        uint32_t there[2] = {0, 0};
        auto request = [&](int batch, int& page, int& place) {
          const int at = ((batch << 5) + lane) << box_log;    // (tile for tile, from the last to the first)
          const int pos = first_key + (T - 1 - at / kKeys) * kKeys + at % kKeys;
          const int i = (int)fast_div((uint32_t)pos, p.cache.div_page);
          page = -1;
          place = pos - i * p.cache.page_size;
          if (pos < hull_hi && pos >= first_key) {     // (before: past the last tile)
            page = p.table[(int64_t)b * p.table_stride + i];
            if (page < 0 || page >= p.cache.num_pages) {
              page = -1;
              if (p.err != nullptr && loader == 0) atomicOr(p.err, ENGRAM_ERR_PAGE);
            }
          }
        };
        int batch = 0;                                // of the values
        if (a.box > 0) {
          request(0, pg[0], pl[0]);
          request(1, pg[1], pl[1]);
          there[0] = __ballot_sync(0xFFFFFFFFu, pg[0] >= 0);
          there[1] = __ballot_sync(0xFFFFFFFFu, pg[1] >= 0);
        }
        const int boxes = kKeys >> box_log;           // of a tile
        int next_k = 0, next_v = 0;
        while (ok && next_v < T) {
          const bool values = next_k == min(T, next_v + lead);
          const int n = values ? next_v : next_k;
          const bool next_batch = a.box > 0 && (n >> batch_log) != batch;
          const int page = next_batch ? pg[1] : pg[0], place = next_batch ? pl[1] : pl[0];
          const int at = (n * boxes) & 31;            // the tile's first box in its batch
          if (!values && loader == 0) {
            const int m = (kn + n) % kMeta;
            if (a.box > 0) {
              const uint32_t all = boxes == 16 ? 0xFFFFu : (1u << boxes) - 1u, has = ((next_batch ? there[1] : there[0]) >> at) & all;
              if (lane < 4) {
                uint32_t live = has == all ? 0xFFFFFFFFu : 0u;
                if (has != all)
                  for (int k = 0; k < 32; k += 1 << min(box_log, 5))
                    if ((has >> ((32 * lane + k) >> box_log)) & 1u) live |= (box_log >= 5 ? 0xFFFFFFFFu : (1u << (1 << box_log)) - 1u) << k;
                ctl->live[m][lane] = live;
              }
            } else {
              for (int w = 0; w < 4; ++w) {
                int y, z;
                request(n * 4 + w, y, z);
                const uint32_t live = __ballot_sync(0xFFFFFFFFu, y >= 0);
                if (lane == w) ctl->live[m][w] = live;
              }
            }
            __syncwarp();
            if (lane == 0) arrive(ctl->k_meta[m]);
          }
          for (int part = 0; part < kSlotsPerTile; ++part) {
            if (kFp8 && a.box > 0 ? !wait_warp(ctl->st_empty[stage], st_phase ^ 1u) : !wait_warp(ctl->empty[slot], phase ^ 1u)) { ok = false; break; }
            if (values && part + 1 == kSlotsPerTile && loader == 0 && partly_seen(s, n)) {
              if (lane == 0) arrive(ctl->v_go[pc % kMeta]);
              ++pc;
            }
            if (a.box > 0) {
              const bool two = !kFp8 && D - part * 128 > 64;   // blocks of 64 values
              const uint32_t dst = kFp8 ? stages + (uint32_t)(stage * kStageBytes) : ring + (uint32_t)(slot * kSlotBytes);
              const uint32_t bar = smem_u32(kFp8 ? &ctl->st_full[stage] : &ctl->full[slot]);
              // this loader's boxes: every so many from its own on
              const int mine = (boxes - loader + loaders - 1) / loaders;
              if (leader) mbar_expect_tx(bar, (uint32_t)((mine << box_log) * (two ? 256 : 128)));
              // One lane requests all boxes (lanes of their own would take turns all the same, at a higher price). A page that
              // is not there reads as zeros.
              const CUtensorMap* map = values ? &tm_v : &tm_k;
              for (int k = loader; k < boxes; k += loaders) {
                const int y = __shfl_sync(0xFFFFFFFFu, place, at + k), z = __shfl_sync(0xFFFFFFFFu, page, at + k);
                const uint32_t to = dst + (uint32_t)((k << box_log) * 128);
                if (leader) {
                  tma_load_4d(to, map, bar, part * 128, y, head, z);
                  if (two) tma_load_4d(to + kBlockBytes, map, bar, part * 128 + 64, y, head, z);
                }
              }
              if (kFp8 && loader == 0) {
                // scale words: keys 4 * lane .. + 3, all in one box
                const int key = 4 * lane, from_lane = at + (key >> box_log);
                const int pb = __shfl_sync(0xFFFFFFFFu, page, from_lane);
                const int first_place = __shfl_sync(0xFFFFFFFFu, place, from_lane) + (key & ((1 << box_log) - 1));
                const uint8_t* from = (values ? p.cache.vs : p.cache.ks) + head * p.cache.shead_b + 4 * part +
                    (pb >= 0 ? (int64_t)((uint64_t)(uint32_t)pb * p.cache.spage_u + (uint64_t)(uint32_t)first_place * p.cache.stok_u) << 2 : 0);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + kBlockBytes + (uint32_t)(key + k) * 4),
                               "l"(from + (pb >= 0 ? k * p.cache.stok_b : 0)), "r"(pb >= 0 ? 4 : 0) : "memory");
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
              }
            }
            // Rows one by one: nothing to bring, but the slot is not full without this warp. What waits for a slot has a part in filling
            // it, everywhere: a barrier that went on without this warp would be two phases ahead of its wait, and parity does not
            // tell that from the phase before
            if (a.box == 0 && lane == 0) arrive(ctl->full[slot]);
            if (kFp8 && a.box > 0) {
              if (++stage == kStages) { stage = 0; st_phase ^= 1u; }
            } else if (++slot == kSlots) {
              slot = 0;
              phase ^= 1u;
            }
          }
          if (values) {
            ++next_v;
            if (a.box > 0 && (next_v >> batch_log) != batch && next_v < T) {
              ++batch;
              pg[0] = pg[1];
              pl[0] = pl[1];
              there[0] = there[1];
              request(batch + 1, pg[1], pl[1]);
              there[1] = __ballot_sync(0xFFFFFFFFu, pg[1] >= 0);
            }
          } else {
            ++next_k;
          }
        }
        if (!ok) break;
        kn += T;
        __syncwarp();
        if (lane == 0) arrive(ctl->seg_empty[seg_n & 1]);
        ++seg_n;
      }
      cp_async_commit();
      cp_async_wait<0>();
      if (lane == 0) ctl->asked[loader] = kFp8 ? stage | st_phase << 8 : slot | phase << 8;
    } else {
      // -------------------------------------------------------------- Q; rows to convert, to fetch or to look through
      const int w = warp < 12 ? warp - 10 : warp - 10 - loaders;
      const bool rows_here = kFp8 || a.box == 0;      // the slots are filled here
      uint32_t pc = 0, q_n = 0, seq = 0;              // tiles that some row sees partly, segments, slots so far
      bool ok = true;
      while (ok && next_segment(true)) {
        const Segment& s = ctl->seg[seg_n & 1];
        const int T = s.tiles, lead = min(T, !kWide && s.nt == 2 ? 1 : 2);
        // ---- Q: boxes of whole tokens where a tile has whole tokens, else 32 rows at a time
        if ((!a.q_box || w == 0) && q_n > 0 && !wait_warp(ctl->q_empty, q_n - 1)) break;
        if (a.q_box) {
          if (w == 0 && elect_one()) {
            const int blocks = (D + 63) / 64;
            const uint32_t bar = smem_u32(&ctl->q_full);
            ctl->asked_q = (int)q_n;
            mbar_expect_tx(bar, (uint32_t)(s.nt * blocks * kBlockBytes));
            for (int t = 0; t < s.nt; ++t)
              for (int k = 0; k < blocks; ++k)
                tma_load_3d(q_smem + (uint32_t)((t * 2 + k) * kBlockBytes), &tm_q, bar, k * 64, s.head * G,
                            s.s0 + (int)fast_div((uint32_t)(s.row0 + t * 128), a.div_g));
          }
          __syncwarp();
        } else {
          const int pieces = D / 8;
          for (int g = w; g < s.nt * 4; g += helpers) {
            const int r = s.row0 + g * 32 + lane;
            int64_t off = -1;
            if (r < s.rows) {
              const int i = (int)fast_div((uint32_t)r, a.div_g);
              off = ((int64_t)s.s0 + i) * p.q.ts + (int64_t)(s.head * G + (r - i * G)) * p.q.hs;
            }
            constexpr int kLanes = kWide ? 32 : 16;   // of a row
            const int c = lane % kLanes, sub = lane / kLanes;
            const uint32_t to = q_smem + (uint32_t)((g >> 2) * 2) * kBlockBytes;
#pragma unroll 4
            for (int k = 0; k < kLanes; ++k) {
              const int row = k * (32 / kLanes) + sub;
              const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row);
              if (c < pieces) copy16_or_zero(to + piece((g & 3) * 32 + row, c), static_cast<const uint16_t*>(p.q.data) + (o < 0 ? 0 : o) + c * 8, o >= 0);
            }
          }
          cp_async_commit();
          cp_async_wait<0>();
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) arrive(ctl->q_full);
        }
        uint32_t bad[4] = {0, 0, 0, 0};               // keys of the tile in which this thread has found a value that is not finite
        // eight bf16 of key `row`: what is not finite becomes zero, and is noted
        auto clean = [&](uint32_t (&v)[4], int row, int first) {
          uint32_t ones = 0;                          // exponents of ones: 0x7F80 + 0x80 carries into the sign's place
#pragma unroll
          for (int e = 0; e < 4; ++e) ones |= (v[e] & 0x7F807F80u) + 0x00800080u;
          if ((ones & 0x80008000u) == 0) return false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t lo = (v[e] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u, hi = (v[e] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
            v[e] &= ~(lo | hi);
          }
          if (first + row < s.hull_hi) {              // (what lies behind the sequence is nobody's)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (row >> 5 == x) bad[x] |= 1u << (row & 31);
          }
          return true;
        };
        // rows [0, before) and [past, kKeys) of tile n are those that some row may not see
        auto seen_before = [&](int n) { return min(max(s.max_lo - first_of(s, n), 0), kKeys); };
        auto seen_past = [&](int n) { return min(max(s.min_hi - first_of(s, n), 0), kKeys); };
        // those of rows [row0, row1) of a slot, two at a time, the next ones `step` on; four turns under way together
        auto look_through = [&](uint32_t slot_at, int pieces, int row0, int row1, int step, int n) {
          const int c = lane & 15, before = seen_before(n), past = seen_past(n), first = first_of(s, n);
          for (int row = row0 + (lane >> 4); row < row1; row += 4 * step) {
            uint32_t v[4][4], ones = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int r = row + u * step;
              v[u][0] = v[u][1] = v[u][2] = v[u][3] = 0;
              if (r < row1 && c < pieces && (r < before || r >= past))
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[u][0]), "=r"(v[u][1]), "=r"(v[u][2]), "=r"(v[u][3])
                             : "r"(slot_at + piece(r, c)) : "memory");
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int e = 0; e < 4; ++e) ones |= (v[u][e] & 0x7F807F80u) + 0x00800080u;
            if ((ones & 0x80008000u) != 0) {
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int r = row + u * step;
                if (clean(v[u], r, first))
                  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(slot_at + piece(r, c)), "r"(v[u][0]), "r"(v[u][1]), "r"(v[u][2]),
                               "r"(v[u][3]) : "memory");
              }
            }
          }
          __syncwarp();
        };
        auto note = [&] {                             // a value tile that some row sees partly is through
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t any = __reduce_or_sync(0xFFFFFFFFu, bad[x]);
            if (lane == x) ctl->v_bad[pc % kMeta][w][x] = any;
            bad[x] = 0;
          }
          __syncwarp();
          if (lane == 0) arrive(ctl->v_meta[pc % kMeta]);
          ++pc;
        };
        if (!rows_here) {
          // value tiles that some row sees partly, once they have landed (and not before they are asked for: the slot's
          // barrier may be a phase behind)
          for (int n = 0; ok && n < T; ++n) {
            if (!partly_seen(s, n)) continue;
            if (!wait_warp(ctl->v_go[pc % kMeta], pc / kMeta)) { ok = false; break; }
            for (int part = 0; part < kSlotsPerTile; ++part) {
              const uint32_t at = seq + (uint32_t)((min(T, n + lead) + n) * kSlotsPerTile + part);
              if (!wait_warp(ctl->full[at % kSlots], at / kSlots)) { ok = false; break; }
              look_through(ring + (at % kSlots) * kSlotBytes, min(16, (D - part * 128) / 8), 2 * w, kKeys, 2 * helpers, n);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (ok) note();
          }
          seq += (uint32_t)(2 * T * kSlotsPerTile);
        } else {
          int next_k = 0, next_v = 0;
          while (ok && next_v < T) {
            const bool values = next_k == min(T, next_v + lead);
            const int n = values ? next_v++ : next_k++;
            const bool partly = values && partly_seen(s, n);
            for (int part = 0; part < kSlotsPerTile; ++part, ++seq) {
              const uint32_t dst = ring + (seq % kSlots) * kSlotBytes;
              const int pieces = min(16, (D - part * 128) / 8);
              // codes (16 of a row) to bf16
              auto convert = [&](const uint4& x, float scale, int row, int c) {
                const uint32_t codes[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  uint32_t y[4];
#pragma unroll
                  for (int z = 0; z < 2; ++z) {
                    uint32_t f0, f1;
                    e4m3x4_to_f16x2(codes[2 * e + z], f0, f1);
                    const float2 g0 = mul2(__half22float2(*reinterpret_cast<const __half2*>(&f0)), {scale, scale});
                    const float2 g1 = mul2(__half22float2(*reinterpret_cast<const __half2*>(&f1)), {scale, scale});
                    y[2 * z] = pack_bf16(g0.x, g0.y);
                    y[2 * z + 1] = pack_bf16(g1.x, g1.y);
                  }
                  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + piece(row, 2 * c + e)), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
                }
              };
              if (kFp8 && a.box > 0) {
                const uint32_t st = seq % kStages, from = stages + st * kStageBytes;
                // Half of the warps take a slot, the others the next one: what a slot costs beside the conversion (barriers, the
                // fence) is then hidden behind the other's. All wait for every stage and give it back, so that no barrier is two
                // phases away from anyone who waits for it (a slot's is behind its stage's)
                if (!wait_warp(ctl->st_full[st], seq / kStages)) { ok = false; break; }
                if ((int)(seq & 1u) != (w >> 2)) {
                  if (lane == 0) arrive(ctl->st_empty[st]);
                  continue;
                }
                if (seq >= kSlots && !wait_warp(ctl->empty[seq % kSlots], seq / kSlots - 1)) { ok = false; break; }
                // a lane takes 16 codes of a row: eight lanes that store at once have four pieces of two rows, which the
                // swizzle keeps in different banks
                const int per_row = pieces / 2, c = (lane & 3) | (lane >> 1 & 4);
#pragma unroll 1
                for (int row = (w & 3) * 4 + ((lane >> 2 & 1) | (lane >> 3 & 2)); row < kKeys; row += helpers * 2) {
                  if (c >= per_row) continue;
                  uint4 x;
                  uint32_t word;
                  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(from + row * 128 + c * 16) : "memory");
                  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(word) : "r"(from + kBlockBytes + row * 4) : "memory");
                  convert(x, __uint_as_float(((word >> (8 * (c >> 1))) & 0xFFu) << 23), row, c);
                }
                __syncwarp();
                if (lane == 0) arrive(ctl->st_empty[st]);
                if (partly) {                         // (the same rows: four of every sixteen)
                  look_through(dst, pieces, (w & 3) * 4, kKeys, helpers * 2, n);
                  look_through(dst, pieces, (w & 3) * 4 + 2, kKeys, helpers * 2, n);
                }
              } else {
                // a run of rows for each warp; a lane looks one up
                if (seq >= kSlots && !wait_warp(ctl->empty[seq % kSlots], seq / kSlots - 1)) { ok = false; break; }
                // (more helpers then: 128 / 5 or 9)
                constexpr int kRows = (kKeys + helpers_of(kFp8) + loaders_of(kFp8) - 2) / (helpers_of(kFp8) + loaders_of(kFp8) - 1);
                const int row0 = w * kRows, rows = min(kRows, kKeys - row0);
                const int pos = first_of(s, n) + row0 + lane;
                int64_t off = -1, soff = 0;
                if (lane < rows && pos < s.hull_hi) {
                  const int i = (int)fast_div((uint32_t)pos, p.cache.div_page), place = pos - i * p.cache.page_size;
                  const int64_t page = p.table[(int64_t)s.b * p.table_stride + i];
                  if (page >= 0 && page < p.cache.num_pages) {
                    off = page * p.cache.page_b + s.head * p.cache.head_b + place * p.cache.tok_b;
                    soff = page * p.cache.spage_b + s.head * p.cache.shead_b + place * p.cache.stok_b;
                  }
                }
                const uint8_t* from = values ? p.cache.v : p.cache.k;
                if (!kFp8) {
                  const int c = lane & 15, sub = lane >> 4;
                  for (int k = 0; k < (kRows + 1) / 2; ++k) {
                    const int row = 2 * k + sub;
                    const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row);
                    if (row < rows && c < pieces) copy16_or_zero(dst + piece(row0 + row, c), from + (o < 0 ? 0 : o) + part * 256 + c * 16, o >= 0);
                  }
                  cp_async_commit();
                  cp_async_wait<0>();
                } else {
                  uint32_t word = 0;
                  if (off >= 0) word = *reinterpret_cast<const uint32_t*>((values ? p.cache.vs : p.cache.ks) + soff + 4 * part);
                  const int c = lane & 7, sub = lane >> 3;
                  for (int k = 0; k < (kRows + 3) / 4; ++k) {
                    const int row = 4 * k + sub;
                    const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row);
                    const uint32_t sw = __shfl_sync(0xFFFFFFFFu, word, row);
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (row < rows && 2 * c < pieces) {
                      if (o >= 0) x = *reinterpret_cast<const uint4*>(from + o + part * 128 + c * 16);
                      convert(x, o >= 0 ? __uint_as_float(((sw >> (8 * (c >> 1))) & 0xFFu) << 23) : 0.f, row0 + row, c);
                    }
                  }
                }
                __syncwarp();
                if (partly) look_through(dst, pieces, row0, row0 + rows, 2, n);
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
              if (lane == 0) arrive(ctl->full[seq % kSlots]);
            }
            if (ok && partly) note();
          }
        }
        if (!ok) break;
        ++q_n;
        __syncwarp();
        if (lane == 0) arrive(ctl->seg_empty[seg_n & 1]);
        ++seg_n;
      }
      cp_async_wait<0>();
    }
  }

  // ---- rows that see nothing, and (a shared prefix) rows of no group
  if (warp < 8) {
    const int64_t E = a.header->entries;
    const int Hq = p.Hk * G;
    for (int64_t e = blockIdx.x; e < E; e += gridDim.x) {
      const Entry x = a.entries[e];
      if (x.units > 0) continue;
      const int n = min(x.rows - x.row0, kPair);
      for (int k = warp; k < n * p.Hk; k += 8) {
        const int r = x.row0 + k % n, i = r / G, h = (k / n) * G + r - i * G;
        const int64_t token = (int64_t)x.s0 + i;
        float z[16];
#pragma unroll
        for (int d = 0; d < 16; ++d) z[d] = 0.f;
        for (int d = lane * 16; d < D; d += 512) emit16(p, token, h, d, z, 0.f, 0.f);
      }
    }
    if (p.out == nullptr) {
      const int64_t first = p.B > 0 ? min((int64_t)max(__ldcg(p.cu), 0), p.T) : 0;
      const int64_t past = p.B > 0 ? min((int64_t)max(__ldcg(p.cu + p.B), 0), p.T) : 0;
      for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < p.T * Hq; k += (int64_t)gridDim.x * 256) {
        const int64_t t = k / Hq;
        if (t < first || t >= past) p.prior_lse[k] = -INFINITY;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    if (*abort_flag && elect_one()) drain<kFp8>(ctl, a.box > 0 ? loaders : 0, a.q_box != 0);
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
}

template <bool kWide, bool kFp8, bool kForm>
cudaError_t launch(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_q, const Args& a, cudaStream_t stream) {
  static PerContextOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(prompt_kernel<kWide, kFp8, kForm>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kFp8));
  });
  if (e != cudaSuccess) return e;
  return launch_k(prompt_kernel<kWide, kFp8, kForm>, dim3((unsigned)a.ctas), dim3(threads_of(kFp8)), smem_bytes(kFp8), stream, true, tm_k, tm_v, tm_q, a);
}

template <bool kFp8>
cudaError_t launch_any(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_q, const Args& a, cudaStream_t stream) {
  const bool form = a.p.form.cap2 > 0.f || a.p.form.slopes != nullptr || !(a.p.scale_log2 > 0.f);
  if (a.p.D > 128) return form ? launch<true, kFp8, true>(tm_k, tm_v, tm_q, a, stream) : launch<true, kFp8, false>(tm_k, tm_v, tm_q, a, stream);
  return form ? launch<false, kFp8, true>(tm_k, tm_v, tm_q, a, stream) : launch<false, kFp8, false>(tm_k, tm_v, tm_q, a, stream);
}

cudaError_t launch_bf16(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_q, const Args& a, cudaStream_t stream);
cudaError_t launch_fp8(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_q, const Args& a, cudaStream_t stream);

}  // namespace prompt
}  // namespace engram
