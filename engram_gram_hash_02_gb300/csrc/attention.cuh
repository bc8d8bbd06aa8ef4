// Attention of one new token per sequence over a paged cache of keys and values.
//
// For query head h of sequence b and the attended keys j (the last `window` of its `len` tokens, or all):
//   s_j = scale * q_h . k_j,   o_h = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse_h = log sum_j exp(s_j)
// in one pass with a running maximum (kept in units of log 2, so that every exponential is one ex2). Heads
// that share a key head are computed together, up to 16, so a key or value row is read from HBM once.
//
// What bounds it: those rows' bytes. Per 16 keys a warp computes two small products on the tensor cores
// (mma.sync m16n8k16, keys or values on the 16 rows, query heads on the 8 columns, fp32 accumulation):
//   S^T[keys, heads] = K Q^T      and      O^T[values, heads] += V^T P^T
// With one token per sequence the heads of a group are the only rows there are; the tensor pipe stays
// mostly idle, and operands in registers (no tensor memory to set up, drain and rescale through) keep a
// warp's chain from a landed copy to the next one short. (ncu: 11 to 17 % of that pipe's cycles in all of the shapes
// below, tcgen05 or not: it has nothing to win here.)
//
// Work is cut at keys, not at sequences: the tiles of all sequences and key heads form one row, sequence by
// sequence, and each CTA takes an equal run of it, so a batch of any mix of lengths keeps every SM busy to the
// end. A tile is a step (step_keys: 16 or 32 keys) of each of a CTA's four rings of shared-memory stages, filled by
// 16-byte cp.async (rows at the addresses their page gives; any page size, stride or tail). A ring belongs to one
// warp, or to two (team_warps) that a named barrier joins at every step; no barrier joins the rings until a
// sequence's run ends. There the four partial results are joined in shared memory. A run that is cut between CTAs is written to the workspace as
// (unnormalised o, maximum, sum); the last CTA to arrive joins the parts in order of their keys, so results
// do not depend on timing.
//
// FP8 rows (codes, one power-of-two scale per 32 values) are converted to f16 in registers (exact). A key
// block's scale multiplies that block's fp32 partial product. The value scales join the weights before those
// are rounded: with 2^e_j the largest scale of value row j's blocks that are not zero (2^-64 at least), the
// running maximum is that of s_j + e_j, the weights w_j = 2^(s_j + e_j - maximum + 15) fill f16's range, and a
// block's own scale enters as f = 2^(scale - e_j), a half that is exact down to 2^-24; the sum takes the weights
// times 2^-e_j. So no spread of the rows' sizes overflows, and what is lost is, per block: f16(f16(w_j) f) is off by
// 2^-11 of itself or, below 2^-14, by 2^-24; that is 2^-39 max_i(p_i 2^e_i) per unit of a code (p the normalised
// weights; the largest is taken over all blocks, so a block that is small in every row has less of its own). Blocks
// whose scale is 2^-24 below their row's largest, or below 2^-88, count as zero, and so do weights 2^-141 below the
// largest s_j + e_j in the sum (fp32; rows' scales that far apart).
//
// Measured on one GB300 (share of the 6.78 TB/s of a plain copy), heads of 128, 8 query heads per key head unless
// said: one sequence of 131072 tokens, 4 key heads, bf16, 49 us, 5.5 TB/s (0.81): 3 us until the first rows are
// there, then 7.3 TB/s, 5 us for the slowest SM and the join. 64 sequences of up to 8192 tokens, 2 key heads of 256,
// bf16, 88 us, 6.1 TB/s (0.90). 256 sequences of up to 4096 tokens, 8 key heads with 4 query heads each, FP8, 173 us,
// 6.4 TB/s (0.95): 710 instructions per 32 keys of 8448 bytes and twelve warps per SM to issue them. 48 windows of
// 1024 tokens, 16 heads of 64, bf16, 37.3 us, 5.2 TB/s (0.77): 1.7 runs per CTA. One sequence of 777 tokens 6.1 us:
// 1.2 us for lengths and page, 1 us for the rows, 0.5 us of computing, 2 us to join 13 parts.
//
// Roundings below 32 bits: with bf16 rows P is fed as the sum of two bf16 (hi + lo: 2^-16 at most); with
// FP8 rows as f16 (2^-11, an eighth of the output's own rounding). bf16 queries enter as they are; fp32
// queries as two bf16 or two f16; for f16 each query row is first scaled by a power of two (its largest
// value below 2^14). Scores, maxima, sums and o are fp32.
#pragma once

#include <atomic>

#include "attn.cuh"

namespace engram {
namespace attn {

constexpr int kRings = 4;                             // of a CTA: its tile is a step of each
constexpr int kGroup = 16;                            // parts of a cut run that one CTA joins
// A run's fixed cost (its queries, the join of its warps), in tiles, when work is divided. One constant for every
// kernel, fitted on three shapes with 16 and more tiles per run (at an earlier state of the kernels): with 2 (0), 64
// sequences of up to 8192 tokens, 2 key heads of 256, take 88 us (92), 256 of up to 4096 over FP8 189 (206), 48 windows
// of 1024, 16 heads of 64, 38.7 (42.6). Runs of one or two tiles pay more than it says.
constexpr int kRunCost = 2;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes to shared memory, or 16 zero bytes (nothing is read then)
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// two 16 x 16 matrices of bytes (row addresses from lanes 0..15 and 16..31), transposed: registers 0 and 1 hold
// columns lane / 4 and lane / 4 + 8 of the first, rows 4 (lane % 4) .. + 3; registers 2 and 3 of the second
__device__ __forceinline__ void ldsm8t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// the first of the two only
__device__ __forceinline__ void ldsm8t_one(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x1.trans.shared.b8 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
  r[2] = r[3] = 0;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool kHalf>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (kHalf)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// releases what the CTA wrote before its last barrier, and acquires what other arrivals released
__device__ __forceinline__ uint32_t atom_add_acq_rel(uint32_t* p, uint32_t v) {
  uint32_t r;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(r) : "l"(p), "r"(v) : "memory");
  return r;
}
// exp2(x - m) for m = max(x, ...): a maximum of -inf (nothing attended yet) gives 0
__device__ __forceinline__ float ex2_rel(float x, float m) { return ex2(x - (m == -INFINITY ? 0.f : m)); }

// How a kernel for heads of up to dp (64, 128 or 256) and `tiles` tiles of 8 query heads runs.
// Two tiles of heads of 256 do not fit a warp's registers: two warps then share a ring, a tile each.
constexpr int team_warps(int dp, int tiles) { return dp == 256 && tiles == 2 ? 2 : 1; }
// FP8 steps of 32 keys (the fixed part of a step is a third of its instructions), 16 where a ring of 32 would leave
// room for four warps only: 64 sequences of up to 4096 tokens, 8 heads of 256 per key head, 36.5 us (40.6 with 32).
constexpr int step_keys(bool fp8, int dp, int tiles) { return fp8 && !(dp == 256 && tiles == 1) ? 32 : 16; }
// CTAs per SM and stages per ring: as many warps as registers and shared memory allow, where instructions count
// (FP8 in one tile: 256 sequences of heads of 128 take 173 us with three CTAs of two stages, 183 with two of three;
// 64 of heads of 64 take 35.6 us with four of two, 37.2 with three of four), else three stages, which keep more
// bytes in flight (bf16: one sequence of 131072 takes 49.3 us, 51.1 with three CTAs of two stages). All measured with
// bf16 queries. Kernels for fp32 queries, which a decode step runs, take the same bounds; over FP8 those for one tile
// of heads of 128 and of 64 spill 64 and 32 bytes, and a step of 256 sequences takes 198 us (its attention with bf16
// queries 175).
constexpr int resident_ctas(bool fp8, int dp, int tiles) {
  return tiles == 2 ? (dp == 256 ? 1 : 2) : (dp == 64 ? 3 : dp == 128 ? 2 : 1) + (fp8 ? 1 : 0);
}
constexpr int ring_stages(bool fp8, int dp, int tiles) { return fp8 && tiles == 1 && dp <= 128 ? 2 : 3; }

template <int DP_, bool kFp8_, int kTiles_, bool kSplit_, bool kForm_>
struct Cfg {
  static constexpr int DP = DP_;                      // head_dim rounded up to 64, 128 or 256
  static constexpr bool kFp8 = kFp8_;
  static constexpr int kTiles = kTiles_;              // tiles of 8 query heads per CTA
  static constexpr int kTeam = team_warps(DP, kTiles);// warps that share a ring
  static constexpr int NQ = kTiles / kTeam;           // tiles per warp
  static constexpr int kHeads = 8 * kTiles;
  static constexpr int kWarps = kRings * kTeam;
  static constexpr int kThreads = kWarps * 32;
  static constexpr bool kSplit = kSplit_;             // fp32 queries: high and low parts
  static constexpr bool kForm = kForm_;               // scores with a form, or a part of the keys attended before
  static constexpr int kStep = step_keys(kFp8, DP, kTiles);   // keys per ring and step
  static constexpr int kTile = kRings * kStep;
  static constexpr int kRowB = kFp8 ? DP : 2 * DP;
  static constexpr int kWords = (DP + 127) / 128;     // scale words per row
  static constexpr int kStageB = 2 * kStep * kRowB + (kFp8 ? 2 * kStep * kWords * 4 : 0);
  static constexpr int kCtas = resident_ctas(kFp8, DP, kTiles);   // per SM
  static constexpr int kStages = ring_stages(kFp8, DP, kTiles);
  static constexpr int kRingB = kRings * kStages * kStageB;
  static constexpr int kQPitch = DP + 8;              // 16-bit values
  static constexpr int kQB = kHeads * kQPitch * 2;    // per part (high, low)
  static constexpr int kMetaB = kRings * kStages * 32;
  static constexpr int kSmall = 1024;                 // maxima, sums, query scales, scan words
  // FP8, per ring and key of a step: key block scales, e and 2^-e, and (two warps per ring) value block scales
  static constexpr int kScaleRow = 4 * kWords + 2 + (kTeam == 2 ? 2 * kWords : 0);
  static constexpr int kScalesB = kFp8 ? kRings * kStep * kScaleRow * 4 : 0;
  static constexpr int kAlign = 512;                  // a row's XORed bits are zero in its stage's address
  static constexpr int kSmemB = kAlign + kRingB + kQB * (kSplit ? 2 : 1) + kMetaB + kSmall + kScalesB;
  static constexpr bool kQRegs = DP / 16 * 2 * NQ * (kSplit ? 2 : 1) <= 32;
  static_assert(kHeads * DP * 4 <= kStageB, "a ring's result is joined in its own last stage");
  static_assert(kStageB % (kRowB < kAlign ? kRowB : kAlign) == 0, "stages keep the rows' alignment");
};

// Rows lie in a stage one after another; 16-byte chunk c of row r is at place c ^ key(r), so that eight rows
// at one chunk fall into eight different bank groups. key(r) as a byte offset:
template <int kRowB>
__host__ __device__ constexpr uint32_t swz(int r) {
  return (uint32_t)(kRowB >= 128 ? (r & 7) << 4 : ((r >> 1) & 3) << 4);
}

// what a warp knows of one step when it consumes it
struct Meta {
  uint32_t mask;               // keys of the step that are attended
  uint32_t ends;               // bit 0: first tile of its run, bit 1: last
  int32_t seq, hc, run0, tiles;// sequence, head * chunks + chunk, place of the run's first tile and its tiles
  int32_t back, pad;           // kForm: the step's first key is `back` tokens before the sequence's last
};

__device__ __forceinline__ int clamp_len(int len, int cap) { return len < 0 ? 0 : len > cap ? cap : len; }
__device__ __forceinline__ int attended(int len, int window) { return window > 0 && len > window ? window : len; }

// log2(l 2^m), l a positive float: l's exponent joins m before the logarithm, as the two may be large and of opposite
// sign (FP8). -inf for l = 0; a NaN or an infinite l comes back as it is.
__device__ __forceinline__ float log2_of_sum(float m, float l) {
  const uint32_t b = __float_as_uint(l);
  const float y = (m + (float)((int)(b >> 23) - 127)) + log2f(__uint_as_float((b & 0x7FFFFFu) | 0x3F800000u));
  return l == 0.f ? -INFINITY : l - l == 0.f ? y : l;
}

// A head's attended values x (four from value d on) over its own keys, whose exponentials sum to 2^own, joined with
// those over the keys that were attended before (prior_o, prior_lse)
__device__ __forceinline__ void emit_joined(const AttnParams& p, int seq, int head, int d, const float (&x)[4], float own) {
  const int64_t row = (int64_t)seq * (p.Hk * p.G) + head;
  const float before = __ldcg(p.prior_lse + row);
  // (nothing attended before: prior_o holds nothing)
  const float4 y = before == -INFINITY ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldcg(reinterpret_cast<const float4*>(p.prior_o + row * p.D + d));
  const float m = fmaxf(own, before);
  const float a = ex2_rel(own, m), b = ex2_rel(before, m), sum = a + b;
  const float fa = sum == 0.f ? 0.f : a / sum, fb = sum == 0.f ? 0.f : b / sum;
  uint2 w;
  w.x = pack_bf16(x[0] * fa + y.x * fb, x[1] * fa + y.y * fb);
  w.y = pack_bf16(x[2] * fa + y.z * fb, x[3] * fa + y.w * fb);
  *reinterpret_cast<uint2*>(p.out + (int64_t)seq * p.out_ts + (int64_t)head * p.out_hs + d) = w;
  if (d == 0 && p.lse != nullptr) p.lse[row] = sum == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(sum));
}

template <typename C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas) attention_kernel(const AttnParams p) {
  constexpr int DP = C::DP, NQ = C::NQ, kStages = C::kStages, kStep = C::kStep, kRowB = C::kRowB;
  constexpr int kThreads = C::kThreads, kWarps = C::kWarps, kTeam = C::kTeam, kHeads = C::kHeads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & (C::kAlign - 1));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, j = lane & 3;             // fragment row and column pair
  const int my_ring = warp / kTeam, rank = warp % kTeam;
  uint8_t* ring = smem + my_ring * kStages * C::kStageB;
  uint8_t* qs = smem + C::kRingB;
  Meta* meta = reinterpret_cast<Meta*>(qs + C::kQB * (C::kSplit ? 2 : 1)) + my_ring * kStages;
  float* small = reinterpret_cast<float*>(qs + C::kQB * (C::kSplit ? 2 : 1) + C::kMetaB);
  float* sm_m = small;                               // [ring][16] maxima (log2 units)
  float* sm_l = small + 64;                          // [ring][16] sums
  float* sm_c = small + 128;                         // [16] softmax scale of each query row, log2 units
  int* sm_i = reinterpret_cast<int*>(small + 160);   // scan and broadcast words
  float* key_scales = small + C::kSmall / 4 + my_ring * kStep * C::kScaleRow;   // (FP8) [key][4 * kWords], then [key][2]
  float* value_scales = key_scales + kStep * 4 * C::kWords;
  uint32_t* own_factors = reinterpret_cast<uint32_t*>(value_scales + kStep * 2);   // (two warps per ring)
  // the warps of a ring: what each has copied, read or written so far is done
  auto sync_ring = [&] {
    if (kTeam == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + my_ring), "n"(32 * kTeam) : "memory");
  };
  const int heads = p.Hk * p.chunks;

  if (!p.lens_ready) pdl_wait();

  // ---- this CTA's share --------------------------------------------------------------------
  // A run (a sequence's tiles for one key head and group of query heads) takes kRunCost + tiles places in a
  // row of all runs; CTA i takes the tiles at places [i * per_cta, (i + 1) * per_cta).
  auto tiles_of = [&](int raw) { return (attended(clamp_len(raw, p.cap), p.window) + C::kTile - 1) / C::kTile; };
  int total, place0, place1, per_cta;
  int seq = 0, hc = 0, tile = 0, run0 = 0;            // the first tile of the share, and its run's first place
  auto divide = [&] {
    per_cta = max((total + (int)gridDim.x - 1) / (int)gridDim.x, 1);
    place0 = min(total, (int)blockIdx.x * per_cta);
    place1 = min(total, place0 + per_cta);
  };
  auto locate = [&](int b, int at, int tiles) {       // place0 lies in sequence b, whose places start at `at`
    const int run = (place0 - at) / (tiles + kRunCost);
    seq = b;
    hc = run;
    run0 = at + run * (tiles + kRunCost) + kRunCost;
    tile = max(place0 - run0, 0);
  };
  auto places_of = [&](int tiles) { return tiles > 0 ? (tiles + kRunCost) * heads : 0; };
  auto read_len = [&](int b) {
    const int raw = __ldcg(p.lens + b);
    if (blockIdx.x == 0 && (raw < 0 || raw > p.cap) && p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_SEQ_LEN);
    return raw;
  };
  // Few sequences: every warp for itself, no barrier before its first copy (one sequence of 777 tokens:
  // 6.05 us, 6.29 by the CTA's sum below, which takes any batch).
  if (p.B <= 32) {
    const int tiles = lane < p.B ? tiles_of(read_len(lane)) : 0;
    int scan = places_of(tiles);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, scan, o);
      if (lane >= o) scan += y;
    }
    total = __shfl_sync(0xFFFFFFFFu, scan, 31);
    divide();
    const int b = __ffs(__ballot_sync(0xFFFFFFFFu, scan > place0)) - 1;   // none past the end
    if (b >= 0) locate(b, __shfl_sync(0xFFFFFFFFu, scan - places_of(tiles), b), __shfl_sync(0xFFFFFFFFu, tiles, b));
  } else {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = tid * per, b1 = min(p.B, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; ++b) mine += places_of(tiles_of(read_len(b)));
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, scan, o);
      if (lane >= o) scan += y;
    }
    if (lane == 31) sm_i[warp] = scan;
    __syncthreads();
    total = 0;
    int before = scan - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm_i[w];
      total += sm_i[w];
    }
    divide();
    if (place0 < place1 && place0 >= before && place0 < before + mine) {
      int at = before;
      for (int b = b0; b < b1; ++b) {
        const int tiles = tiles_of(__ldcg(p.lens + b));
        if (place0 < at + places_of(tiles)) {
          locate(b, at, tiles);
          sm_i[8] = seq;
          sm_i[9] = hc;
          sm_i[10] = tile;
          sm_i[11] = run0;
          break;
        }
        at += places_of(tiles);
      }
    }
    __syncthreads();
    seq = sm_i[8];
    hc = sm_i[9];
    tile = sm_i[10];
    run0 = sm_i[11];
  }
  if (p.lens_ready) pdl_wait();

  // ---- the producer: one tile after another ------------------------------------------------------
  int first = 0, end = 0, tiles = 0;
  int64_t head_off = 0, shead_off = 0;
  auto enter_head = [&] {
    const int head = p.chunks == 1 ? hc : hc / p.chunks;
    head_off = head * p.cache.head_b;
    if (C::kFp8) shead_off = head * p.cache.shead_b;
  };
  auto enter = [&] {                                  // seq is new
    const int len = clamp_len(__ldcg(p.lens + seq), p.cap);
    const int n = attended(len, p.window);
    first = len - n;
    end = len;
    tiles = (n + C::kTile - 1) / C::kTile;
  };
  auto advance = [&] {
    if (++tile < tiles) return;
    run0 += tiles + kRunCost;                         // the next run's first tile
    tile = 0;
    if (++hc == heads) {
      hc = 0;
      do {
        if (++seq >= p.B) return;                     // past the last place: never fetched
        enter();
      } while (tiles == 0);
    }
    enter_head();
  };
  auto more = [&] { return run0 + tile < place1; };
  // the page of this lane's row, requested one step before its copies
  int page = -1, at = 0;
  bool inside = false;
  auto request = [&] {
    const int pos = first + tile * C::kTile + my_ring * kStep + (lane & (kStep - 1));
    inside = pos < end;
    page = -1;
    if (inside) {
      const int n = (int)fast_div((uint32_t)pos, p.cache.div_page);
      at = pos - n * p.cache.page_size;
      page = p.table[(int64_t)seq * p.table_stride + n];
    }
  };
  // a lane copies chunk c of rows sub, sub + kRows, ... (the warps of a ring take turns at these passes)
  constexpr int kChunks = kRowB / 16, kRows = 32 / kChunks;
  const int c = lane & (kChunks - 1), sub = lane / kChunks;
  const bool in_row = c * 16 < (C::kFp8 ? p.D : 2 * p.D);
  const uint32_t lane_dst = (uint32_t)(sub * kRowB) + ((uint32_t)(c << 4) ^ swz<kRowB>(sub));
  const uint32_t ring_u = smem_u32(ring);
  auto my_pass = [&](int r0) { return kTeam == 1 || (r0 / kRows) % kTeam == rank; };
  auto issue = [&](int stage) {
    const bool live = inside && page >= 0 && page < p.cache.num_pages;
    if (inside && !live && p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_PAGE);
    constexpr uint32_t kAll = kStep == 32 ? 0xFFFFFFFFu : 0xFFFFu;
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, live) & kAll;
    if (lane == 0 && rank == 0) {
      Meta m;
      m.mask = mask; m.ends = (tile == 0 ? 1u : 0u) | (tile + 1 == tiles ? 2u : 0u);
      m.seq = seq; m.hc = hc; m.run0 = run0; m.tiles = tiles;
      if (C::kForm) m.back = end - 1 - (first + tile * C::kTile + my_ring * kStep);
      meta[stage] = m;
    }
    if (mask == 0) return;                            // no keys for this warp: the stage is not read
    const uint32_t dst = ring_u + stage * C::kStageB;
    const uint32_t to = dst + lane_dst;
    const int64_t off = live ? ((int64_t)((uint64_t)(uint32_t)page * p.cache.page_u + (uint64_t)(uint32_t)at * p.cache.tok_u) << 4) + head_off : 0;
    // All rows attended and in one page: equal steps from the first one, without a shuffle for each row (one
    // sequence of 131072 tokens: 48.4 us, 50.1 without this; 256 FP8 sequences: 170.9, 173.1).
    const int at0 = __shfl_sync(0xFFFFFFFFu, at, 0);
    if (mask == kAll && at0 + kStep <= p.cache.page_size) {
      const uint8_t* kp = p.cache.k + (__shfl_sync(0xFFFFFFFFu, off, 0) + sub * p.cache.tok_b + c * 16);
      const uint8_t* vp = kp + (p.cache.v - p.cache.k);
      if (in_row) {
        const int64_t step = kRows * p.cache.tok_b;
#pragma unroll
        for (int r0 = 0; r0 < kStep; r0 += kRows) {
          if (my_pass(r0)) {
            cp_async16((to ^ swz<kRowB>(r0)) + r0 * kRowB, kp);
            cp_async16((to ^ swz<kRowB>(r0)) + (kStep + r0) * kRowB, vp);
          }
          kp += step;
          vp += step;
        }
      }
    } else {
#pragma unroll
      for (int r0 = 0; r0 < kStep; r0 += kRows) {
        const int r = r0 + sub;
        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r) + c * 16;
        const bool row_live = (mask >> r) & 1u;
        if (in_row && my_pass(r0)) {
          cp_async16_or_zero((to ^ swz<kRowB>(r0)) + r0 * kRowB, p.cache.k + o, row_live);
          cp_async16_or_zero((to ^ swz<kRowB>(r0)) + (kStep + r0) * kRowB, p.cache.v + o, row_live);
        }
      }
    }
    if (C::kFp8 && lane < kStep) {
      const int64_t so = live ? ((int64_t)((uint64_t)(uint32_t)page * p.cache.spage_u + (uint64_t)(uint32_t)at * p.cache.stok_u) << 2) + shead_off : 0;
      const uint32_t sd = dst + 2 * kStep * kRowB + lane * C::kWords * 4;
#pragma unroll
      for (int w = 0; w < C::kWords; ++w) {
        if (rank == 0) cp_async4_or_zero(sd + 4 * w, p.cache.ks + so + 4 * w, live);
        if (rank == kTeam - 1) cp_async4_or_zero(sd + kStep * C::kWords * 4 + 4 * w, p.cache.vs + so + 4 * w, live);
      }
    }
  };
  // rows narrower than DP: the products run over their pad, which is zero in every stage
  auto clear_pad = [&](int stage) {
    for (int r = sub + rank * kRows; r < 2 * kStep; r += kTeam * kRows)
      if (!in_row) *reinterpret_cast<uint4*>(ring + stage * C::kStageB + r * kRowB + ((uint32_t)(c << 4) ^ swz<kRowB>(r))) = make_uint4(0, 0, 0, 0);
  };
  const bool padded = p.D < DP;
  const uint32_t scale_bytes = p.D % 128 == 0 ? 0xFFFFFFFFu : (1u << (8 * (p.D % 128 / 32))) - 1u;   // of the last word

  int ahead = 0;                                      // steps requested so far
  if (place0 < place1) {
    if (padded) {
      for (int s = 0; s < kStages; ++s) clear_pad(s);
      __syncwarp();
    }
    enter();
    enter_head();
    if (more()) request();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      if (more()) {
        issue(s);
        ++ahead;
        advance();
        if (more()) request();
      }
      cp_async_commit();
    }
  }

  // ---- the consumer ----------------------------------------------------------------------------
  float o[DP / 16][NQ][4];
  float m_run[NQ][2], l_run[NQ][2];
  uint32_t qf[C::kQRegs ? NQ : 1][C::kQRegs ? DP / 16 : 1][C::kSplit ? 4 : 2];
  int rows = 0;                                       // query heads of this run
  // Scores with a form, in units of log 2
  float slope[C::kForm ? NQ : 1][2];                  // of this lane's two heads per tile
  auto form = [&](float x, float slope, int back) {
    if (p.form.cap2 > 0.f) x = capped(x, p.form.cap2, p.form.cap_inv);
    return p.form.slopes != nullptr ? fmaf(-slope, (float)back, x) : x;
  };

  auto q_frag = [&](int nq, int ks, uint32_t (&b)[4]) {
    const uint8_t* row = qs + (((rank * NQ + nq) * 8 + g) * C::kQPitch + ks * 16) * 2;
    if (C::kFp8) {                                    // the pairs of values a lane's four codes hold
      const uint2 hi = *reinterpret_cast<const uint2*>(row + 8 * j);
      b[0] = hi.x; b[1] = hi.y;
      if (C::kSplit) {
        const uint2 lo = *reinterpret_cast<const uint2*>(row + C::kQB + 8 * j);
        b[2] = lo.x; b[3] = lo.y;
      }
    } else {
      b[0] = *reinterpret_cast<const uint32_t*>(row + 4 * j);
      b[1] = *reinterpret_cast<const uint32_t*>(row + 4 * j + 16);
      if (C::kSplit) {
        b[2] = *reinterpret_cast<const uint32_t*>(row + C::kQB + 4 * j);
        b[3] = *reinterpret_cast<const uint32_t*>(row + C::kQB + 4 * j + 16);
      }
    }
  };

  // A run's query rows: two or four per warp, DP / 32 consecutive values per lane. They are requested
  // while the run before is still computed.
  constexpr int kQRows = kHeads / kWarps, kQVals = DP / 32;
  constexpr int kQWords = C::kSplit ? kQVals : (kQVals + 1) / 2;
  uint32_t q_raw[kQRows][kQWords];
  auto chunk_of = [&](int hc) { return p.chunks == 1 ? 0 : hc % p.chunks; };
  auto first_head = [&](int hc) { return (p.chunks == 1 ? hc : hc / p.chunks) * p.G + chunk_of(hc) * kHeads; };
  auto heads_of = [&](int hc) { return min(kHeads, p.G - chunk_of(hc) * kHeads); };
  auto request_q = [&](int seq, int hc) {
    const int h0 = first_head(hc), have = heads_of(hc);
#pragma unroll
    for (int k = 0; k < kQRows; ++k) {
      const int r = warp + k * kWarps;
#pragma unroll
      for (int e = 0; e < kQWords; ++e) q_raw[k][e] = 0;
      if (r < have && lane * kQVals < p.D) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.q.data) +
            ((int64_t)seq * p.q.ts + (int64_t)(h0 + r) * p.q.hs + lane * kQVals) * (C::kSplit ? 4 : 2));
#pragma unroll
        for (int e = 0; e < kQWords; e += 4) {
          if (kQWords >= 4) {
            const uint4 y = *reinterpret_cast<const uint4*>(src + e);
            q_raw[k][e] = y.x; q_raw[k][kQWords > 1 ? e + 1 : e] = y.y;
            q_raw[k][kQWords > 2 ? e + 2 : e] = y.z; q_raw[k][kQWords > 3 ? e + 3 : e] = y.w;
          } else if (kQWords == 2) {
            const uint2 y = *reinterpret_cast<const uint2*>(src);
            q_raw[k][0] = y.x; q_raw[k][kQWords > 1 ? 1 : 0] = y.y;
          } else {
            q_raw[k][0] = *src;
          }
        }
      }
    }
  };

  int stage = 0;
  for (int i = 0; i < ahead; ++i) {
    cp_async_wait<kStages - 2>();
    sync_ring();
    const uint32_t mask = meta[stage].mask, ends = meta[stage].ends;
    const int back = C::kForm ? meta[stage].back : 0;

    if (i == 0 || (ends & 1u)) {
      // a new run: its query rows to shared memory (16-bit, zero rows and columns as padding)
      if (i == 0) request_q(meta[stage].seq, meta[stage].hc);
      rows = heads_of(meta[stage].hc);
#pragma unroll
      for (int k = 0; k < kQRows; ++k) {
        const int r = warp + k * kWarps;
        float x[kQVals];
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < kQVals; ++e) {
          const uint32_t w = q_raw[k][C::kSplit ? e : e / 2];
          x[e] = C::kSplit ? __uint_as_float(w) : (e & 1) ? bf16_hi(w) : bf16_lo(w);
          amax = fmaxf(amax, fabsf(x[e]));
        }
        int up = 0;                                   // x * 2^up in f16
        if (C::kFp8) {
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, s));
          const int field = (int)(__float_as_uint(amax) >> 23);
          if (amax > 0.f && field < 255) up = 140 - max(field, 1);   // amax * 2^up in [2^13, 2^14)
          if (lane == 0) sm_c[r] = ldexpf(p.scale_log2, -up);
        }
        uint32_t* dst = reinterpret_cast<uint32_t*>(qs + (r * C::kQPitch + lane * kQVals) * 2);
#pragma unroll
        for (int e = 0; e < kQVals; e += 2) {
          float hi[2], lo[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float y = C::kFp8 ? ldexpf(x[e + z], up) : x[e + z];
            hi[z] = C::kFp8 ? __half2float(__float2half_rn(y)) : __bfloat162float(__float2bfloat16_rn(y));
            lo[z] = y - hi[z];
            if (lo[z] != lo[z]) lo[z] = 0.f;          // inf - inf: the high part says it all
          }
          dst[e / 2] = C::kFp8 ? pack_f16(hi[0], hi[1]) : pack_bf16(hi[0], hi[1]);
          if (C::kSplit) dst[e / 2 + C::kQB / 4] = C::kFp8 ? pack_f16(lo[0], lo[1]) : pack_bf16(lo[0], lo[1]);
        }
      }
      __syncthreads();
      if (C::kQRegs) {
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks) {
            uint32_t b[4];
            q_frag(nq, ks, b);
#pragma unroll
            for (int e = 0; e < (C::kSplit ? 4 : 2); ++e) qf[nq][ks][e] = b[e];
          }
      }
      if (C::kForm && p.form.slopes != nullptr) {
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = (rank * NQ + nq) * 8 + 2 * j + e;
            slope[C::kForm ? nq : 0][e] = h < rows ? p.form.slopes[first_head(meta[stage].hc) + h] * 1.44269504f : 0.f;
          }
      }
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
#pragma unroll
        for (int e = 0; e < 2; ++e) { m_run[nq][e] = -INFINITY; l_run[nq][e] = 0.f; }
#pragma unroll
        for (int mt = 0; mt < DP / 16; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][nq][e] = 0.f;
      }
    }

    // the stage consumed in the last step is refilled while this one is computed
    if (more()) {
      issue(stage == 0 ? kStages - 1 : stage - 1);
      ++ahead;
      advance();
      if (more()) request();
    }
    cp_async_commit();
    if ((ends & 2u) && i + 1 < ahead) {
      __syncwarp();                                   // lane 0 may have just written the next step's
      const Meta* next = meta + (stage + 1 == kStages ? 0 : stage + 1);
      request_q(next->seq, next->hc);
    }

    if (mask != 0) {
      // This lane's row and chunk of every ldmatrix. bf16, keys and values: rows 0..7 and 8..15, chunks 2x and
      // 2x + 1. FP8 keys: the key of row r of the product is kr(r), such that the transposed weights have the
      // keys in the order in which a register of the transposed value codes holds them.
      auto kr = [](int r) { return C::kFp8 ? ((r & 6) << 1) | (r & 1) | ((r >> 3) << 1) : r; };
      constexpr int kHi = C::kFp8 ? 4 : 3, kRow8 = C::kFp8 ? 3 : 4;
      const int lrow = kr(((lane >> kRow8) & 1) * 8 + (lane & 7));
      const uint32_t tiles_u = (ring_u + stage * C::kStageB + lrow * kRowB) + ((((lane >> kHi) & 1) << 4) ^ swz<kRowB>(lrow));
      constexpr int kRowMask = kStep - 1;             // FP8 values: a lane addresses row lane & kRowMask
      const uint32_t codes_u = ring_u + stage * C::kStageB + (kStep + (lane & kRowMask)) * kRowB + swz<kRowB>(lane & kRowMask);
      const int k0 = kr(g), k8 = kr(g + 8);           // keys of this lane's fragment rows
      constexpr int KT = kStep / 16;
      uint32_t pb[KT][NQ][C::kFp8 ? 2 : 4];            // P as the second product's operand (bf16: high, low)
      float t[KT][NQ][4];
      uint32_t* kw = reinterpret_cast<uint32_t*>(ring + stage * C::kStageB + 2 * kStep * kRowB);
      const uint32_t* vw = kw + kStep * C::kWords;
      uint32_t* factors = kTeam == 1 ? kw : own_factors;

      // FP8: the scales of this lane's key for all lanes. Key blocks' scales as floats; e = the largest value scale
      // and 2^-e; value blocks' scales relative to e as halves ([key][2 * kWords] words: in the place of the step's
      // scale words where no other warp reads them, else apart from them). A block that holds an infinity (bytes
      // 254 and 255) has an infinite factor and no part in e: it spoils its own 32 values only. A block of zeros (byte
      // 127, however small the values around it) has no part in e either: with one, the other blocks' weights and
      // factors would be in units of a contribution that is not there. Byte 127 is rare else (values up to 224 to
      // 448), so codes are looked at only in steps that have one (256 sequences of heads of 128 take 173 us, 185 if
      // every scale is 1).
      if (C::kFp8) {
        const int own = lane & (kStep - 1);
        const bool writes = kTeam == 1 || own / (kStep / kTeam) == rank;   // two warps spread half of the keys each
        int top = 63;                                 // e + 127, at least -64 + 127: the sum takes 2^-e
        uint32_t kb[C::kWords], vb[C::kWords], f[2 * C::kWords], ones = 0;
#pragma unroll
        for (int w = 0; w < C::kWords; ++w) {
          const uint32_t used = w + 1 == C::kWords ? scale_bytes : 0xFFFFFFFFu;
          kb[w] = kw[own * C::kWords + w] & used;
          vb[w] = vw[own * C::kWords + w] & used;
          float y[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) y[z] = __uint_as_float(((kb[w] >> (8 * z)) & 0xFFu) << 23);
          if (writes) *reinterpret_cast<float4*>(key_scales + (own * C::kWords + w) * 4) = make_float4(y[0], y[1], y[2], y[3]);
          const uint32_t x = vb[w] ^ 0x7F7F7F7Fu;     // (a zero byte here: a byte 127 there)
          ones |= (x - 0x01010101u) & ~x & 0x80808080u;
        }
        if (__any_sync(0xFFFFFFFFu, ones != 0)) {
          const uint8_t* codes = ring + stage * C::kStageB + (kStep + own) * kRowB;
#pragma unroll
          for (int b = 0; b < DP / 32; ++b) {
            const uint32_t byte = 0xFFu << (8 * (b & 3));
            if ((vb[b / 4] & byte) == (0x7F7F7F7Fu & byte)) {
              const uint4 x = *reinterpret_cast<const uint4*>(codes + ((uint32_t)(b << 5) ^ swz<kRowB>(own)));
              const uint4 y = *reinterpret_cast<const uint4*>(codes + ((uint32_t)(b << 5 | 16) ^ swz<kRowB>(own)));
              if (((x.x | x.y | x.z | x.w | y.x | y.y | y.z | y.w) & 0x7F7F7F7Fu) == 0) vb[b / 4] &= ~byte;
            }
          }
        }
#pragma unroll
        for (int b = 0; b < 4 * C::kWords; ++b) {
          const int by = (int)((vb[b / 4] >> (8 * (b & 3))) & 0xFFu);
          if (by < 254) top = max(top, by);
        }
        // e as a float: the integer behind 2^23
        if (writes)
          *reinterpret_cast<float2*>(value_scales + 2 * own) = make_float2(
              __uint_as_float(0x4B000000u + top) - 8388735.f, __uint_as_float((uint32_t)(254 - top) << 23));
#pragma unroll
        for (int x = 0; x < 2 * C::kWords; ++x) {
          float y[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int by = (int)((vb[x / 2] >> (16 * (x & 1) + 8 * z)) & 0xFFu);
            y[z] = __uint_as_float(by >= 254 ? 0x7F800000u : (uint32_t)max(127 + by - top, 0) << 23);
          }
          f[x] = pack_f16(y[0], y[1]);
        }
        if (kTeam == 1) __syncwarp();                 // every lane has read the scale words
#pragma unroll
        for (int x = 0; x < 2 * C::kWords; ++x)
          if (writes) factors[own * 2 * C::kWords + x] = f[x];
        sync_ring();
      }

      // S^T = K Q^T
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        if (C::kFp8) {
          float s0[4 * C::kWords], s1[4 * C::kWords];
#pragma unroll
          for (int w = 0; w < C::kWords; ++w) {
            *reinterpret_cast<float4*>(s0 + 4 * w) = *reinterpret_cast<const float4*>(key_scales + ((kt * 16 + k0) * C::kWords + w) * 4);
            *reinterpret_cast<float4*>(s1 + 4 * w) = *reinterpret_cast<const float4*>(key_scales + ((kt * 16 + k8) * C::kWords + w) * 4);
          }
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 4; ++e) t[kt][nq][e] = 0.f;
#pragma unroll
          for (int b = 0; b < DP / 32; ++b) {
            uint32_t a[4];                             // codes: keys of rows g, g + 8 (values 0..15), the same (16..31)
            ldsm4(a, (tiles_u ^ (b << 5)) + kt * 16 * kRowB);
            uint32_t f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_f16x2(a[e], f[2 * e], f[2 * e + 1]);
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
              float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t q4[4];
                if (C::kQRegs) {
#pragma unroll
                  for (int x = 0; x < (C::kSplit ? 4 : 2); ++x) q4[x] = qf[nq][2 * b + e][x];
                } else {
                  q_frag(nq, 2 * b + e, q4);
                }
                mma<true>(acc, f[4 * e], f[4 * e + 2], f[4 * e + 1], f[4 * e + 3], q4[0], q4[1]);
                if (C::kSplit) mma<true>(acc, f[4 * e], f[4 * e + 2], f[4 * e + 1], f[4 * e + 3], q4[2], q4[3]);
              }
              t[kt][nq][0] += acc[0] * s0[b];
              t[kt][nq][1] += acc[1] * s0[b];
              t[kt][nq][2] += acc[2] * s1[b];
              t[kt][nq][3] += acc[3] * s1[b];
            }
          }
        } else {
          float acc[NQ][2][4];                         // two chains: even and odd steps
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nq][0][e] = acc[nq][1][e] = 0.f;
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks) {
            uint32_t a[4];                             // keys 0..7 (values 0..7, 8..15), keys 8..15
            ldsm4(a, tiles_u ^ (ks << 5));
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
              uint32_t q4[4];
              if (C::kQRegs) {
#pragma unroll
                for (int x = 0; x < (C::kSplit ? 4 : 2); ++x) q4[x] = qf[nq][ks][x];
              } else {
                q_frag(nq, ks, q4);
              }
              mma<false>(acc[nq][ks & 1], a[0], a[2], a[1], a[3], q4[0], q4[1]);
              if (C::kSplit) mma<false>(acc[nq][ks & 1], a[0], a[2], a[1], a[3], q4[2], q4[3]);
            }
          }
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 4; ++e) t[kt][nq][e] = acc[nq][0][e] + acc[nq][1][e];
        }
      }

      // softmax over the step's keys, for each of this lane's two heads per tile
      bool moved = false;
      float alpha[NQ][2];                             // what o is multiplied by
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
        float mx[2] = {-INFINITY, -INFINITY};
        float un[KT][2];                              // FP8: 2^-e of this lane's two keys
        const float c0 = C::kFp8 ? sm_c[(rank * NQ + nq) * 8 + 2 * j] : p.scale_log2;
        const float c1 = C::kFp8 ? sm_c[(rank * NQ + nq) * 8 + 2 * j + 1] : p.scale_log2;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          float(&x)[4] = t[kt][nq];
          if (C::kFp8) {
            const float2 v0 = *reinterpret_cast<const float2*>(value_scales + 2 * (kt * 16 + k0));
            const float2 v1 = *reinterpret_cast<const float2*>(value_scales + 2 * (kt * 16 + k8));
            const float e0 = v0.x, e1 = v1.x;
            un[kt][0] = v0.y;
            un[kt][1] = v1.y;
            if (C::kForm) {
              const float s0 = slope[C::kForm ? nq : 0][0], s1 = slope[C::kForm ? nq : 0][1];
              x[0] = form(x[0] * c0, s0, back - (kt * 16 + k0)) + e0;
              x[1] = form(x[1] * c1, s1, back - (kt * 16 + k0)) + e0;
              x[2] = form(x[2] * c0, s0, back - (kt * 16 + k8)) + e1;
              x[3] = form(x[3] * c1, s1, back - (kt * 16 + k8)) + e1;
            } else {
              x[0] = x[0] * c0 + e0; x[1] = x[1] * c1 + e0; x[2] = x[2] * c0 + e1; x[3] = x[3] * c1 + e1;
            }
          } else {
            x[0] *= c0; x[1] *= c1; x[2] *= c0; x[3] *= c1;
            if (C::kForm) {
              const float s0 = slope[C::kForm ? nq : 0][0], s1 = slope[C::kForm ? nq : 0][1];
              x[0] = form(x[0], s0, back - (kt * 16 + k0));
              x[1] = form(x[1], s1, back - (kt * 16 + k0));
              x[2] = form(x[2], s0, back - (kt * 16 + k8));
              x[3] = form(x[3], s1, back - (kt * 16 + k8));
            }
          }
          if (mask != (kStep == 32 ? 0xFFFFFFFFu : 0xFFFFu)) {
            if (!((mask >> (kt * 16 + k0)) & 1u)) x[0] = x[1] = -INFINITY;
            if (!((mask >> (kt * 16 + k8)) & 1u)) x[2] = x[3] = -INFINITY;
          }
          mx[0] = fmaxf(mx[0], fmaxf(x[0], x[2]));
          mx[1] = fmaxf(mx[1], fmaxf(x[1], x[3]));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], s));
          // (FP8: weights up to 2^15, so the units of o and the sum are 2^(maximum - 15))
          const float m = fmaxf(m_run[nq][e], C::kFp8 ? mx[e] - 15.f : mx[e]);
          alpha[nq][e] = ex2_rel(m_run[nq][e], m);
          moved |= m != m_run[nq][e];
          m_run[nq][e] = m;
          const float base = m == -INFINITY ? 0.f : m;
          float sum = 0.f;
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            float(&x)[4] = t[kt][nq];
            x[e] = ex2(x[e] - base);
            x[e + 2] = ex2(x[e + 2] - base);
            if (C::kFp8)
              sum += x[e] * un[kt][0] + x[e + 2] * un[kt][1];
            else
              sum += x[e] + x[e + 2];
          }
          l_run[nq][e] = l_run[nq][e] * alpha[nq][e] + sum;
        }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const float(&x)[4] = t[kt][nq];
          if (C::kFp8) {
            pb[kt][nq][0] = transpose8(pack_f16(x[0], x[1]));
            pb[kt][nq][1] = transpose8(pack_f16(x[2], x[3]));
          } else {
            const uint32_t h0 = pack_bf16(x[0], x[1]), h1 = pack_bf16(x[2], x[3]);
            pb[kt][nq][0] = transpose8(h0);
            pb[kt][nq][1] = transpose8(h1);
            pb[kt][nq][C::kFp8 ? 0 : 2] = transpose8(pack_bf16(x[0] - bf16_lo(h0), x[1] - bf16_hi(h0)));
            pb[kt][nq][C::kFp8 ? 0 : 3] = transpose8(pack_bf16(x[2] - bf16_lo(h1), x[3] - bf16_hi(h1)));
          }
        }
      }

      // o in the new units
      if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
        for (int mt = 0; mt < DP / 16; ++mt)
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq) {
            o[mt][nq][0] *= alpha[nq][0];
            o[mt][nq][1] *= alpha[nq][1];
            o[mt][nq][2] *= alpha[nq][0];
            o[mt][nq][3] *= alpha[nq][1];
          }
      }

      // O^T += V^T P^T
      if (C::kFp8) {
        uint32_t sc[KT][4][2 * C::kWords];            // block scales of keys 4j .. 4j + 3
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int x = 0; x < 2 * C::kWords; ++x) sc[kt][k][x] = factors[(kt * 16 + 4 * j + k) * 2 * C::kWords + x];
#pragma unroll
        for (int b = 0; b < DP / 32; ++b) {
          uint32_t ps[KT][NQ][2];                     // the weights times the block's scales
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            const uint32_t y0 = __byte_perm(sc[kt][0][b / 2], sc[kt][1][b / 2], (b & 1) ? 0x7632 : 0x5410);
            const uint32_t y1 = __byte_perm(sc[kt][2][b / 2], sc[kt][3][b / 2], (b & 1) ? 0x7632 : 0x5410);
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
              const __half2 p0 = __hmul2(*reinterpret_cast<const __half2*>(&pb[kt][nq][0]), *reinterpret_cast<const __half2*>(&y0));
              const __half2 p1 = __hmul2(*reinterpret_cast<const __half2*>(&pb[kt][nq][1]), *reinterpret_cast<const __half2*>(&y1));
              ps[kt][nq][0] = *reinterpret_cast<const uint32_t*>(&p0);
              ps[kt][nq][1] = *reinterpret_cast<const uint32_t*>(&p1);
            }
          }
#pragma unroll
          for (int mt = 2 * b; mt < 2 * b + 2; ++mt) {
            uint32_t a[4];                            // codes of values g, g + 8: keys 4j .. 4j + 3 of 0..15, of 16..31
            if (KT == 2)
              ldsm8t(a, codes_u ^ (mt << 4));
            else
              ldsm8t_one(a, codes_u ^ (mt << 4));
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              uint32_t f[4];
              e4m3x4_to_f16x2(a[2 * kt], f[0], f[2]);
              e4m3x4_to_f16x2(a[(2 * kt + 1) & 3], f[1], f[3]);
#pragma unroll
              for (int nq = 0; nq < NQ; ++nq) mma<true>(o[mt][nq], f[0], f[1], f[2], f[3], ps[kt][nq][0], ps[kt][nq][1]);
            }
          }
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < DP / 16; ++mt) {
          uint32_t a[4];                               // values 0..7, 8..15 (keys 0..7), the same of keys 8..15
          ldsm4t(a, (tiles_u ^ (mt << 5)) + kStep * kRowB);
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq) {
            mma<false>(o[mt][nq], a[0], a[1], a[2], a[3], pb[0][nq][0], pb[0][nq][1]);
            mma<false>(o[mt][nq], a[0], a[1], a[2], a[3], pb[0][nq][C::kFp8 ? 0 : 2], pb[0][nq][C::kFp8 ? 1 : 3]);
          }
        }
      }
    }

    if ((ends & 2u) || i + 1 == ahead) {
      // ---- the run ends here, or this CTA's part of it: join the rings -----------------------
      const Meta me = meta[stage];
      sync_ring();                                   // the stage is read: it takes its warps' o
      float* mine_o = reinterpret_cast<float*>(ring + stage * C::kStageB) + rank * NQ * 8 * DP;
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float l = l_run[nq][e];
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, s);
          if (g == 0) {
            sm_m[my_ring * 16 + (rank * NQ + nq) * 8 + 2 * j + e] = m_run[nq][e];
            sm_l[my_ring * 16 + (rank * NQ + nq) * 8 + 2 * j + e] = l;
          }
        }
#pragma unroll
        for (int mt = 0; mt < DP / 16; ++mt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int q = nq * 8 + 2 * j + (e & 1);
            const int d = mt * 16 + g + 8 * (e >> 1);
            mine_o[q * DP + (d ^ (((q >> 1) & 3) << 3))] = o[mt][nq][e];
          }
        }
      }
      __syncthreads();

      const int c_first = me.run0 / per_cta, c_last = (me.run0 + me.tiles - 1) / per_cta;
      const bool whole = c_first == c_last;
      const int h0 = first_head(me.hc);
      const int q_heads = p.Hk * p.G;
      constexpr int kSlot = kHeads * (DP + 2);        // floats of a part: o, then (maximum, sum) per head
      // a CTA has at most two parts of cut runs: slot 1 for the one that starts in its share, slot 0 for the one before
      auto slot_of = [&](int cta) { return p.part + (int64_t)(2 * cta + (cta == c_first ? 1 : 0)) * kSlot; };
      auto emit = [&](int q, int d, const float (&x)[4], float m, float l) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (C::kForm && p.prior_lse != nullptr) {
          const float y[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
          emit_joined(p, me.seq, h0 + q, d, y, log2_of_sum(m, l));
          return;
        }
        uint2 w;
        w.x = pack_bf16(x[0] * inv, x[1] * inv);
        w.y = pack_bf16(x[2] * inv, x[3] * inv);
        *reinterpret_cast<uint2*>(p.out + (int64_t)me.seq * p.out_ts + (int64_t)(h0 + q) * p.out_hs + d) = w;
        if (d == 0 && p.lse != nullptr) {
          const float sum = log2_of_sum(m, l);
          p.lse[(int64_t)me.seq * q_heads + h0 + q] = l == 0.f ? -INFINITY : l - l == 0.f ? 0.6931471805599453f * sum : l;
        }
      };
      auto put = [&](float* part, int q, int d, const float (&x)[4], float m, float l) {
        __stcg(reinterpret_cast<float4*>(part + q * DP + d), make_float4(x[0], x[1], x[2], x[3]));
        if (d == 0) __stcg(reinterpret_cast<float2*>(part + kHeads * DP + 2 * q), make_float2(m, l));
      };
      for (int e = tid; e < rows * (DP / 4); e += kThreads) {
        const int q = e / (DP / 4), d = (e % (DP / 4)) * 4;
        if (d >= p.D) continue;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kRings; ++w) m = fmaxf(m, sm_m[w * 16 + q]);
        float l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kRings; ++w) {
          const float f = ex2_rel(sm_m[w * 16 + q], m);
          l += sm_l[w * 16 + q] * f;
          const float4 y = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(smem + (w * kStages + stage) * C::kStageB) + q * DP + (d ^ (((q >> 1) & 3) << 3)));
          x[0] += y.x * f; x[1] += y.y * f; x[2] += y.z * f; x[3] += y.w * f;
        }
        if (whole)
          emit(q, d, x, m, l);
        else
          put(slot_of(blockIdx.x), q, d, x, m, l);
      }
      if (!whole) {
        // The last CTA to arrive of each group of kGroup joins the group's parts into the group's first slot,
        // the last group to be joined joins the groups: 2 * sqrt(parts) reads in a row instead of all of them
        // through one SM (one sequence of 131072 tokens: 48.4 us, 55.3 in one level). A counter belongs to its
        // group by the group's first CTA; a run's first group may share that CTA with the end of another run,
        // so it has an array of its own.
        auto arrive_last = [&](uint32_t* counter, int parties) {
          __syncthreads();                            // every thread's part is written
          if (tid == 0) {
            const int last = atom_add_acq_rel(counter, 1u) == (uint32_t)(parties - 1);
            if (last) *counter = 0;                   // the next call finds it zero
            sm_i[12] = last;
          }
          __syncthreads();
          return sm_i[12] != 0;
        };
        auto join = [&](int from, int step, int parts, bool final) {
          for (int e0 = 0; e0 < rows * (DP / 4); e0 += kThreads) {
            const int e = e0 + tid;
            const int q = e / (DP / 4), d = (e % (DP / 4)) * 4;
            const bool mine = e < rows * (DP / 4) && d < p.D;
            float m = -INFINITY, l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
            if (mine) {
              constexpr int kBatch = C::kTiles == 2 ? 16 : 8;   // parts in flight per thread (registers are free here)
              for (int k0 = 0; k0 < parts; k0 += kBatch) {
                float2 ml[kBatch];
                float4 y[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                  ml[k] = make_float2(-INFINITY, 0.f);
                  y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                  if (k0 + k < parts) {
                    const float* s = slot_of(from + (k0 + k) * step);
                    ml[k] = __ldcg(reinterpret_cast<const float2*>(s + kHeads * DP + 2 * q));
                    y[k] = __ldcg(reinterpret_cast<const float4*>(s + q * DP + d));
                  }
                }
                float mn = m;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, ml[k].x);
                const float fo = ex2_rel(m, mn);
                m = mn;
                l *= fo;
#pragma unroll
                for (int z = 0; z < 4; ++z) x[z] *= fo;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                  const float f = ex2_rel(ml[k].x, mn);
                  l += ml[k].y * f;
                  x[0] += y[k].x * f; x[1] += y[k].y * f; x[2] += y[k].z * f; x[3] += y[k].w * f;
                }
              }
              if (final) emit(q, d, x, m, l);
            }
            if (!final) {
              __syncthreads();                        // a head's (maximum, sum) is read by all its threads
              if (mine) put(slot_of(from), q, d, x, m, l);
            }
          }
        };
        const int parts = c_last - c_first + 1;
        if (parts <= kGroup) {
          if (arrive_last(p.counters + c_first, parts)) join(c_first, 1, parts, true);
        } else {
          const int group = ((int)blockIdx.x - c_first) / kGroup, from = c_first + group * kGroup;
          const int size = min(kGroup, c_last + 1 - from), groups = (parts + kGroup - 1) / kGroup;
          if (arrive_last(p.counters + (group == 0 ? 1 : 2) * kMaxAttnCtas + from, size)) {
            join(from, 1, size, false);
            if (arrive_last(p.counters + c_first, groups)) join(c_first, kGroup, groups, true);
          }
        }
      }
      __syncthreads();                                // the stages and maxima are read: they may be refilled
      if (padded) {
        clear_pad(stage);
        __syncwarp();
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();

  // ---- sequences with nothing to attend to -----------------------------------------------------
  const int q_heads = p.Hk * p.G;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (clamp_len(__ldcg(p.lens + b), p.cap) > 0) continue;
    for (int e = tid; e < q_heads * (p.D / 4); e += kThreads) {
      const int h = e / (p.D / 4), d = (e % (p.D / 4)) * 4;
      if (C::kForm && p.prior_lse != nullptr) {
        const float none[4] = {0.f, 0.f, 0.f, 0.f};
        emit_joined(p, b, h, d, none, -INFINITY);
        continue;
      }
      *reinterpret_cast<uint2*>(p.out + (int64_t)b * p.out_ts + (int64_t)h * p.out_hs + d) = make_uint2(0, 0);
      if (d == 0 && p.lse != nullptr) p.lse[(int64_t)b * q_heads + h] = -INFINITY;
    }
  }
}

template <typename C>
cudaError_t launch(const AttnParams& p, const AttnPlan& plan, int64_t max_tiles, cudaStream_t stream, bool pdl) {
  static PerContextOnce once;
  static std::atomic<int> resident{C::kCtas};          // what fits an SM: the work is divided over one wave of CTAs
  const cudaError_t e = once.run([] {
    cudaError_t e = cudaFuncSetAttribute(attention_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemB);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attention_kernel<C>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attention_kernel<C>, C::kThreads, C::kSmemB);
    if (e == cudaSuccess) resident = n < 1 ? 1 : n < C::kCtas ? n : C::kCtas;
    return e;
  });
  if (e != cudaSuccess) return e;
  int64_t grid = max_tiles * (1 + kRunCost);
  if (grid > plan.grid_max) grid = plan.grid_max;
  if (grid > (int64_t)num_sms() * resident) grid = (int64_t)num_sms() * resident;
  return launch_k(attention_kernel<C>, dim3((unsigned)grid), dim3(C::kThreads), C::kSmemB, stream, pdl, p);
}

template <int DP, bool kFp8, bool kForm>
cudaError_t launch_nq(const AttnParams& p, const AttnPlan& plan, int64_t max_tiles, cudaStream_t stream, bool pdl) {
  if (plan.nq == 1)
    return p.q.f32 ? launch<Cfg<DP, kFp8, 1, true, kForm>>(p, plan, max_tiles, stream, pdl)
                   : launch<Cfg<DP, kFp8, 1, false, kForm>>(p, plan, max_tiles, stream, pdl);
  return p.q.f32 ? launch<Cfg<DP, kFp8, 2, true, kForm>>(p, plan, max_tiles, stream, pdl)
                 : launch<Cfg<DP, kFp8, 2, false, kForm>>(p, plan, max_tiles, stream, pdl);
}

template <bool kFp8, bool kForm>
cudaError_t launch_any(const AttnParams& p, const AttnPlan& plan, int64_t max_tiles, cudaStream_t stream, bool pdl) {
  return p.D <= 64    ? launch_nq<64, kFp8, kForm>(p, plan, max_tiles, stream, pdl)
         : p.D <= 128 ? launch_nq<128, kFp8, kForm>(p, plan, max_tiles, stream, pdl)
                      : launch_nq<256, kFp8, kForm>(p, plan, max_tiles, stream, pdl);
}

}  // namespace attn
}  // namespace engram
