// Attention of prompts: the list of its work (one CTA), the join of pairs that many CTAs share, and the launches.
#include "prompt.cuh"

#include <mutex>

namespace engram {
namespace prompt {
namespace {

constexpr int kPlanThreads = 1024;

// inclusive sum over the block; `total` for all
__device__ int64_t block_scan(int64_t x, int64_t* warps, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                                    // the last call's sums are read
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll 4
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += warps[w];
    total += warps[w];
  }
  return before + x;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Args a) {
  __shared__ int64_t warps[kPlanThreads / 32];
  const PromptParams& p = a.p;
  const int R = pair_rows(p.D);
  pdl_wait();
  pdl_trigger();
  if (a.join)
    for (int k = threadIdx.x; k < a.ctas * 8; k += kPlanThreads) a.counters[k] = 0;
  auto bounds = [&](int b, int& s0, int& n, int& len) {
    const int c0 = __ldcg(p.cu + b), c1 = __ldcg(p.cu + b + 1), raw = __ldcg(p.lens + b);
    s0 = (int)min((int64_t)max(c0, 0), p.T);
    n = (int)min((int64_t)max(c1, 0), p.T) - s0;
    len = clamp_len(raw, p.cap);
    const bool odd = c0 < 0 || c0 > p.T || c1 > p.T || c1 < c0 || raw != len || (p.own_lens == nullptr && n > len);
    n = max(n, 0);
    return odd;
  };
  // ---- the sequences' pairs of tiles
  int64_t run = 0, total;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int64_t pairs = 0;
    if (b < p.B) {
      int s0, n, len;
      if (bounds(b, s0, n, len) && p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_SEQ_LEN);
      pairs = ((int64_t)n * p.G + R - 1) / R;
    }
    const int64_t sum = block_scan(pairs, warps, total);
    // (sequences that share rows, against the rules, may come to more pairs than there are rows for: the rest is left out)
    if (b < p.B) a.offsets[b] = (int32_t)min(run + sum - pairs, a.max_entries);
    run += total;
  }
  const int E = (int)min(run, a.max_entries);
  __syncthreads();
  // ---- what their rows see: up to 32 lanes to an entry, which look at its tokens in turn
  const int lanes_log = E <= kPlanThreads / 32 ? 5 : E <= kPlanThreads / 16 ? 4 : E <= kPlanThreads / 8 ? 3 : E <= kPlanThreads / 4 ? 2 : E <= kPlanThreads / 2 ? 1 : 0, lanes = 1 << lanes_log;
  const bool arrays = p.doc_starts != nullptr || p.prefix_ends != nullptr;
  for (int e0 = 0; e0 < E; e0 += kPlanThreads >> lanes_log) {
    const int e = e0 + (threadIdx.x >> lanes_log), sub = threadIdx.x & (lanes - 1);
    Entry x{};
    int lo = 0x7FFFFFFF, hi = 0, max_lo = 0, min_hi = 0x7FFFFFFF;
    auto take = [&](int i) {
      int l, h, pos;
      visible(p, x.s0, x.n, x.len, i, l, h, pos);
      if (l < h) {
        lo = min(lo, l);
        hi = max(hi, h);
        max_lo = max(max_lo, l);
        min_hi = min(min_hi, h);
      }
    };
    if (e < E) {
      int first = 0, past = p.B;                      // the last sequence whose first pair is e or before
      while (past - first > 1) {
        const int mid = (first + past) / 2;
        (a.offsets[mid] <= e ? first : past) = mid;
      }
      x.b = first;
      bounds(x.b, x.s0, x.n, x.len);
      x.row0 = (e - a.offsets[x.b]) * R;
      x.rows = (int)min((int64_t)x.n * p.G, (int64_t)x.row0 + R);
      const int i0 = (int)fast_div((uint32_t)x.row0, a.div_g), i1 = (int)fast_div((uint32_t)(x.rows - 1), a.div_g);
      if (arrays) {
#pragma unroll 4
        for (int i = i0 + sub; i <= i1; i += lanes) take(i);
      } else if (sub == 0) {
        // without arrays lo and hi only grow along the tokens: the first that sees anything and the last say it all
        const int from = p.own_lens == nullptr && p.causal ? max(i0, x.n - x.len) : i0;
        if (from <= i1) {
          take(from);
          take(i1);
        }
      }
    }
    for (int o = 1; o < lanes; o <<= 1) {
      lo = min(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
      max_lo = max(max_lo, __shfl_xor_sync(0xFFFFFFFFu, max_lo, o));
      min_hi = min(min_hi, __shfl_xor_sync(0xFFFFFFFFu, min_hi, o));
    }
    if (e < E && sub == 0) {
      x.hi = hi;
      x.max_lo = max_lo;
      x.min_hi = min_hi;
      x.key0 = a.box > 0 ? lo & ~(a.box - 1) : lo;    // boxes start where they do in their pages
      x.units = lo < hi ? (hi - x.key0 + kKeys - 1) / kKeys : 0;
      a.entries[e] = x;
    }
  }
  __syncthreads();
  // ---- their places, and what every CTA takes
  run = 0;
  for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
    const int e = e0 + threadIdx.x;
    const int units = e < E ? a.entries[e].units : 0;
    const int64_t mine = units > 0 ? units + kRunCost : 0;
    const int64_t sum = block_scan(mine, warps, total);
    if (e < E) a.entries[e].place = run + sum - mine;
    run += total;
  }
  const int64_t U = run, all = U * p.Hk, per = max((all + a.ctas - 1) / a.ctas, (int64_t)1);
  if (threadIdx.x == 0) {
    a.header->entries = E;
    a.header->places = U;
    a.header->per_cta = per;
  }
  __syncthreads();
  // a CTA's first place is in the last entry of work that starts there or before
  for (int c = threadIdx.x; c < a.ctas; c += kPlanThreads) {
    const int64_t at = c * per;
    if (at >= all) continue;
    const int head = (int)(at / U);
    const int64_t in_head = at - head * U;
    int first = 0, past = E;
    while (past - first > 1) {
      const int mid = (first + past) / 2;
      (a.entries[mid].place <= in_head ? first : past) = mid;
    }
    a.starts[c] = Start{head, first};
  }
}

// rows of pairs that were cut, joined by as many warps as there are blocks of 32 rows by 16 values
__global__ void __launch_bounds__(256) join_kernel(const Args a) {
  const PromptParams& p = a.p;
  const int R = pair_rows(p.D), lane = threadIdx.x & 31;
  pdl_wait();
  const int64_t E = a.header->entries, U = a.header->places, per = a.header->per_cta;
  const int64_t warps = (int64_t)gridDim.x * 8, items = E * p.Hk;
  // where there are pairs enough, a warp goes through a pair's rows itself: most of them may be short of rows
  const int chunks = p.D / 16, split = items * chunks >= warps / 2 ? 1 : R / 32;
  for (int64_t k = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); k < items * chunks * split; k += warps) {
    const int64_t item = k / (chunks * split);
    const int rest = (int)(k - item * (chunks * split)), head = (int)(item / E);
    const Entry& x = a.entries[item - head * E];
    if (x.units == 0) continue;
    const int64_t run0 = head * U + x.place + kRunCost;
    const int first = (int)(run0 / per), last = (int)((run0 + x.units - 1) / per);
    if (first == last) continue;
    for (int r_in = (rest % split) * 32 + lane; r_in < x.rows - x.row0; r_in += split * 32) {
      const int r = x.row0 + r_in, i = (int)fast_div((uint32_t)r, a.div_g);
      join16(a, first, last, R, r_in, (int64_t)x.s0 + i, head * p.G + r - i * p.G, (rest / split) * 16);
    }
  }
}

// Tokens of a TMA box: the largest power of two up to 64 that divides a page, 8 at least (eight 128-byte rows are the
// swizzle's pattern); 0: rows are fetched one by one. (Larger boxes would only start key tiles further ahead of a window.)
int box_of(const CacheRef& c) {
  int box = 64;
  while (c.page_size % box != 0) box /= 2;
  return box >= 8 && c.num_pages > 0 ? box : 0;
}

// A tensor map with the values of a row innermost; an axis of one entry is never stepped along, whatever its stride says.
// False if the strides do not fit one.
bool make_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const int64_t* dims, const int64_t* strides_b,
              const uint32_t* box, bool swizzle, int64_t row_b) {
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Encode fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<Encode>(f);
  });
  if (fn == nullptr) return false;
  cuuint64_t n[4], step[3];
  cuuint32_t b[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    n[i] = (cuuint64_t)dims[i];
    b[i] = box[i];
    if (i == 0) continue;
    step[i - 1] = (cuuint64_t)(dims[i] == 1 ? row_b : strides_b[i - 1]);
    if (step[i - 1] == 0 || step[i - 1] >= (cuuint64_t)1 << 40) return false;
  }
  return fn(m, type, (cuuint32_t)rank, const_cast<void*>(base), n, step, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the cache's keys or values as [page][head][place][value], boxes of `box` tokens by 128 bytes: bf16 in the MMAs' swizzle,
// codes as they are
bool map_pages(CUtensorMap* m, const void* base, const PromptParams& p, int box) {
  const CacheRef& c = p.cache;
  const int64_t dims[4] = {p.D, c.page_size, p.Hk, c.num_pages}, strides[3] = {c.tok_b, c.head_b, c.page_b};
  const uint32_t boxes[4] = {c.fp8 ? 128u : 64u, (uint32_t)box, 1, 1};
  return make_map(m, c.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, boxes, !c.fp8,
                  (int64_t)p.D * (c.fp8 ? 1 : 2));
}

// queries as [token][head][value], a tile's worth of whole tokens to a box
bool map_queries(CUtensorMap* m, const PromptParams& p) {
  if (128 % p.G != 0) return false;
  const int64_t dims[3] = {p.D, (int64_t)p.Hk * p.G, p.T}, strides[2] = {p.q.hs * 2, p.q.ts * 2};
  const uint32_t box[3] = {64, (uint32_t)p.G, (uint32_t)(128 / p.G)};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.q.data, dims, strides, box, true, (int64_t)p.D * 2);
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

Layout layout_of(int32_t G, int32_t D, int64_t T, int32_t B, int ctas) {
  Layout l;
  const int R = pair_rows(D);
  l.max_entries = (T * G + R - 1) / R + B;
  l.slot_floats = R * (D + 2);
  l.header = kAttnZeroBytes;
  l.counters = l.header + 256;
  l.starts = l.counters + round256((size_t)ctas * 8 * sizeof(uint32_t));
  l.offsets = l.starts + round256((size_t)ctas * sizeof(Start));
  l.entries = l.offsets + round256(((size_t)B + 1) * sizeof(int32_t));
  l.parts = l.entries + round256((size_t)l.max_entries * sizeof(Entry));
  l.all = l.parts + (size_t)2 * ctas * l.slot_floats * sizeof(float);
  return l;
}

}  // namespace
}  // namespace prompt

size_t prompt_workspace_bytes(int32_t Hk, int32_t G, int32_t D, bool fp8, int64_t T, int32_t B, int sms) {
  return prompt::layout_of(G, D, T, B, sms).all;
}

cudaError_t launch_prompt(const PromptParams& p, cudaStream_t stream) {
  using namespace prompt;
  Args a{};
  a.p = p;
  a.ctas = num_sms();
  const Layout l = layout_of(p.G, p.D, p.T, p.B, a.ctas);
  a.header = reinterpret_cast<Header*>(p.workspace + l.header);
  a.starts = reinterpret_cast<Start*>(p.workspace + l.starts);
  a.offsets = reinterpret_cast<int32_t*>(p.workspace + l.offsets);
  a.entries = reinterpret_cast<Entry*>(p.workspace + l.entries);
  a.counters = reinterpret_cast<uint32_t*>(p.workspace + l.counters);
  a.parts = reinterpret_cast<float*>(p.workspace + l.parts);
  a.slot_floats = l.slot_floats;
  a.max_entries = l.max_entries;
  a.div_g = make_fastdiv((uint32_t)p.G);
  // Few pairs have many parts each: a kernel behind this one joins them on all SMs. With a pair per CTA and more a pair is
  // cut once or twice, and the last to arrive joins it.
  const int R = pair_rows(p.D);
  a.join = (p.T * p.G + R - 1) / R * p.Hk >= a.ctas;
  CUtensorMap tm_k{}, tm_v{}, tm_q{};
  a.box = box_of(p.cache);
  if (a.box > 0 && !(map_pages(&tm_k, p.cache.k, p, a.box) && map_pages(&tm_v, p.cache.v, p, a.box))) a.box = 0;
  a.q_box = map_queries(&tm_q, p);
  cudaError_t e = launch_k(plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, true, a);
  if (e == cudaSuccess) e = p.cache.fp8 ? launch_fp8(tm_k, tm_v, tm_q, a, stream) : launch_bf16(tm_k, tm_v, tm_q, a, stream);
  if (e == cudaSuccess && !a.join) e = launch_k(join_kernel, dim3((unsigned)a.ctas * 2), dim3(256), 0, stream, true, a);
  return e;
}

}  // namespace engram
