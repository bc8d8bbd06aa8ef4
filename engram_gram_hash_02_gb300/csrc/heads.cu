// Rows of heads on their way to and from the attention's paged cache.
//
// qkv_kernel takes the query, key and value rows of T tokens. A query or key row x of D values becomes
//   y = x / sqrt(mean(x^2) + eps) * w,
// and pairs (a, b) of its part [start, start + R) are turned by the angle of their position:
//   a' = a cos - b sin, b' = b cos + a sin
// (pairs i and i + R/2, or 2i and 2i + 1). The result is rounded once, to an output row or to the cache.
// Value rows go to the cache as they are. A row of an FP8 cache is cut into blocks of 32: the block's
// scale is the smallest 2^e with max|x| / 2^e <= 448, e >= -126, and a code is x / 2^e rounded to the
// nearest e4m3 value, ties to even (the convention of the FP8 tables; an all-zero block has byte 127).
//
// Bound by HBM: a row is read once and written once. A row is held by 8, 16 or 32 lanes, 8 values
// each (16-byte loads of bf16), so a norm is a few shuffles; a group of lanes takes several heads of one
// token when there are enough rows to fill the GPU, so the token's angles are read once for all of them.
#include "attn.cuh"

namespace engram {
namespace {

constexpr int kThreads = 128;

template <bool kF32>
struct Raw;
template <>
struct Raw<false> {
  uint4 a;
  __device__ void load(const void* p) { a = *static_cast<const uint4*>(p); }   // not ld.nc: the output may be the input
  __device__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&x)[8]) const {
    x[0] = bf16_lo(a.x); x[1] = bf16_hi(a.x); x[2] = bf16_lo(a.y); x[3] = bf16_hi(a.y);
    x[4] = bf16_lo(a.z); x[5] = bf16_hi(a.z); x[6] = bf16_lo(a.w); x[7] = bf16_hi(a.w);
  }
};
template <>
struct Raw<true> {
  float4 a, b;
  __device__ void load(const void* p) {
    a = *static_cast<const float4*>(p);
    b = *(static_cast<const float4*>(p) + 1);
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

__device__ __forceinline__ void store8(const HeadRows& o, int64_t t, int h, int d0, const float (&x)[8]) {
  const int64_t i = t * o.ts + h * o.hs + d0;
  if (o.f32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(o.data) + i);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.data) + i) = pack8(x);
  }
}

// byte offsets of slot's row of head h: false if the slot is out of range
__device__ __forceinline__ bool place(const CacheRef& c, int64_t slot, int64_t* page, int64_t* at) {
  if (slot < 0 || slot >= c.slots) return false;
  if (slot < ((int64_t)1 << 31)) {
    *page = fast_div((uint32_t)slot, c.div_page);
  } else {
    *page = slot / c.page_size;
  }
  *at = slot - *page * c.page_size;
  return true;
}

__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// 2^e for e in [-149, 127], exactly (a subnormal below -126)
__device__ __forceinline__ float pow2(int e) {
  return e >= -126 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(1u << (149 + e));
}

// one row's 8 values of this thread to the cache; the four lanes of a block of 32 values share its scale
__device__ __forceinline__ void cache_store(const CacheRef& c, uint8_t* rows, uint8_t* scales, int64_t page, int64_t at,
                                            int h, int d0, bool live, unsigned group, const float (&x)[8]) {
  if (!c.fp8) {
    if (live) *reinterpret_cast<uint4*>(rows + page * c.page_b + h * c.head_b + at * c.tok_b + 2 * d0) = pack8(x);
    return;
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(group, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(group, amax, 2));
  // amax = 1.m * 2^(field - 127) is at most 448 * 2^e = 1.75 * 2^(8 + e) from e = field - 135 on, one more
  // when 1.m > 1.75. An infinity gets 2^127: 448 * 2^127 reads back as infinite.
  const uint32_t bits = __float_as_uint(amax);
  const int field = (int)(bits >> 23);
  int e = field - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, -126);
  if (field == 255) e = 127;
  if (amax == 0.f) e = 0;
  const float inv = pow2(-e);                  // e <= 127: 2^-127 is a subnormal, exact
  if (live) {
    uint2 w;
    w.x = code4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    w.y = code4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
    *reinterpret_cast<uint2*>(rows + page * c.page_b + h * c.head_b + at * c.tok_b + d0) = w;
    if ((d0 & 31) == 0)
      scales[page * c.spage_b + h * c.shead_b + at * c.stok_b + (d0 >> 5)] = (uint8_t)(127 + e);
  }
}

// kLanes lanes hold one row (8 values each); a group of lanes takes kRows heads of one token
template <int kLanes, bool kF32, int kRows>
__global__ void __launch_bounds__(kThreads) qkv_kernel(const QkvParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int sub = lane & (kLanes - 1);
  const unsigned group = (kLanes == 32 ? 0xFFFFFFFFu : ((1u << (kLanes & 31)) - 1u)) << (lane - sub);
  const int per_token = p.nq + p.nk + p.nv;
  const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
  if (item >= p.T * per_token) return;
  const int64_t t = item < ((int64_t)1 << 31) ? fast_div((uint32_t)item, p.div_token) : item / per_token;
  int c = (int)(item - t * per_token);
  const bool is_q = c < p.nq;
  const bool is_v = c >= p.nq + p.nk;
  if (!is_q) c -= is_v ? p.nq + p.nk : p.nq;
  const HeadRows& in = is_q ? p.q : is_v ? p.v : p.k;
  const int h0 = c * kRows;
  const int d0 = sub * 8;
  const bool live = d0 < p.D;

  Raw<kF32> raw[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (live && h0 + r < in.heads)
      raw[r].load(static_cast<const uint8_t*>(in.data) + (kF32 ? 4 : 2) * (t * in.ts + (h0 + r) * in.hs + d0));
    else
      raw[r].zero();
  }

  // the token's angles for this thread's 8 values
  const NormRope& nr = p.nr;
  const int half = nr.R >> 1;
  const int r0 = d0 - nr.start;
  const bool turn = !is_v && nr.R > 0;
  const bool turned = turn && r0 >= 0 && r0 < nr.R;
  const bool second = r0 >= half;
  float cs[8], sn[8];
  if (turned) {
    int64_t pos = __ldg(p.positions + t);
    if (pos < 0 || pos >= nr.rows) {
      if (p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_POSITION);
      pos = pos < 0 ? 0 : nr.rows - 1;
    }
    const float* row = nr.table + pos * nr.R;
    if (nr.interleaved) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + (r0 >> 1)));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + half + (r0 >> 1)));
      cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w;
      sn[0] = b.x; sn[1] = b.y; sn[2] = b.z; sn[3] = b.w;
    } else {
      const int i = second ? r0 - half : r0;
      load8(row + i, cs);
      load8(row + half + i, sn);
    }
  }
  const uint16_t* wp = is_v ? nullptr : is_q ? nr.qw : nr.kw;
  float w[8];
  if (wp != nullptr && live) {
    Raw<false> rw;
    rw.load(wp + d0);
    rw.get(w);
  }
  int64_t page = 0, at = 0;
  const bool to_cache = !is_q && p.cache.k != nullptr;
  bool stored = false;
  if (to_cache) {
    const int64_t slot = __ldg(p.slots + t);
    stored = place(p.cache, slot, &page, &at);
    if (slot >= p.cache.slots && sub == 0 && p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_SLOT);
  }

#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int h = h0 + r;
    if (h >= in.heads) break;
    float x[8];
    raw[r].get(x);
    if (wp != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
      const float inv = rsqrtf(ss / (float)p.D + nr.eps);
      if (live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
      }
    }
    if (turn) {
      if (nr.interleaved) {
        if (turned) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * cs[i] - b * sn[i];
            x[2 * i + 1] = b * cs[i] + a * sn[i];
          }
        }
      } else {
        const int other = turned ? (second ? sub - (half >> 3) : sub + (half >> 3)) : sub;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = __shfl_sync(group, x[i], other, kLanes);
          if (turned) x[i] = second ? x[i] * cs[i] + y * sn[i] : x[i] * cs[i] - y * sn[i];
        }
      }
    }
    if (is_q) {
      if (live) store8(p.q_out, t, h, d0, x);
    } else {
      if (!is_v && p.k_out.data != nullptr && live) store8(p.k_out, t, h, d0, x);
      if (stored)
        cache_store(p.cache, is_v ? p.cache.v : p.cache.k, is_v ? p.cache.vs : p.cache.ks, page, at, h, d0, live, group, x);
    }
  }
}

// rows of the cache by slot: 8 values per thread, rounded once to the output's type; a slot below 0 or
// past the cache reads as zeros
template <int kLanes, bool kFp8>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadParams p) {
  const int sub = threadIdx.x & (kLanes - 1);
  const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
  const int per_token = 2 * p.heads;
  if (item >= p.T * per_token) return;
  const int64_t t = item < ((int64_t)1 << 31) ? fast_div((uint32_t)item, p.div_token) : item / per_token;
  int h = (int)(item - t * per_token);
  const bool is_v = h >= p.heads;
  if (is_v) h -= p.heads;
  const int d0 = sub * 8;
  if (d0 >= p.D) return;
  const CacheRef& c = p.cache;
  const int64_t slot = __ldg(p.slots + t);
  int64_t page, at;
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (place(c, slot, &page, &at)) {
    const uint8_t* row = (is_v ? c.v : c.k) + page * c.page_b + h * c.head_b + at * c.tok_b;
    if (kFp8) {
      const uint2 codes = __ldg(reinterpret_cast<const uint2*>(row + d0));
      const uint8_t byte = __ldg((is_v ? c.vs : c.ks) + page * c.spage_b + h * c.shead_b + at * c.stok_b + (d0 >> 5));
      const float scale = __uint_as_float((uint32_t)byte << 23);
      uint32_t hh[4];
      e4m3x4_to_f16x2(codes.x, hh[0], hh[1]);
      e4m3x4_to_f16x2(codes.y, hh[2], hh[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hh[i]));
        x[2 * i] = f.x * scale;
        x[2 * i + 1] = f.y * scale;
      }
    } else {
      Raw<false> r;
      r.load(row + 2 * d0);
      r.get(x);
    }
  } else if (slot >= c.slots && sub == 0 && p.err != nullptr) {
    atomicOr(p.err, ENGRAM_ERR_SLOT);
  }
  store8(is_v ? p.v_out : p.k_out, t, h, d0, x);
}

template <int kLanes, bool kF32, int kRows>
cudaError_t go(QkvParams p, cudaStream_t stream) {
  p.nq = (p.q.heads + kRows - 1) / kRows;
  p.nk = (p.k.heads + kRows - 1) / kRows;
  p.nv = (p.v.heads + kRows - 1) / kRows;
  const int per_token = p.nq + p.nk + p.nv;
  p.div_token = make_fastdiv((uint32_t)per_token);
  const int64_t blocks = (p.T * per_token * kLanes + kThreads - 1) / kThreads;
  if (blocks >= (int64_t)1 << 31) return cudaErrorInvalidValue;
  return launch_k(qkv_kernel<kLanes, kF32, kRows>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, false, p);
}

template <int kLanes, bool kF32>
cudaError_t go_rows(const QkvParams& p, cudaStream_t stream) {
  // four heads per group of lanes share the token's angles and keep four loads in flight; with fewer rows
  // than four per resident group of lanes every row gets its own lanes
  const int64_t rows = p.T * (p.q.heads + p.k.heads + p.v.heads);
  return rows * kLanes > (int64_t)num_sms() * 2048 * 4 ? go<kLanes, kF32, 4>(p, stream) : go<kLanes, kF32, 1>(p, stream);
}

template <bool kF32>
cudaError_t go_lanes(const QkvParams& p, cudaStream_t stream) {
  return p.D <= 64 ? go_rows<8, kF32>(p, stream) : p.D <= 128 ? go_rows<16, kF32>(p, stream) : go_rows<32, kF32>(p, stream);
}

template <int kLanes>
cudaError_t go_read(KvReadParams p, cudaStream_t stream) {
  p.div_token = make_fastdiv((uint32_t)(2 * p.heads));
  const int64_t blocks = (p.T * 2 * p.heads * kLanes + kThreads - 1) / kThreads;
  if (blocks >= (int64_t)1 << 31) return cudaErrorInvalidValue;
  return launch_k(p.cache.fp8 ? kv_read_kernel<kLanes, true> : kv_read_kernel<kLanes, false>, dim3((unsigned)blocks),
                  dim3(kThreads), 0, stream, false, p);
}

}  // namespace

cudaError_t launch_qkv(const QkvParams& p, cudaStream_t stream) {
  const bool f32 = p.q.data != nullptr ? p.q.f32 : p.k.f32;
  return f32 ? go_lanes<true>(p, stream) : go_lanes<false>(p, stream);
}

cudaError_t launch_kv_read(const KvReadParams& p, cudaStream_t stream) {
  return p.D <= 64 ? go_read<8>(p, stream) : p.D <= 128 ? go_read<16>(p, stream) : go_read<32>(p, stream);
}

}  // namespace engram
