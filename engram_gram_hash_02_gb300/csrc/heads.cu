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

// The exponent of a block's scale: amax = 1.m * 2^(field - 127) is at most 448 * 2^e = 1.75 * 2^(8 + e) from
// e = field - 135 on, one more when 1.m > 1.75. An infinity gets 2^127: 448 * 2^127 reads back as infinite.
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int field = (int)(bits >> 23);
  const int e = max(field - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);
  return amax == 0.f ? 0 : field == 255 ? 127 : e;
}

// kLanes lanes hold one row (8 values each); a group of lanes takes kRows heads of one token. A block's rows
// are all queries, all keys or all values, so what is done to them is uniform and every shuffle has the whole
// warp; rows past the end are computed on zeros and not stored.
template <int kLanes, bool kF32, int kRows>
__global__ void __launch_bounds__(kThreads) qkv_kernel(const __grid_constant__ QkvParams p) {
  pdl_wait();
  pdl_trigger();
  constexpr unsigned kWarp = 0xFFFFFFFFu;
  const bool is_q = blockIdx.x < p.first_k, is_v = blockIdx.x >= p.first_v;
  const HeadRows in = is_q ? p.q : is_v ? p.v : p.k;
  const HeadRows out = is_q ? p.q_out : is_v ? HeadRows{} : p.k_out;
  const uint16_t* wp = is_q ? p.nr.qw : is_v ? nullptr : p.nr.kw;
  const bool turn = !is_v && p.nr.R > 0;
  const bool to_cache = !is_q && p.cache.k != nullptr;
  const int sub = threadIdx.x & (kLanes - 1);
  const uint32_t block = blockIdx.x - (is_q ? 0u : is_v ? p.first_v : p.first_k);
  const int64_t item = (int64_t)block * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int groups = (in.heads + kRows - 1) / kRows;
  const FastDiv div = is_q ? p.div_q : p.div_kv;
  int64_t t = item < ((int64_t)1 << 31) ? fast_div((uint32_t)item, div) : item / groups;
  const int h0 = (int)(item - t * groups) * kRows;
  const bool there = t < p.T;
  if (!there) t = 0;
  const int d0 = sub * 8;
  const bool live = there && d0 < p.D;

  Raw<kF32> raw[kRows];
  const uint8_t* src = static_cast<const uint8_t*>(in.data) + (kF32 ? 4 : 2) * (t * in.ts + h0 * in.hs + d0);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (live && h0 + r < in.heads)
      raw[r].load(src + (kF32 ? 4 : 2) * (r * in.hs));
    else
      raw[r].zero();
  }

  // the token's angles for this thread's 8 values; values outside the turned part get angle 0. A value of a
  // second half takes + sin times its partner, one of a first half - sin.
  const int half = p.nr.R >> 1;
  const int r0 = d0 - p.nr.start;
  const bool turned = turn && r0 >= 0 && r0 < p.nr.R;
  const bool pairs = p.nr.interleaved;
  int other = sub;
  float cs[8], sn[8];
  if (turn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) { cs[i] = 1.f; sn[i] = 0.f; }
    if (turned) {
      int64_t pos = __ldg(p.positions + t);
      if (pos < 0 || pos >= p.nr.rows) {
        if (there && p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_POSITION);
        pos = pos < 0 ? 0 : p.nr.rows - 1;
      }
      const float* row = p.nr.table + pos * p.nr.R;
      if (pairs) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(row + (r0 >> 1)));
        const float4 b = __ldg(reinterpret_cast<const float4*>(row + half + (r0 >> 1)));
        cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w;
        sn[0] = b.x; sn[1] = b.y; sn[2] = b.z; sn[3] = b.w;
      } else {
        const bool second = r0 >= half;
        const int i = second ? r0 - half : r0;
        load8(row + i, cs);
        load8(row + half + i, sn);
        other = second ? sub - (half >> 3) : sub + (half >> 3);
        if (!second) {
#pragma unroll
          for (int k = 0; k < 8; ++k) sn[k] = -sn[k];
        }
      }
    }
  }
  float w[8];
  if (wp != nullptr) {
    Raw<false> rw;
    rw.zero();
    if (d0 < p.D) rw.load(wp + d0);
    rw.get(w);
  }
  uint8_t *rows = nullptr, *scales = nullptr;         // the token's place in the cache
  if (to_cache) {
    const int64_t slot = __ldg(p.slots + t);
    int64_t page, at;
    if (place(p.cache, slot, &page, &at) && there) {
      rows = (is_v ? p.cache.v : p.cache.k) + page * p.cache.page_b + at * p.cache.tok_b;
      scales = (is_v ? p.cache.vs : p.cache.ks) + page * p.cache.spage_b + at * p.cache.stok_b;
    }
    if (there && slot >= p.cache.slots && sub == 0 && p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_SLOT);
  }

#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int h = h0 + r;
    const bool mine = live && h < in.heads;
    float x[8];
    raw[r].get(x);
    if (wp != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kWarp, ss, o);
      const float inv = rsqrtf(ss * p.inv_d + p.nr.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
    }
    if (turn) {
      if (pairs) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[2 * i], b = x[2 * i + 1];
          x[2 * i] = a * cs[i] - b * sn[i];
          x[2 * i + 1] = b * cs[i] + a * sn[i];
        }
      } else {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(kWarp, x[i], other, kLanes);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * cs[i] + y[i] * sn[i];
      }
    }
    if (out.data != nullptr && mine) store8(out, t, h, d0, x);
    if (to_cache) {
      if (!p.cache.fp8) {
        if (mine && rows != nullptr) *reinterpret_cast<uint4*>(rows + h * p.cache.head_b + 2 * d0) = pack8(x);
      } else {
        // the four lanes of a block of 32 values share its scale
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
        amax = fmaxf(amax, __shfl_xor_sync(kWarp, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kWarp, amax, 2));
        const int e = block_exponent(amax);
        const float inv = pow2(-e);            // e <= 127: 2^-127 is a subnormal, exact
        if (mine && rows != nullptr) {
          uint2 codes;
          codes.x = code4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
          codes.y = code4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
          *reinterpret_cast<uint2*>(rows + h * p.cache.head_b + d0) = codes;
          if ((d0 & 31) == 0) scales[h * p.cache.shead_b + (d0 >> 5)] = (uint8_t)(127 + e);
        }
      }
    }
  }
}

// Rows of the cache by slot, rounded once to the output's type; a slot below 0 or past the cache reads as
// zeros. A thread takes 16 bytes of kRows heads of a token (16 codes or 8 bf16): with the slot known, that
// is kRows loads in flight.
template <int kLanes, bool kFp8, int kRows>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ KvReadParams p) {
  constexpr int kVals = kFp8 ? 16 : 8;
  const int sub = threadIdx.x & (kLanes - 1);
  const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
  const int groups = (p.heads + kRows - 1) / kRows;
  const int64_t t = item < ((int64_t)1 << 31) ? fast_div((uint32_t)item, p.div_token) : item / (2 * groups);
  if (t >= p.T) return;
  const int group = (int)(item - t * 2 * groups);
  const bool is_v = group >= groups;
  const int h0 = (group - (is_v ? groups : 0)) * kRows;
  const int d0 = sub * kVals;
  if (d0 >= p.D) return;
  const CacheRef& c = p.cache;
  const int64_t slot = __ldg(p.slots + t);
  int64_t page = 0, at = 0;
  const bool ok = place(c, slot, &page, &at);
  if (slot >= c.slots && sub == 0 && p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_SLOT);
  const uint8_t* row = (is_v ? c.v : c.k) + page * c.page_b + at * c.tok_b + h0 * c.head_b + sub * 16;
  const uint8_t* scale = (is_v ? c.vs : c.ks) + page * c.spage_b + at * c.stok_b + h0 * c.shead_b + (d0 >> 5);
  uint4 raw[kRows];
  uint32_t byte[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    raw[r] = make_uint4(0, 0, 0, 0);
    byte[r] = 0;
    if (ok && h0 + r < p.heads) {
      raw[r] = __ldg(reinterpret_cast<const uint4*>(row + r * c.head_b));
      if (kFp8) byte[r] = __ldg(scale + r * c.shead_b);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (h0 + r >= p.heads) break;
    float x[8];
    if (kFp8) {
      const float f = __uint_as_float(byte[r] << 23);
      const uint32_t w[4] = {raw[r].x, raw[r].y, raw[r].z, raw[r].w};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t hh[4];
        e4m3x4_to_f16x2(w[2 * half], hh[0], hh[1]);
        e4m3x4_to_f16x2(w[2 * half + 1], hh[2], hh[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hh[i]));
          x[2 * i] = v.x * f;
          x[2 * i + 1] = v.y * f;
        }
        store8(is_v ? p.v_out : p.k_out, t, h0 + r, d0 + 8 * half, x);
      }
    } else {
      Raw<false> b;
      b.a = raw[r];
      b.get(x);
      store8(is_v ? p.v_out : p.k_out, t, h0 + r, d0, x);
    }
  }
}

template <int kLanes, bool kF32, int kRows>
cudaError_t go(QkvParams p, cudaStream_t stream) {
  const int64_t per_block = kThreads / kLanes;
  auto blocks = [&](const HeadRows& r) {
    const int64_t items = p.T * ((r.heads + kRows - 1) / kRows);
    return (items + per_block - 1) / per_block;
  };
  const int64_t nq = blocks(p.q), nk = blocks(p.k), nv = blocks(p.v);
  if (nq + nk + nv >= (int64_t)1 << 31) return cudaErrorInvalidValue;
  p.first_k = (uint32_t)nq;
  p.first_v = (uint32_t)(nq + nk);
  p.div_q = make_fastdiv((uint32_t)max((p.q.heads + kRows - 1) / kRows, 1));
  p.div_kv = make_fastdiv((uint32_t)max((p.k.heads + kRows - 1) / kRows, 1));   // v has k's heads
  p.inv_d = 1.f / (float)p.D;
  return launch_k(qkv_kernel<kLanes, kF32, kRows>, dim3((unsigned)(nq + nk + nv)), dim3(kThreads), 0, stream, false, p);
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

template <int kLanes, bool kFp8, int kRows>
cudaError_t go_read(KvReadParams p, cudaStream_t stream) {
  const int groups = (p.heads + kRows - 1) / kRows;
  p.div_token = make_fastdiv((uint32_t)(2 * groups));
  const int64_t blocks = (p.T * 2 * groups * kLanes + kThreads - 1) / kThreads;
  if (blocks >= (int64_t)1 << 31) return cudaErrorInvalidValue;
  return launch_k(kv_read_kernel<kLanes, kFp8, kRows>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, false, p);
}

template <bool kFp8, int kRows>
cudaError_t go_read_lanes(const KvReadParams& p, cudaStream_t stream) {
  const int bytes = kFp8 ? p.D : 2 * p.D;              // 16 per lane
  return bytes <= 64    ? go_read<4, kFp8, kRows>(p, stream)
         : bytes <= 128 ? go_read<8, kFp8, kRows>(p, stream)
         : bytes <= 256 ? go_read<16, kFp8, kRows>(p, stream)
                        : go_read<32, kFp8, kRows>(p, stream);
}

}  // namespace

cudaError_t launch_qkv(const QkvParams& p, cudaStream_t stream) {
  const bool f32 = p.q.data != nullptr ? p.q.f32 : p.k.f32;
  return f32 ? go_lanes<true>(p, stream) : go_lanes<false>(p, stream);
}

cudaError_t launch_kv_read(const KvReadParams& p, cudaStream_t stream) {
  // as above: four rows per thread once every resident thread has that many
  const bool many = p.T * p.heads * p.D / 8 > (int64_t)num_sms() * 2048 * 4;
  if (p.cache.fp8) return many ? go_read_lanes<true, 4>(p, stream) : go_read_lanes<true, 1>(p, stream);
  return many ? go_read_lanes<false, 4>(p, stream) : go_read_lanes<false, 1>(p, stream);
}

}  // namespace engram
