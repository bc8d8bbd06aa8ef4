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
// Bound by HBM: a row is read once and written once. A row is held by 8, 16 or 32 lanes, 8 values each, so a
// norm is a few shuffles. Measured on a GB300 (share of the 6.78 TB/s of a plain copy): 32768 tokens of 32 + 8
// heads of 128 normed and turned in 103 us, 6.7 TB/s (0.98), 106 to 108 us (0.95) where three sets of rows take
// turns; 8 + 8 heads written as FP8 in 35 us (0.85), as bf16 in 41 us (0.96); read back in 34 us (0.88) and 41 us
// (0.96).
#include "attn.cuh"

namespace engram {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ void unpack8(uint4 a, float (&x)[8]) {
  x[0] = bf16_lo(a.x); x[1] = bf16_hi(a.x); x[2] = bf16_lo(a.y); x[3] = bf16_hi(a.y);
  x[4] = bf16_lo(a.z); x[5] = bf16_hi(a.z); x[6] = bf16_lo(a.w); x[7] = bf16_hi(a.w);
}

// (Weights and angles too are read with ordinary loads: this kernel may start before the one that writes them ends,
// and the non-coherent path wants data that nothing writes while a kernel lives.)
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// 8 values at p, as fp32 or bf16
__device__ __forceinline__ void store8(void* p, bool f32, const float (&x)[8]) {
  if (f32) {
    static_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    static_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *static_cast<uint4*>(p) = pack8(x);
  }
}
__device__ __forceinline__ uint8_t* row_of(const HeadRows& o, int64_t t, int h, int d0) {
  return static_cast<uint8_t*>(o.data) + (t * o.ts + h * o.hs + d0) * (o.f32 ? 4 : 2);
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

// The scale byte of a block: amax = 1.m * 2^(field - 127) is at most 448 * 2^e = 1.75 * 2^(8 + e) from
// e = field - 135 on, one more when 1.m > 1.75 (the sum below carries into the field then); byte 127 + e, at
// least 1, and 127 for an all-zero block. An infinity gets 2^127: 448 * 2^127 reads back as infinite.
__device__ __forceinline__ int scale_byte(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int byte = max((int)((bits + 0x1FFFFFu) >> 23) - 8, 1);
  return bits == 0 ? 127 : bits == 0x7F800000u ? 254 : byte;
}
// 2^-e of a scale byte 127 + e in [1, 254]: exact (a subnormal at the end)
__device__ __forceinline__ float inverse_scale(int byte) {
  return __uint_as_float(byte == 254 ? 0x00400000u : (uint32_t)(254 - byte) << 23);
}

// until at most n of a thread's copies are in flight (n < kRows, known when the loop is unrolled)
template <int kRows>
__device__ __forceinline__ void wait_rows(int n) {
  switch (n) {
    case 0: cp_async_wait<0>(); break;
    case 1: cp_async_wait<1>(); break;
    case 2: cp_async_wait<2>(); break;
    case 3: cp_async_wait<3>(); break;
    case 4: cp_async_wait<4>(); break;
    case 5: cp_async_wait<5>(); break;
    case 6: cp_async_wait<6>(); break;
    default: cp_async_wait<7>(); break;
  }
  static_assert(kRows <= 8, "");
}

// kLanes lanes hold one row (8 values each); a group of lanes takes kRows heads of one token. A block's rows
// are all queries, all keys or all values, so what is done to them is uniform and every shuffle has the whole
// warp; rows past the end are computed on zeros and not stored.
//
// All rows of a thread are requested at once by cp.async into places of its own in shared memory, so their
// bytes in flight do not depend on registers, and the angles are fetched behind them. Norm and turn are
//   out_i = r * (x_i * A_i + y_i * B_i),  r = 1 / sqrt(mean(x^2) + eps),  y_i the other value of x_i's pair,
// with A_i = w_i cos, B_i = -+ w_y sin formed once per token; y comes from the partner lane's place. Nine CTAs
// per SM (registers for them: up to 56): with eight 118 us instead of 110 for 32768 tokens of 32 + 8 heads, with ten
// spills, 133. That is bf16 rows; fp32 rows with 8 per group have 32 KB of places and six CTAs fit.
// kPairs: values 2i and 2i + 1 are turned, else i and i + R/2 (one kernel for both has a quarter more instructions:
// 110 us instead of 103 for the 32768 tokens above).
template <int kLanes, bool kF32, bool kPairs, int kRows>
__global__ void __launch_bounds__(kThreads, 9) qkv_kernel(const __grid_constant__ QkvParams p) {
  constexpr unsigned kWarp = 0xFFFFFFFFu;
  constexpr int kBytes = kF32 ? 4 : 2;
  constexpr int kParts = kF32 ? 2 : 1;                // 16-byte chunks per lane
  __shared__ uint4 place_of[kRows][kThreads * kParts];
  pdl_wait();
  pdl_trigger();                                      // never before the wait: a step's attention reads lengths at its start
  const bool is_q = blockIdx.x < p.first_k, is_v = blockIdx.x >= p.first_v;
  const HeadRows in = is_q ? p.q : is_v ? p.v : p.k;
  const HeadRows out = is_q ? p.q_out : is_v ? HeadRows{} : p.k_out;
  const uint16_t* wp = is_q ? p.nr.qw : is_v ? nullptr : p.nr.kw;
  const bool turn = !is_v && p.nr.R > 0;
  const bool to_cache = !is_q && p.cache.k != nullptr;
  const int tid = threadIdx.x, sub = tid & (kLanes - 1);
  const uint32_t block = blockIdx.x - (is_q ? 0u : is_v ? p.first_v : p.first_k);
  const int64_t item = (int64_t)block * (kThreads / kLanes) + tid / kLanes;
  const int groups = (in.heads + kRows - 1) / kRows;
  int64_t t = item < ((int64_t)1 << 31) ? fast_div((uint32_t)item, is_q ? p.div_q : p.div_kv) : item / groups;
  const int h0 = (int)(item - t * groups) * kRows;
  const bool there = t < p.T;
  if (!there) t = 0;
  const int d0 = sub * 8;
  const bool live = there && d0 < p.D;
  const int rows = live ? min(in.heads - h0, kRows) : 0;

  const int half = p.nr.R >> 1;
  const int r0 = d0 - p.nr.start;
  const bool turned = turn && live && r0 >= 0 && r0 < p.nr.R;
  int64_t pos = turned ? p.positions[t] : 0;  // (its angles are two loads away)
  // a group's lanes copy consecutive chunks; chunk c of a row lies at c ^ (c / 8 & 1), so that reads of two
  // chunks per lane (fp32) meet no bank twice
  auto chunk_at = [&](int c) { return (tid - sub) * kParts + (kF32 ? c ^ ((c >> 3) & 1) : c); };
  const uint8_t* src = static_cast<const uint8_t*>(in.data) + kBytes * (t * in.ts + h0 * in.hs);
  const int64_t step = kBytes * in.hs;
  const int there_rows = there ? in.heads - h0 : 0;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int z = 0; z < kParts; ++z) {
      const int c = sub + z * kLanes;
      if (r < there_rows && c * 16 < p.D * kBytes)
        cp_async16((uint32_t)__cvta_generic_to_shared(&place_of[r][chunk_at(c)]), src + 16 * c);
      else
        place_of[r][chunk_at(c)] = make_uint4(0, 0, 0, 0);
    }
    cp_async_commit();
    src += step;
  }

  // A and B of this thread's 8 values. A value of a second half takes + sin times its partner, one of a first
  // half - sin.
  int other = sub;
  float A[8], B[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { A[i] = 1.f; B[i] = 0.f; }
  if (turned) {
    if (pos < 0 || pos >= p.nr.rows) {
      if (p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_POSITION);
      pos = pos < 0 ? 0 : p.nr.rows - 1;
    }
    const float* row = p.nr.table + pos * p.nr.R;
    if (kPairs) {
      const float4 c = *reinterpret_cast<const float4*>(row + (r0 >> 1));
      const float4 s = *reinterpret_cast<const float4*>(row + half + (r0 >> 1));
      A[0] = A[1] = c.x; A[2] = A[3] = c.y; A[4] = A[5] = c.z; A[6] = A[7] = c.w;
      B[0] = -s.x; B[1] = s.x; B[2] = -s.y; B[3] = s.y; B[4] = -s.z; B[5] = s.z; B[6] = -s.w; B[7] = s.w;
    } else {
      const bool second = r0 >= half;
      const int i = second ? r0 - half : r0;
      load8(row + i, A);
      load8(row + half + i, B);
      other = second ? sub - (half >> 3) : sub + (half >> 3);
      if (!second) {
#pragma unroll
        for (int k = 0; k < 8; ++k) B[k] = -B[k];
      }
    }
  }
  if (wp != nullptr && live) {
    float w[8];
    unpack8(*reinterpret_cast<const uint4*>(wp + d0), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) A[i] *= w[i];
    if (turned) {
      if (!kPairs) unpack8(*reinterpret_cast<const uint4*>(wp + 8 * other), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) B[i] *= w[kPairs ? i ^ 1 : i];
    }
  }
  uint8_t *dst = nullptr, *scales = nullptr;          // this thread's place in the token's first row of the cache
  bool stored = false;
  if (to_cache) {
    const int64_t slot = p.slots[t];
    int64_t page, at;
    stored = place(p.cache, slot, &page, &at);
    if (stored) {
      dst = (is_v ? p.cache.v : p.cache.k) + page * p.cache.page_b + at * p.cache.tok_b + h0 * p.cache.head_b + (p.cache.fp8 ? d0 : 2 * d0);
      scales = (is_v ? p.cache.vs : p.cache.ks) + page * p.cache.spage_b + at * p.cache.stok_b + h0 * p.cache.shead_b + (d0 >> 5);
    }
    if (live && slot >= p.cache.slots && sub == 0 && p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_SLOT);
  }
  uint8_t* to = row_of(out, t, h0, d0);
  const int64_t to_step = out.hs * (out.f32 ? 4 : 2);

#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    wait_rows<kRows>(kRows - 1 - r);
    __syncwarp();                                     // what the warp's other lanes copied is there too
    auto values = [&](int s, float (&v)[8]) {         // lane s's of the group
      if (kF32) {
        const uint4 a = place_of[r][chunk_at(2 * s)], b = place_of[r][chunk_at(2 * s + 1)];
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
      } else {
        unpack8(place_of[r][chunk_at(s)], v);
      }
    };
    float x[8];
    values(sub, x);
    float inv = 1.f;
    if (wp != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kWarp, ss, o);
      inv = rsqrtf(ss * p.inv_d + p.nr.eps);
    }
    if (turn || wp != nullptr) {
      float y[8];
      if (kPairs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
      } else if (turn) {
        values(other, y);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= A[i];
      if (turned) {                                   // (a value that is not turned takes nothing from another)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += y[i] * B[i];
      }
      if (wp != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= inv;
      }
    }
    if (out.data != nullptr) {
      if (r < rows) store8(to, out.f32, x);
      to += to_step;
    }
    if (to_cache) {
      if (!p.cache.fp8) {
        if (r < rows && stored) *reinterpret_cast<uint4*>(dst) = pack8(x);
      } else {
        // the four lanes of a block of 32 values share its scale
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
        amax = fmaxf(amax, __shfl_xor_sync(kWarp, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kWarp, amax, 2));
        const int byte = scale_byte(amax);
        const float down = inverse_scale(byte);
        if (r < rows && stored) {
          uint2 codes;
          codes.x = code4(x[0] * down, x[1] * down, x[2] * down, x[3] * down);
          codes.y = code4(x[4] * down, x[5] * down, x[6] * down, x[7] * down);
          *reinterpret_cast<uint2*>(dst) = codes;
          if ((sub & 3) == 0) *scales = (uint8_t)byte;
        }
        scales += p.cache.shead_b;
      }
      dst += p.cache.head_b;
    }
  }
}

// Rows of the cache by slot, rounded once to the output's type; a slot below 0 or past the cache reads as
// zeros. A thread takes 8 values of kRows heads of a token: with the slot known, that is kRows loads in
// flight, and every store of the warp is a run of full sectors.
template <int kLanes, bool kFp8, int kRows>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ KvReadParams p) {
  pdl_wait();
  const int sub = threadIdx.x & (kLanes - 1);
  const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
  const int groups = (p.heads + kRows - 1) / kRows;
  const int64_t t = item < ((int64_t)1 << 31) ? fast_div((uint32_t)item, p.div_token) : item / (2 * groups);
  if (t >= p.T) return;
  const int group = (int)(item - t * 2 * groups);
  const bool is_v = group >= groups;
  const int h0 = (group - (is_v ? groups : 0)) * kRows;
  const int d0 = sub * 8;
  if (d0 >= p.D) return;
  const CacheRef& c = p.cache;
  const int64_t slot = p.slots[t];
  int64_t page = 0, at = 0;
  const bool ok = place(c, slot, &page, &at);
  if (slot >= c.slots && sub == 0 && p.err != nullptr) atomicOr(p.err, ENGRAM_ERR_SLOT);
  const uint8_t* row = (is_v ? c.v : c.k) + page * c.page_b + at * c.tok_b + h0 * c.head_b + (kFp8 ? d0 : 2 * d0);
  const uint8_t* scale = (is_v ? c.vs : c.ks) + page * c.spage_b + at * c.stok_b + h0 * c.shead_b + (d0 >> 5);
  uint4 raw[kRows];
  uint32_t byte[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    raw[r] = make_uint4(0, 0, 0, 0);
    byte[r] = 0;
    if (ok && h0 + r < p.heads) {
      if (kFp8) {
        const uint2 codes = *reinterpret_cast<const uint2*>(row + r * c.head_b);
        raw[r].x = codes.x;
        raw[r].y = codes.y;
        byte[r] = scale[r * c.shead_b];
      } else {
        raw[r] = *reinterpret_cast<const uint4*>(row + r * c.head_b);
      }
    }
  }
  const HeadRows& out = is_v ? p.v_out : p.k_out;
  const bool f32 = out.f32;
  uint8_t* to = row_of(out, t, h0, d0);
  const int64_t step = out.hs * (f32 ? 4 : 2);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (h0 + r >= p.heads) break;
    float x[8];
    if (kFp8) {
      const float f = __uint_as_float(byte[r] << 23);
      uint32_t hh[4];
      e4m3x4_to_f16x2(raw[r].x, hh[0], hh[1]);
      e4m3x4_to_f16x2(raw[r].y, hh[2], hh[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hh[i]));
        x[2 * i] = v.x * f;
        x[2 * i + 1] = v.y * f;
      }
    } else {
      unpack8(raw[r], x);
    }
    store8(to, f32, x);
    to += step;
  }
}

// Heads of one token that a group of lanes takes. More of them share the token's angles and slot and are in
// flight together: 32768 tokens of 32 + 8 heads of 128 are normed and turned in 312, 195, 133 and 110 us with 1,
// 2, 4 and 8. But few rows want lanes of their own: 256 tokens of 8 + 8 heads are written in 2.3 us with 1 and
// 3.7 us with 8 (half of the GPU's lanes or less), 1024 tokens in 4.1, 3.2, 3.2 and 4.0 us. Within those limits
// the choice wastes least: a group costs what its rows do, a part-filled one as much as a full one, and
// about three rows more.
int rows_per_group(int64_t T, const int (&heads)[3], int lanes) {
  const double fill = (double)T * (heads[0] + heads[1] + heads[2]) * lanes / (num_sms() * 2048.0);
  const int most = fill < 0.5 ? 1 : fill < 2.0 ? 4 : 8;
  int best = 1, least = 0;
  for (int r = 1; r <= most; r *= 2) {
    int cost = 0;
    for (int h : heads) cost += (h + r - 1) / r * (r + 3);
    if (r == 1 || cost < least) {
      best = r;
      least = cost;
    }
  }
  return best;
}

template <int kLanes, bool kF32, bool kPairs, int kRows>
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
  return launch_k(qkv_kernel<kLanes, kF32, kPairs, kRows>, dim3((unsigned)(nq + nk + nv)), dim3(kThreads), 0, stream, true, p);
}

template <int kLanes, bool kF32, bool kPairs>
cudaError_t go_rows(const QkvParams& p, cudaStream_t stream) {
  const int heads[3] = {p.q.heads, p.k.heads, p.v.heads};
  switch (rows_per_group(p.T, heads, kLanes)) {
    case 8: return go<kLanes, kF32, kPairs, 8>(p, stream);
    case 4: return go<kLanes, kF32, kPairs, 4>(p, stream);
    case 2: return go<kLanes, kF32, kPairs, 2>(p, stream);
    default: return go<kLanes, kF32, kPairs, 1>(p, stream);
  }
}

template <bool kF32, bool kPairs>
cudaError_t go_lanes(const QkvParams& p, cudaStream_t stream) {
  return p.D <= 64    ? go_rows<8, kF32, kPairs>(p, stream)
         : p.D <= 128 ? go_rows<16, kF32, kPairs>(p, stream)
                      : go_rows<32, kF32, kPairs>(p, stream);
}

template <int kLanes, bool kFp8, int kRows>
cudaError_t go_read(KvReadParams p, cudaStream_t stream) {
  const int groups = (p.heads + kRows - 1) / kRows;
  p.div_token = make_fastdiv((uint32_t)(2 * groups));
  const int64_t blocks = (p.T * 2 * groups * kLanes + kThreads - 1) / kThreads;
  if (blocks >= (int64_t)1 << 31) return cudaErrorInvalidValue;
  return launch_k(kv_read_kernel<kLanes, kFp8, kRows>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, true, p);
}

template <bool kFp8, int kRows>
cudaError_t go_read_lanes(const KvReadParams& p, cudaStream_t stream) {
  return p.D <= 64    ? go_read<8, kFp8, kRows>(p, stream)
         : p.D <= 128 ? go_read<16, kFp8, kRows>(p, stream)
                      : go_read<32, kFp8, kRows>(p, stream);
}
template <bool kFp8>
cudaError_t go_read_rows(const KvReadParams& p, cudaStream_t stream) {
  const int heads[3] = {0, p.heads, p.heads};
  switch (rows_per_group(p.T, heads, p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32)) {
    case 8: return go_read_lanes<kFp8, 8>(p, stream);
    case 4: return go_read_lanes<kFp8, 4>(p, stream);
    case 2: return go_read_lanes<kFp8, 2>(p, stream);
    default: return go_read_lanes<kFp8, 1>(p, stream);
  }
}

}  // namespace

cudaError_t launch_qkv(const QkvParams& p, cudaStream_t stream) {
  const bool f32 = p.q.data != nullptr ? p.q.f32 : p.k.f32;
  const bool pairs = p.nr.R > 0 && p.nr.interleaved;
  if (f32) return pairs ? go_lanes<true, true>(p, stream) : go_lanes<true, false>(p, stream);
  return pairs ? go_lanes<false, true>(p, stream) : go_lanes<false, false>(p, stream);
}

cudaError_t launch_kv_read(const KvReadParams& p, cudaStream_t stream) {
  return p.cache.fp8 ? go_read_rows<true>(p, stream) : go_read_rows<false>(p, stream);
}

}  // namespace engram
