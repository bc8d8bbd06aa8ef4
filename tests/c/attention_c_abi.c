/* The attention calls from plain C: four tokens of two sequences normed, turned and written to an FP8
 * cache, read back, and attended to, with values that can be told beforehand. Prints "ok". */
#include <cuda_runtime_api.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "engram.h"

#define HQ 4
#define HK 2
#define D 64
#define PAGE 2
#define PAGES 4
#define T 4

#define CHECK(x)                                                                                        \
  do {                                                                                                  \
    int rc_ = (int)(x);                                                                                 \
    if (rc_ != 0) {                                                                                     \
      printf("line %d: %d %s\n", __LINE__, rc_, engram_last_error());                                   \
      return 1;                                                                                         \
    }                                                                                                   \
  } while (0)

static float bf16(uint16_t b) {
  uint32_t u = (uint32_t)b << 16;
  float f;
  memcpy(&f, &u, 4);
  return f;
}

static void* upload(const void* src, size_t n) {
  void* d = NULL;
  if (cudaMalloc(&d, n) != cudaSuccess) exit(2);
  if (src ? cudaMemcpy(d, src, n, cudaMemcpyHostToDevice) : cudaMemset(d, 0, n)) exit(2);
  return d;
}

int main(void) {
  static float q[T][HQ][D], k[T][HK][D], v[T][HK][D], table[8][D];
  static uint16_t ones[D], out[2][HQ][D];
  static float back[T][HK][D], kept[T][HK][D], lse[2][HQ];
  int t, h, i;
  for (i = 0; i < D; ++i) ones[i] = 0x3F80;
  for (t = 0; t < 8; ++t)
    for (i = 0; i < D / 2; ++i) {
      table[t][i] = (float)cos(t * pow(10000.0, -2.0 * i / D));
      table[t][D / 2 + i] = (float)sin(t * pow(10000.0, -2.0 * i / D));
    }
  /* constant rows: normed to ones; token t's values are all 2^t */
  for (t = 0; t < T; ++t) {
    for (h = 0; h < HQ; ++h)
      for (i = 0; i < D; ++i) q[t][h][i] = 3.0f;
    for (h = 0; h < HK; ++h)
      for (i = 0; i < D; ++i) {
        k[t][h][i] = 0.25f;
        v[t][h][i] = (float)(1 << t);
      }
  }
  /* tokens 0, 1 and 2 are sequence 0 (pages 3 and 1), token 3 is sequence 1 (page 0) */
  const int32_t positions[T] = {0, 1, 2, 0};
  const int64_t slots[T] = {6, 7, 2, 0};
  const int32_t pages[2][2] = {{3, 1}, {0, -1}};
  const int32_t lens[2] = {3, 1};

  EngramNormRope nr = {upload(ones, sizeof ones), upload(ones, sizeof ones), 0.0f, upload(table, sizeof table), 8, D, 0, 0};
  EngramHeads hq = {upload(q, sizeof q), HQ * D, D, HQ, ENGRAM_F32}, hk = {upload(k, sizeof k), HK * D, D, HK, ENGRAM_F32};
  EngramHeads hv = {upload(v, sizeof v), HK * D, D, HK, ENGRAM_F32};
  EngramHeads tq = {upload(NULL, sizeof q), HQ * D, D, HQ, ENGRAM_F32}, tk = {upload(NULL, sizeof k), HK * D, D, HK, ENGRAM_F32};
  EngramHeads rk = {upload(NULL, sizeof back), HK * D, D, HK, ENGRAM_F32}, rv = {upload(NULL, sizeof back), HK * D, D, HK, ENGRAM_F32};
  EngramKVCache cache;
  memset(&cache, 0, sizeof cache);
  cache.format = ENGRAM_CACHE_FP8_E8M0;
  cache.kv_heads = HK;
  cache.head_dim = D;
  cache.page_size = PAGE;
  cache.num_pages = PAGES;
  cache.k = upload(NULL, PAGES * HK * PAGE * D);
  cache.v = upload(NULL, PAGES * HK * PAGE * D);
  cache.page_stride = HK * PAGE * D;
  cache.head_stride = PAGE * D;
  cache.token_stride = D;
  cache.k_scales = upload(NULL, PAGES * HK * PAGE * 4);
  cache.v_scales = upload(NULL, PAGES * HK * PAGE * 4);
  cache.scale_page_stride = HK * PAGE * 4;
  cache.scale_head_stride = PAGE * 4;
  cache.scale_token_stride = 4;
  int32_t* err = upload(NULL, 4);
  int32_t* pos = upload(positions, sizeof positions);
  int64_t* sl = upload(slots, sizeof slots);

  CHECK(engram_qk_norm_rope(&nr, T, D, &hq, &hk, pos, &tq, &tk, err, NULL));
  CHECK(engram_kv_write(&cache, T, &tk, &hv, sl, err, NULL));
  CHECK(engram_kv_read(&cache, T, sl, &rk, &rv, err, NULL));
  CHECK(engram_sync_status(err, NULL));
  CHECK(cudaMemcpy(back, rk.data, sizeof back, cudaMemcpyDeviceToHost));
  for (t = 0; t < T; ++t)
    for (i = 0; i < D / 2; ++i) {
      /* (1, 1) turned by the position's angle, then three bits behind the leading one of at most 1.4143 */
      const float a = table[positions[t]][i] - table[positions[t]][D / 2 + i];
      if (fabsf(back[t][0][i] - a) > 0.0625f) {
        printf("token %d value %d: %f, not %f\n", t, i, back[t][0][i], a);
        return 1;
      }
    }
  CHECK(cudaMemcpy(kept, rv.data, sizeof kept, cudaMemcpyDeviceToHost));
  if (memcmp(kept, v, sizeof v) != 0) {
    printf("powers of two are not kept\n");
    return 1;
  }

  /* queries at sequence 0's last token and sequence 1's only one: scale 0 gives the mean of the values */
  EngramPagedSeqs seqs = {2, upload(pages, sizeof pages), 2, 2, upload(lens, sizeof lens)};
  EngramHeads two = {(float*)tq.data + 2 * HQ * D, HQ * D, D, HQ, ENGRAM_F32};
  EngramHeads o = {upload(NULL, sizeof out), HQ * D, D, HQ, ENGRAM_BF16};
  float* dl = upload(NULL, sizeof lse);
  const size_t n = engram_attention_workspace_bytes(&cache, HQ, 2);
  void* ws = upload(NULL, n);
  CHECK(engram_paged_attention(&cache, &seqs, &two, 0.0f, 0, &o, dl, ws, n, err, NULL));
  CHECK(engram_sync_status(err, NULL));
  CHECK(cudaMemcpy(out, o.data, sizeof out, cudaMemcpyDeviceToHost));
  CHECK(cudaMemcpy(lse, dl, sizeof lse, cudaMemcpyDeviceToHost));
  for (h = 0; h < HQ; ++h)
    for (i = 0; i < D; ++i)
      if (fabsf(bf16(out[0][h][i]) - 7.0f / 3.0f) > 0.01f || bf16(out[1][h][i]) != 8.0f || fabsf(lse[0][h] - logf(3.0f)) > 1e-5f ||
          fabsf(lse[1][h]) > 1e-6f) {
        printf("head %d value %d: %f %f, lse %f %f\n", h, i, bf16(out[0][h][i]), bf16(out[1][h][i]), lse[0][h], lse[1][h]);
        return 1;
      }

  /* a page outside the cache is reported */
  seqs.block_table = upload("\x7f\0\0\0\x7f\0\0\0\0\0\0\0\0\0\0", 16);
  CHECK(engram_paged_attention(&cache, &seqs, &two, 0.0f, 0, &o, dl, ws, n, err, NULL));
  if (engram_sync_status(err, NULL) != ENGRAM_EDATA || strstr(engram_last_error(), "page number") == NULL) {
    printf("a bad page is not reported: %s\n", engram_last_error());
    return 1;
  }
  printf("ok\n");
  return 0;
}
