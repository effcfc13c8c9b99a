// fb_attn_cache.h -- arguments of the attention over a paged cache, shared by
// its kernels (fb_attn_cache*.cu) and the entry points (fb_cache_bias.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fb {

// Ranks up to this one are products in fp32 on the CUDA cores; larger ones go
// to the tensor cores as two fp16 parts.
constexpr int kCacheBiasExact = 4;

struct CacheAttnArgs {
  const __nv_bfloat16 *Q;  // [B, Hq, T, d]
  const void *kp, *vp;     // pools [pages, H, page, d]
  const uint8_t *ks, *vs;  // row scales [pages, H, page] (e4m3)
  const int *table, *prefix, *counts, *depths;
  const uint32_t *mask;  // [B, T, mask_words], or null: drafted token u is visible to t >= u
  int mask_words;
  __nv_bfloat16 *O;  // [B, Hq, T, d]
  float *LSE;        // [B, Hq, T]
  float *part;       // partial rows of items that cross CTAs
  unsigned *counters;
  int B, Hq, H, G, T, d, rows, chunks;  // G = Hq / H, rows = G T, chunks of rows per item
  int page_shift, num_pages, max_pages;
  float scale;
  int R, RP;  // bias rank, and the padded rank of its fp16 rows
  // prepared factors: R <= kCacheBiasExact: float4 rows [heads, P]; else rows of RP / 4 groups of (4 hi, 4 lo) fp16
  const void *fq, *fk;
  int P, fq_heads, fk_heads;
  int *flags;
};

// The kernel for few query rows: floats of partial rows that a call can need, and the launch (a cudaError_t).
size_t cache_attn_part_floats(int d, int T, int G, int sms);
cudaError_t launch_attn_cache(CacheAttnArgs a, int e4m3, int sms, cudaStream_t st);

// The kernel for many: the same.
size_t cache_tile_part_floats(int d, int sms);
cudaError_t launch_attn_cache_tile(CacheAttnArgs a, int e4m3, int sms, cudaStream_t st);

}  // namespace fb
