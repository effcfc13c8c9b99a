// fb_attn_cache.cuh -- what the kernels of attention over a paged cache share:
// a sequence's lengths, which keys a row sees, the CTA's run of work, and an
// output row.
#pragma once

#include <cuda_fp8.h>

#include "fb_attn_cache.h"
#include "fb_internal.h"
#include "fb_ptx_cache.cuh"

namespace fb {

constexpr float kCacheLog2e = 1.4426950408889634f;

// 2^e for an integer e, clamped to the normal range.
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(uint32_t(min(max(e, -126), 127) + 127) << 23); }

// Asynchronous copy of 8 bytes to shared memory.
__device__ __forceinline__ void copy8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

struct Seq {
  int prefix, count, len;
};

__device__ __forceinline__ Seq sequence(const CacheAttnArgs &a, int b, bool check) {
  Seq s;
  int p = a.prefix[b], c = a.counts ? a.counts[b] : a.T;
  const long long room = (long long)a.max_pages << a.page_shift;
  bool bad = p < 0 || c < 0 || c > a.T;
  p = max(p, 0);
  c = min(max(c, 0), a.T);
  if ((long long)p + c > room) {  // the table does not reach that far
    bad = true;
    p = int(min((long long)p, room));
    c = int(min((long long)c, room - p));
  }
  if (bad && check) atomicOr(a.flags, kFlagRange);
  s.prefix = p, s.count = c, s.len = c > 0 ? p + c : 0;
  return s;
}

__device__ __forceinline__ bool drafted_visible(const CacheAttnArgs &a, int b, int t, int u) {
  if (!a.mask) return u <= t;
  return (a.mask[((long long)b * a.T + t) * a.mask_words + (u >> 5)] >> (u & 31)) & 1u;
}

// Position of new token u of sequence b in the factor tables.
__device__ __forceinline__ int new_position(const CacheAttnArgs &a, int b, const Seq &s, int u) {
  const long long p = (long long)s.prefix + (a.depths ? a.depths[(long long)b * a.T + u] : u);
  if (p < 0 || p >= a.P) {
    atomicOr(a.flags, kFlagRange);
    return p < 0 ? 0 : a.P - 1;
  }
  return int(p);
}

// A word of value codes without its non-finite values.
template <bool E4M3>
__device__ __forceinline__ uint32_t even_word(uint32_t w) {
  if constexpr (E4M3) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
      if (((w >> i) & 0x7fu) == 0x7fu) w &= ~(0xffu << i);
  } else {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  }
  return w;
}
// One of them, or 0: value `at` of a row. AS_BF16: an 8-bit value left the products as bf16, times its row's scale, and may
// lie beyond that type's range.
template <bool E4M3, bool AS_BF16>
__device__ __forceinline__ float odd_value(const uint8_t *row, int at, uint32_t scale) {
  if constexpr (E4M3 && AS_BF16) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(row[at], __NV_E4M3);
    const float v = __bfloat162float(__float2bfloat16_rn(__low2float(__half2(r)) * scale_value(scale)));
    return fabsf(v) < INFINITY ? 0.f : v;
  } else if constexpr (E4M3) {
    return (row[at] & 0x7fu) == 0x7fu ? __uint_as_float(0x7fffffffu) : 0.f;
  } else {
    const uint32_t v = reinterpret_cast<const uint16_t *>(row)[at];
    return (v & 0x7f80u) == 0x7f80u ? __uint_as_float(v << 16) : 0.f;
  }
}

// The non-finite values at d = dd of the keys j0 .. j1 - 1 that token t sees.
template <bool E4M3, bool AS_BF16>
__device__ __forceinline__ float odd_sum(const CacheAttnArgs &a, const Seq &s, int b, int h, int t, int dd, int j0, int j1) {
  float sum = 0.f;
  for (int j = j0; j < j1; ++j) {
    const int page = a.table[(long long)b * a.max_pages + (j >> a.page_shift)], u = j - s.prefix;
    if (page < 0 || page >= a.num_pages || !(u < 0 || drafted_visible(a, b, t, u))) continue;
    const long long row = (((long long)page * a.H + h) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
    const uint32_t scale = E4M3 ? a.vs[row] : 0u;
    if (E4M3 && scale == 255u) return __uint_as_float(0x7fffffffu);
    sum += odd_value<E4M3, AS_BF16>(static_cast<const uint8_t *>(a.vp) + row * a.d * (E4M3 ? 1 : 2), dd, scale);
  }
  return sum;
}

// Whether a part of a row has seen no key. A maximum of -inf alone does not say so: it passes over NaN, which the sum keeps.
__device__ __forceinline__ bool saw_none(float top, float sum) { return top == -INFINITY && sum == 0.f; }

// Value dd of one output row, from the sums relative to exp(top); row t of a sequence that brings fewer tokens is 0.
__device__ __forceinline__ void write_row(const CacheAttnArgs &a, const Seq &s, long long row, int t, int dd, float top,
                                          float sum, float val) {
  const bool none = t >= s.count || saw_none(top, sum);
  if (dd < a.d) a.O[row * a.d + dd] = __float2bfloat16_rn(none ? 0.f : val / sum);
  if (dd == 0) a.LSE[row] = none ? -INFINITY : top + logf(sum);
}

// One CTA's part of an item (a sequence's rows of one key/value head): blocks k0 .. k1 - 1 of its `blocks`.
struct Segment {
  Seq s;
  int b, item, blocks, k0, k1;
  long long start;  // the number of the item's first block
};

// All blocks of keys of all items, numbered sequence by sequence and item by item, are dealt out in equal runs: CTA c
// of `ctas` takes first(c) .. first(c + 1) - 1. Built and walked by whole warps. Before an item's blocks `extra` numbers
// stand for what an item costs beside them, so that CTAs with more items get fewer blocks.
struct Walk {
  long long total, ctas, pos, hi, bstart;
  int b, keys, extra, per_seq;

  __device__ __forceinline__ int blocks_of(const Seq &s) const { return max(1, int(((long long)s.len + keys - 1) / keys)); }
  __device__ __forceinline__ int numbers_of(const Seq &s) const { return blocks_of(s) + extra; }
  __device__ __forceinline__ long long first(long long c) const { return c * total / ctas; }

  __device__ __forceinline__ Walk(const CacheAttnArgs &a, int block_keys, int item_extra, int lane) {
    keys = block_keys, extra = item_extra;
    per_seq = a.H * a.chunks;
    total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32)
      total += __reduce_add_sync(0xffffffffu, b0 + lane < a.B ? numbers_of(sequence(a, b0 + lane, false)) : 0);
    total *= per_seq;
    ctas = min((long long)gridDim.x, total);
    pos = hi = 0;
    b = 0;
    bstart = 0;
    if (blockIdx.x >= ctas) return;
    pos = first(blockIdx.x), hi = first(blockIdx.x + 1);
    for (int b0 = 0; b0 < a.B; b0 += 32) {  // the sequence that block `pos` is in
      const int mine = b0 + lane < a.B ? numbers_of(sequence(a, b0 + lane, false)) : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned vote = __ballot_sync(0xffffffffu, b0 + lane >= a.B || bstart + (long long)incl * per_seq > pos);
      if (vote) {
        const int f = __ffs(vote) - 1;
        b = b0 + f;
        bstart += (long long)(__shfl_sync(0xffffffffu, incl, f) - __shfl_sync(0xffffffffu, mine, f)) * per_seq;
        break;
      }
      bstart += (long long)__shfl_sync(0xffffffffu, incl, 31) * per_seq;
    }
  }

  __device__ __forceinline__ bool next(const CacheAttnArgs &a, Segment &g) {
    while (pos < hi && b < a.B) {
      g.s = sequence(a, b, true);
      const int n = numbers_of(g.s);
      if (pos >= bstart + (long long)n * per_seq) {
        bstart += (long long)n * per_seq;
        ++b;
        continue;
      }
      g.b = b;
      g.blocks = n - extra;
      g.item = int((pos - bstart) / n);
      const long long start = bstart + (long long)g.item * n;
      const int n0 = int(pos - start), n1 = int(min((long long)n, n0 + (hi - pos)));
      pos += n1 - n0;
      if (n1 <= extra) continue;  // the item's blocks begin in the next run
      g.start = start + extra;
      g.k0 = max(n0 - extra, 0);
      g.k1 = n1 - extra;
      return true;
    }
    return false;
  }

  // The CTA whose run holds block x.
  __device__ __forceinline__ int owner(long long x) const {
    long long c = x * ctas / total;
    while (c + 1 < ctas && first(c + 1) <= x) ++c;
    while (c > 0 && first(c) > x) --c;
    return int(c);
  }
};

}  // namespace fb
