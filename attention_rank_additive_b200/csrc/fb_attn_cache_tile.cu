// fb_attn_cache_tile.cu -- attention of many query rows (drafted trees, grouped
// heads) over a paged cache on the tcgen05 tensor cores. The mathematics, the
// masks and the work split are those of fb_attn_cache.cu; here the matrix
// products bound the time, so they run as tiles of 128 rows by 96 keys.
//
// A CTA (one per SM) holds one or two tiles of 128 query rows of an item and
// walks over its run of 96-key tiles (two of K, V and factors fit beside the queries
// at the largest head dim and ranks up to 32; of 128 keys only one K would):
//   warp 0          MMA issuer: S = Q K^T (+ phi_q phi_k^T), O += P V
//   warps 1-3, 4-7  V and K loader: codes or bf16 from the pages to swizzled bf16
//                   tiles; the K loader also the factors and the query tiles
//   warps 8-11, 12-15  softmax of stream 0 and 1: a thread per row (TMEM lane)
// Stream t is row tile t (both walk over the same keys), or, when an item has
// 128 rows or fewer, every second key tile of the one row tile: the streams
// then end with a maximum, sum and O each and are joined like two CTAs' parts.
// Either way the tensor cores work on one stream while the softmax of the other
// runs: S_0(i), PV_1(i-1), S_1(i), PV_0(i). P overwrites the first half of S.
//
// 8-bit rows become bf16 in the loaders, exactly from 2^-126 on: a code's 3 bits of
// mantissa fit, and its exponent with the row's power of two as well, so scores and
// values need no further scaling. (Beyond bf16's range a value is infinite.)
//
// The roles run side by side out of one instruction cache, which decides more than
// the instructions do: loops stay rolled, K and V share the loaders' loop, and
// what is rare is out of line. Measured, 16 trees of 61 tokens on contexts up to
// 8131, 32 query and 8 key/value heads of 128, rank 32, 8-bit cache: 190 us, 432
// TFLOP/s (972 us with everything unrolled). Of a CTA's 330 thousand clocks the
// tensor cores work 150, the issuer waits 95 for a softmax and the joins of
// items that cross CTAs take 10 to 30. Tiles of 64 keys with two score buffers a
// stream, so that no softmax waits for its product, took 205 us: a product of 64
// keys takes as long as one of 96, and the loaders set the pace.
//
// The bias joins S in the same accumulator: phi_q / scale, split into fp16 parts
// again, times the keys' prepared parts (three products). Ranks up to 4 are fp32
// multiply-adds in the softmax.
#include <cuda_fp8.h>

#include <algorithm>

#include "fb_attn_cache.cuh"

namespace fb {
namespace {

constexpr int kThreads = 16 * 32;  // four warps a scheduler: 128 registers a thread
constexpr int kVThreads = 96;
constexpr int kIssuer = 0, kVWarp = 1, kKWarp = 4, kSoftmaxWarp = 8;
constexpr int kTileKeys = 96, kGroups = kTileKeys / 16;
constexpr int kItemExtra = 3;  // what the queries' loads and the parts' joins of an item cost, in tiles (found on grouped trees)
constexpr float kRaise = 8.f;  // log2 units: O is rescaled when the maximum grows by more

struct TilePlan {
  int tiles;  // row tiles of an item's chunk: 1 or 2
  int split;  // one row tile, its key tiles dealt to two streams
  int ks;     // slots of K and its factors: 1 or 2 (V has two)
  int rpb;    // bias: columns reserved for the hi and for the lo parts (32, 64, 128), or 0
  uint32_t q, fq, k, fk, v, planes, ctrl;  // shared memory offsets from the 1024-byte aligned base
  uint32_t smem;
};

struct Ctrl {
  uint64_t q_full;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_final[2];
  uint64_t drain;
  unsigned alive[4];              // [tile & 3]: bit i: 16-key group i has a page
  int odd[8];                     // [tile & 7]: tile number + 1 where a non-finite value left the products
  uint32_t tmem;
  int abort, last[2][2];
};

// 16-byte chunk `ch` of row `row` in a tile of 128-byte rows, swizzled; columns past 64 go to the next block of ROWS rows.
template <int ROWS>
__device__ __forceinline__ uint32_t tile_at(int row, int ch) {
  return uint32_t(ch >> 3) * (ROWS * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
}
// Low word of the matrix descriptor of a K-major tile, and of V, at shared memory address `at`; the start address is its
// lowest field, so that a step is added to it. The high word is a constant.
__device__ __forceinline__ uint32_t low_k(uint32_t at) { return (at >> 4) | (16u >> 4) << 16; }
__device__ __forceinline__ uint32_t low_v(uint32_t at) { return (at >> 4) | uint32_t(kTileKeys * 128 >> 4) << 16; }
__device__ __forceinline__ uint64_t desc(uint32_t low) {
  constexpr uint32_t high = (1024u >> 4) | (1u << 14) | (swizzle_code(128) << 29);
  return (uint64_t(high) << 32) | low;
}
// Start-address offsets (16-byte units) of 16-column step kk of a K-major tile of ROWS rows, and of 16-key step kk of V.
template <int ROWS>
__device__ __forceinline__ uint32_t step_k(int kk) {
  return uint32_t((kk >> 2) * (ROWS * 128) + (kk & 3) * 32) >> 4;
}
__device__ __forceinline__ uint32_t step_v(int kk) { return uint32_t(kk * 16 * 128) >> 4; }

// Visibility of keys j0 .. j0 + 31 to new token t, a bit each (t < 0: none past the context).
__device__ __noinline__ uint32_t sees(const CacheAttnArgs &a, int prefix, int count, int b, int t, int j0) {
  auto word = [&](int w) -> uint32_t {  // new tokens 32 w .. 32 w + 31
    if (t < 0 || w * 32 >= count) return 0u;
    uint32_t m;
    if (a.mask)
      m = a.mask[((long long)b * a.T + t) * a.mask_words + w];
    else
      m = t >= w * 32 + 31 ? 0xffffffffu : (t < w * 32 ? 0u : (2u << (t - w * 32)) - 1u);
    const int n = count - w * 32;
    return n >= 32 ? m : m & ((1u << n) - 1u);
  };
  const int u0 = j0 - prefix;
  if (u0 <= -32) return 0xffffffffu;
  if (u0 < 0) return ((1u << -u0) - 1u) | (word(0) << -u0);
  return __funnelshift_r(word(u0 >> 5), u0 & 31 ? word((u0 >> 5) + 1) : 0u, u0 & 31);
}

// The non-finite values at d = dd that left the products of the key tiles k, k + stride, ... below k1 (those that reach
// past the context), of the keys that token t sees.
template <bool E4M3>
__device__ __noinline__ float odd_sum_of(const CacheAttnArgs &a, Seq s, int b, int h, int t, int dd, int k, int k1, int stride) {
  const int first = s.prefix / kTileKeys;
  if (k < first) k += (first - k + stride - 1) / stride * stride;
  float sum = 0.f;
  for (; k < k1; k += stride)
    sum += odd_sum<E4M3, true>(a, s, b, h, t, dd, k * kTileKeys, min(s.len, (k + 1) * kTileKeys));
  return sum;
}

// Two e4m3 codes (half `hi` of w) times a scale, as bf16; NaN codes stay NaN.
__device__ __forceinline__ uint32_t e4m3_to_bf16(uint32_t w, bool hi, float scale) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(hi ? w >> 16 : w & 0xffffu), __NV_E4M3);
  const float2 f = __half22float2(__half2(r));
  return pack_bf16x2(f.x * scale, f.y * scale);
}

__device__ __forceinline__ void sts16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  st_shared_v4(at, a, b, c, d);
}

// The pages of a segment's key tiles, for a loader warp: lane i (< kGroups) holds the page of 16-key group i, fetched
// a tile ahead, so that no load of a row waits for its page number.
struct Pages {
  int now, next;
  __device__ __forceinline__ int fetch(const CacheAttnArgs &a, int b, int j, int len, int lane) const {
    j += 16 * lane;
    return lane < kGroups && j < len ? __ldg(a.table + (long long)b * a.max_pages + (j >> a.page_shift)) : 0;
  }
  // Bit i: group i of the present tile has a page or lies behind the last key.
  __device__ __forceinline__ unsigned alive(const CacheAttnArgs &a) const {
    return __ballot_sync(0xffffffffu, now >= 0 && now < a.num_pages) & ((1u << kGroups) - 1u);
  }
};
// Pool row of the tile's row `row`, given the lanes' pages (one outside the pool counts as page 0: it is cleared).
__device__ __forceinline__ long long pool_row(const CacheAttnArgs &a, int pages, int h, int j, int row) {
  const int page = __shfl_sync(0xffffffffu, pages >= 0 && pages < a.num_pages ? pages : 0, row >> 4);
  return (((long long)page * a.H + h) << a.page_shift) + ((j + row) & ((1 << a.page_shift) - 1));
}

struct Chunks {
  uint4 x, y;
};
// The chunks without their non-finite values; `odd` where there were any.
__device__ __noinline__ Chunks clear_odd(Chunks c, int *odd, int stamp) {
  uint32_t w[8] = {c.x.x, c.x.y, c.x.z, c.x.w, c.y.x, c.y.y, c.y.z, c.y.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t even = even_word<false>(w[k]);
    if (even != w[k]) *odd = stamp;
    w[k] = even;
  }
  c.x = make_uint4(w[0], w[1], w[2], w[3]), c.y = make_uint4(w[4], w[5], w[6], w[7]);
  return c;
}

__device__ __noinline__ void wait_long(uint64_t *bar, uint32_t parity, volatile int *abort) {
  mbar_wait(bar, parity, abort);
}
__device__ __forceinline__ void wait_for(uint64_t *bar, uint32_t parity, volatile int *abort) {
  if (!mbar_try_wait(bar, parity)) wait_long(bar, parity, abort);
}

template <int DP, bool E4M3, int BIAS>
__global__ void __launch_bounds__(kThreads, 1) attn_cache_tile_kernel(const __grid_constant__ CacheAttnArgs a, const TilePlan p) {
  constexpr int ES = E4M3 ? 1 : 2;
  constexpr int CPR = DP * ES / 16;  // 16-byte chunks of a pool row (padded); also the chunks of a tile per loader thread
  constexpr uint32_t kTile = kTileKeys * DP * 2, kQTile = 128 * DP * 2;
  extern __shared__ __align__(16) uint8_t smem_dyn[];
  uint8_t *sm = smem_dyn + ((1024u - (smem_u32(smem_dyn) & 1023u)) & 1023u);
  Ctrl &c = *reinterpret_cast<Ctrl *>(sm + p.ctrl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(sm);
  // [tile & 3][rank][key]: the keys' factors, ranks up to 4
  float(*planes)[4][kTileKeys] = reinterpret_cast<float(*)[4][kTileKeys]>(sm + p.planes);
  const uint32_t fq_tile = 128 * 4 * p.rpb, fk_tile = kTileKeys * 4 * p.rpb;

  if (threadIdx.x == 0) {
    mbar_init(&c.q_full, 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.k_full[i], 128), mbar_init(&c.v_full[i], kVThreads);
      mbar_init(&c.k_empty[i], 1), mbar_init(&c.v_empty[i], 1);
      mbar_init(&c.s_full[i], 1), mbar_init(&c.p_full[i], 128), mbar_init(&c.o_final[i], 1);
    }
    mbar_init(&c.drain, 1);
    for (int i = 0; i < 8; ++i) c.odd[i] = 0;
    c.abort = 0;
    fence_mbar_init();
  }
  if (warp == kIssuer) tmem_alloc(&c.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  volatile int *abort = &c.abort;
  griddep_wait();

  // A wait that runs out marks the CTA: every role then runs on through its loops without waiting (all addresses stay
  // in bounds, the result is garbage) and the call is flagged.
  Walk walk(a, kTileKeys, kItemExtra, lane);
  Segment g;
  const int nstreams = p.split || p.tiles == 2 ? 2 : 1;
  // what a segment's streams do: stream t takes steps of key tiles first + t, first + t + 2, ... (split) or all
  auto steps_of = [&](int t, int n, int rows) {
    if (p.split) return (n + 1 - t) >> 1;
    return t == 0 || rows > 128 ? n : 0;
  };

  if (blockIdx.x >= walk.ctas) {
    // no work: only the teardown below
  } else if (warp >= kSoftmaxWarp) {
    // ------------------------------------------------------------- softmax
    const int t = (warp - kSoftmaxWarp) >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + 128u * t, o_tm = tmem + lane_base + 256u + 128u * t;
    const float unit = BIAS == 1 ? kCacheLog2e : a.scale * kCacheLog2e;  // of the maximum, in log2
    unsigned done = 0;  // key tiles of the segments before
    uint32_t sphase = 0, ophase = 0;
    int seg = 0;
    constexpr int kSlot = 256 * (DP + 2);
    for (; walk.next(a, g); ++seg) {
      const Seq &s = g.s;
      const int n = g.k1 - g.k0, h = g.item / a.chunks, chunk0 = (g.item - h * a.chunks) * p.tiles * 128;
      const int rows = min(p.tiles * 128, a.rows - chunk0);
      const int r = (p.split ? 0 : t * 128) + row;  // row of the chunk
      const bool have = r < rows;
      const long long qrow = ((long long)g.b * a.Hq + (long long)h * a.G) * a.T + chunk0 + (have ? r : 0);
      const int tok_all = have ? (chunk0 + r) % a.T : 0;
      const int tok = have && tok_all < s.count ? tok_all : -1;
      const int steps = t < nstreams ? steps_of(t, n, rows) : 0;
      // A stream without steps would let the other one run any number of tiles ahead of a warp that has yet to read the
      // last segment's marks (odd, last).
      if (!p.split && steps_of(1, n, rows) == 0) named_bar_sync(1, 256);
      float fq[4] = {0.f, 0.f, 0.f, 0.f};
      if (BIAS == 1 && tok >= 0) {
        const int hq = a.fq_heads > 1 ? h * a.G + (chunk0 + r) / a.T : 0;
        const float4 f = __ldg(static_cast<const float4 *>(a.fq) + (long long)hq * a.P + new_position(a, g.b, s, tok));
        fq[0] = f.x, fq[1] = f.y, fq[2] = f.z, fq[3] = f.w;
      }
      const bool busy = __any_sync(0xffffffffu, tok >= 0);  // rows of this warp that want a result
      float m = -INFINITY, l = 0.f;
      int odd = 0;
      for (int i = 0; i < steps; ++i) {
        const int idx = p.split ? 2 * i + t : i;
        const int j0 = (g.k0 + idx) * kTileKeys;
        const unsigned tile = done + unsigned(idx);
        wait_for(&c.s_full[t], sphase & 1u, abort);
        ++sphase;
        tc_fence_after();
        if (i > 0 && c.odd[(tile - (p.split ? 2 : 1)) & 7] == int(tile - (p.split ? 2 : 1)) + 1) odd = 1;
        if (busy) {
          const unsigned alive = c.alive[tile & 3];
          const bool tail = j0 + kTileKeys > s.prefix || alive != (1u << kGroups) - 1u;
          // which keys this row sees, found before its scores take the registers
          constexpr int kParts = kTileKeys / 32;
          uint32_t see[kParts];
          if (__builtin_expect(tail, 0)) {
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
              see[q] = sees(a, s.prefix, s.count, g.b, tok, j0 + 32 * q);
              if (!((alive >> (2 * q)) & 1u)) see[q] &= 0xffff0000u;
              if (!((alive >> (2 * q + 1)) & 1u)) see[q] &= 0x0000ffffu;
            }
          }
          // the scores of columns 32 q .. 32 q + 31: biased (rank <= 4), masked
          auto finish = [&](int q, uint32_t *x) {
            if constexpr (BIAS == 1) {
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int rr = 0; rr < 4; ++rr)
                  if (rr < a.R) {
                    const float4 f = *reinterpret_cast<const float4 *>(&planes[tile & 3][rr][32 * q + k]);
                    y[0] = fmaf(f.x, fq[rr], y[0]), y[1] = fmaf(f.y, fq[rr], y[1]);
                    y[2] = fmaf(f.z, fq[rr], y[2]), y[3] = fmaf(f.w, fq[rr], y[3]);
                  }
#pragma unroll
                for (int e = 0; e < 4; ++e) x[k + e] = __float_as_uint(fmaf(__uint_as_float(x[k + e]), a.scale, y[e]));
              }
            }
            if (__builtin_expect(tail, 0)) {
              const uint32_t mine = q == 0 ? see[0] : (q == 1 ? see[1] : see[2]);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!((mine >> k) & 1u)) x[k] = 0xff800000u;
            }
          };
          // Two passes over S in rolled loops of 32 columns. (One pass, with all scores or all of P in registers, reads S
          // once but needs a copy of the loop's body per 32 columns: 300 to 350 us for grouped trees.)
          float top = -INFINITY;
#pragma unroll 1
          for (int q = 0; q < kParts; ++q) {
            uint32_t x[32];
            tmem_ld32(s_tm + 32u * q, x);
            tmem_ld_wait32(x);
            finish(q, x);
#pragma unroll
            for (int k = 0; k < 32; k += 2) top = fmax3(top, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
          }
          const bool raise = (top - m) * unit > kRaise;  // the first finite score too: m is -inf
          if (__any_sync(0xffffffffu, raise)) {
            const float alpha = raise ? ex2_approx((m - top) * unit) : 1.f;
            if (raise) m = top;
            l *= alpha;
            if (i > 0) {
#pragma unroll 1
              for (int q = 0; q < DP / 16; ++q) {
                uint32_t y[16];
                tmem_ld16(o_tm + 16u * q, y);
                tmem_ld_wait16(y);
#pragma unroll
                for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * alpha);
                tmem_st16(o_tm + 16u * q, y);
              }
            }
          }
          const float mu = m == -INFINITY ? 0.f : m, shift = -mu * unit;
          const uint64_t unit2 = f2_pack(unit, unit), shift2 = f2_pack(shift, shift), mu2 = f2_pack(mu, mu);
          uint64_t acc = 0;
#pragma unroll 1
          for (int q = 0; q < kParts; ++q) {
            uint32_t x[32], w[16];
            tmem_ld32(s_tm + 32u * q, x);
            tmem_ld_wait32(x);
            finish(q, x);
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const uint64_t x2 = f2_pack(__uint_as_float(x[k]), __uint_as_float(x[k + 1]));
              // rank <= 4: the difference first, which holds at scores of the type's lowest value too
              const uint64_t y2 = BIAS == 1 ? f2_fma(f2_sub(x2, mu2), unit2, 0) : f2_fma(x2, unit2, shift2);
              float y0, y1;
              f2_unpack(y2, y0, y1);
              const float e0 = ex2_approx(y0), e1 = ex2_approx(y1);
              acc = f2_add(acc, f2_pack(e0, e1));
              w[k / 2] = pack_bf16x2(e0, e1);
            }
            tmem_st16(s_tm + 16u * q, w);
          }
          float a0, a1;
          f2_unpack(acc, a0, a1);
          l += a0 + a1;
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(&c.p_full[t]);
      }
      // ---- the segment's end
      if (steps > 0) {
        wait_for(&c.o_final[t], ophase & 1u, abort);
        ++ophase;
        tc_fence_after();
        const unsigned tile = done + unsigned(p.split ? 2 * (steps - 1) + t : steps - 1);
        if (c.odd[tile & 7] == int(tile) + 1) odd = 1;
      }
      done += n;
      float nat = BIAS == 1 || m == -INFINITY ? m : m * a.scale;  // the maximum in natural units
      const bool whole = g.k0 == 0 && g.k1 == g.blocks;
      float *mine = a.part + (2ll * blockIdx.x + (g.k0 == 0)) * kSlot;
      if (!busy) nat = -INFINITY, l = 0.f;
      // Parts (O, maximum, sum) of an item that crosses CTAs, and of the two streams of a split (rows 128 and up for
      // stream 1), go to this CTA's slots; the item's last CTA joins them in order. Non-finite values that left a stream's
      // products come back into its own part: another may have seen no key of the row, or weigh nothing beside it.
      const int at = p.split ? t * 128 + row : r;
      const bool real = steps > 0 && busy;  // uniform over the warp; other parts have a maximum of -inf and no O
      // columns 16 q .. 16 q + 15 of this row's O
      auto own = [&](int q, float *x) {
        uint32_t w[16];
        tmem_ld16(o_tm + 16u * q, w);
        tmem_ld_wait16(w);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(w[k]);
        if (__builtin_expect(odd && tok >= 0, 0)) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (16 * q + k < a.d) x[k] += odd_sum_of<E4M3>(a, s, g.b, h, tok, 16 * q + k, g.k0 + (p.split ? t : 0), g.k1,
                                                           p.split ? 2 : 1);
        }
      };
      auto write_part = [&]() {
        mine[DP * 256 + at] = nat, mine[(DP + 1) * 256 + at] = l;
        if (!real) return;
#pragma unroll 1
        for (int q = 0; q < DP / 16; ++q) {
          float x[16];
          own(q, x);
#pragma unroll
          for (int k = 0; k < 16; ++k) mine[(16 * q + k) * 256 + at] = x[k];
        }
      };
      // 16 columns of an output row
      auto store = [&](long long out_row, int k, const float *y) {
        uint4 *o = reinterpret_cast<uint4 *>(a.O + out_row * a.d + k);
#pragma unroll
        for (int e = 0; e < 16; e += 8)
          if (k + e < a.d)
            o[e / 8] = make_uint4(pack_bf16x2(y[e], y[e + 1]), pack_bf16x2(y[e + 2], y[e + 3]),
                                  pack_bf16x2(y[e + 4], y[e + 5]), pack_bf16x2(y[e + 6], y[e + 7]));
      };
      int c0 = blockIdx.x, c1 = blockIdx.x;
      bool last = true;
      if (!whole) c0 = walk.owner(g.start), c1 = walk.owner(g.start + g.blocks - 1);
      if (!p.split) {
        // Row tiles: a thread joins its row, with this CTA's part out of TMEM. A CTA that finds all others done does not
        // write its part at all: CTAs end together, and writing and reading all parts then took 15 us of 200.
        if (!whole) {
          const bool leader = threadIdx.x == kSoftmaxWarp * 32;
          int *flag = c.last[seg & 1];
          if (leader) flag[0] = atomicAdd(a.counters + c0, 0u) == unsigned(c1 - c0);
          named_bar_sync(1, 256);
          last = flag[0];
          if (!last) {
            write_part();
            __threadfence();
            named_bar_sync(1, 256);
            if (leader) flag[1] = atomicAdd(a.counters + c0, 1u) == unsigned(c1 - c0);
            named_bar_sync(1, 256);
            last = flag[1];
          }
          if (last) {
            __threadfence();
            if (leader) a.counters[c0] = 0u;  // for the next call
          }
        }
        if (last) {
          auto part = [&](int cc) { return a.part + (2ll * cc + (cc == c0)) * kSlot + r; };
          float top = -INFINITY, sum = 0.f;
#pragma unroll 4
          for (int cc = c0; cc <= c1; ++cc) {
            const bool here = cc == int(blockIdx.x);
            const float mc = here ? nat : __ldcg(part(cc) + DP * 256), lc = here ? l : __ldcg(part(cc) + (DP + 1) * 256);
            const float mn = fmaxf(top, mc), z = mn == -INFINITY ? 0.f : mn;
            sum = sum * ex2_approx((top - z) * kCacheLog2e) + lc * ex2_approx((mc - z) * kCacheLog2e);
            top = mn;
          }
          const bool none = tok < 0 || saw_none(top, sum);
          const float inv = none ? 0.f : 1.f / sum, z = top == -INFINITY ? 0.f : top;
          if (have) a.LSE[qrow] = none ? -INFINITY : top + logf(sum);
#pragma unroll 1
          for (int q = 0; q < DP / 16; ++q) {
            float x[16], y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = y[e] = 0.f;
            if (real) own(q, x);
            if (!none) {
#pragma unroll 2
              for (int cc = c0; cc <= c1; ++cc) {
                const bool here = cc == int(blockIdx.x);
                const float *from = part(cc);
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = here ? x[e] : __ldcg(from + (16 * q + e) * 256);
                const float mc = here ? nat : __ldcg(from + DP * 256), lc = here ? l : __ldcg(from + (DP + 1) * 256);
                const bool seen = !saw_none(mc, lc);  // else its O was not written
                const float f = ex2_approx((mc - z) * kCacheLog2e) * inv;
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = seen ? fmaf(v[e], f, y[e]) : y[e];
              }
            }
            if (have) store(qrow, 16 * q, y);
          }
        }
      } else {
        write_part();
        __threadfence();
        named_bar_sync(1, 256);
        if (!whole) {
          if (threadIdx.x == kSoftmaxWarp * 32) {
            c.last[0][0] = atomicAdd(a.counters + c0, 1u) == unsigned(c1 - c0);
            if (c.last[0][0]) a.counters[c0] = 0u;  // for the next call
          }
          named_bar_sync(1, 256);
          last = c.last[0][0];
          if (last) __threadfence();
        }
        if (last) {
          // Part i: CTA c0 + i / 2, stream i % 2. A warp takes 32 rows by 16 columns at a time: with few rows all warps have
          // some.
          const int parts = (c1 - c0 + 1) * 2, row_blocks = (rows + 31) >> 5;
          const long long row0 = ((long long)g.b * a.Hq + (long long)h * a.G) * a.T + chunk0;
#pragma unroll 1
          for (int task = warp - kSoftmaxWarp; task < row_blocks * (DP / 16); task += 8) {
            const int k = task / row_blocks * 16, rr = task % row_blocks * 32 + lane;
            if (rr >= rows) continue;
            float top = -INFINITY, sum = 0.f, y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = 0.f;
#pragma unroll 2
            for (int i = 0; i < parts; ++i) {
              const int cc = c0 + (i >> 1);
              const float *x = a.part + (2ll * cc + (cc == c0)) * kSlot + (i & 1) * 128 + rr;
              const float mc = __ldcg(x + DP * 256), lc = __ldcg(x + (DP + 1) * 256);
              float v[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __ldcg(x + (k + e) * 256);
              const bool seen = !saw_none(mc, lc);
              const float mn = fmaxf(top, mc), z = mn == -INFINITY ? 0.f : mn;
              const float f0 = ex2_approx((top - z) * kCacheLog2e), f1 = ex2_approx((mc - z) * kCacheLog2e);
              sum = sum * f0 + lc * f1;
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = fmaf(seen ? v[e] : 0.f, f1, y[e] * f0);
              top = mn;
            }
            const bool none = (chunk0 + rr) % a.T >= s.count || saw_none(top, sum);
            if (k == 0) a.LSE[row0 + rr] = none ? -INFINITY : top + logf(sum);
            const float inv = none ? 0.f : 1.f / sum;
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = none ? 0.f : y[e] * inv;
            store(row0 + rr, k, y);
          }
        }
        named_bar_sync(1, 256);  // the slot's parts have been read
      }
    }
  } else if (warp != kIssuer) {
    // ------------------------------------------------------------- loaders
    const bool is_v = warp < kKWarp;
    const int l = is_v ? threadIdx.x - kVWarp * 32 : threadIdx.x - kKWarp * 32, threads = is_v ? kVThreads : 128;
    const uint8_t *pool = static_cast<const uint8_t *>(is_v ? a.vp : a.kp), *scales = is_v ? a.vs : a.ks;
    const int slots = is_v ? 2 : p.ks;
    const uint32_t dst0 = base + (is_v ? p.v : p.k);
    uint64_t *full = is_v ? c.v_full : c.k_full, *empty = is_v ? c.v_empty : c.k_empty;
    // This thread's chunks, 16 bytes of a pool row each, which become one (bf16) or two (e4m3) of the tile's: at ch of
    // rows row0, row0 + stride, ... A chunk's registers take the next tile's load as soon as it is stored.
    const int ch = threadIdx.x % CPR, row0 = l / CPR, stride = threads / CPR, mine = kTileKeys / stride;
    static_assert(kTileKeys * CPR / kVThreads == CPR, "chunks of a V loader thread; a K loader thread has fewer");
    const int rb = a.d * ES;  // bytes of a pool row
    const bool inside = ch * 16 < rb;
    const int at = inside ? ch * 16 : 0;
    unsigned tile = 0;
    Pages pages;
    while (walk.next(a, g)) {
      const Seq &s = g.s;
      const int h = g.item / a.chunks;
      pages.now = pages.fetch(a, g.b, g.k0 * kTileKeys, s.len, lane);
      pages.next = pages.fetch(a, g.b, (g.k0 + 1) * kTileKeys, s.len, lane);
      uint4 raw[CPR];
      uint32_t sc[E4M3 ? CPR : 1];
      auto load = [&](int i, int pg, int j) {  // rows behind the last key read what lies there and are cleared below
        const long long pr = pool_row(a, pg, h, j, row0 + i * stride);
        raw[i] = __ldg(reinterpret_cast<const uint4 *>(pool + pr * rb + at));
        if (E4M3) sc[E4M3 ? i : 0] = __ldg(scales + pr);
      };
#pragma unroll
      for (int i = 0; i < CPR; ++i)
        if (i < mine) load(i, pages.now, g.k0 * kTileKeys);
      if (!is_v) {
        // ---- the query tiles, a thread per row, and their factors; their last readers are the S of all tiles so far
        for (unsigned n = 1; n <= unsigned(slots) && n <= tile; ++n)
          wait_for(&empty[(tile - n) % slots], ((tile - n) / slots) & 1u, abort);
        const int chunk0 = (g.item - h * a.chunks) * p.tiles * 128, rows = min(p.tiles * 128, a.rows - chunk0);
        const float inv = 1.f / a.scale;
#pragma unroll 1
        for (int t = 0; t < p.tiles; ++t) {
          const int r = t * 128 + l, tok_all = (chunk0 + r) % a.T;
          const bool have = r < rows;
          const uint32_t qt = base + p.q + t * kQTile;
          const uint4 *q = reinterpret_cast<const uint4 *>(
              a.Q + (((long long)g.b * a.Hq + (long long)h * a.G) * a.T + chunk0 + (have ? r : 0)) * a.d);
          constexpr int kLoads = DP == 128 && !E4M3 ? 8 : DP / 8;  // in flight, beside the registers of the first rows of K
#pragma unroll 1
          for (int c0 = 0; c0 < DP / 8; c0 += kLoads) {
            uint4 v[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
              v[i] = make_uint4(0u, 0u, 0u, 0u);
              if (have && (c0 + i) * 8 < a.d) v[i] = __ldg(q + c0 + i);
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i) sts16(qt + tile_at<128>(l, c0 + i), v[i].x, v[i].y, v[i].z, v[i].w);
          }
          if constexpr (BIAS == 2) {
            const uint32_t ft = base + p.fq + t * fq_tile;
            const bool real = have && tok_all < s.count;
            const int hq = a.fq_heads > 1 && have ? h * a.G + (chunk0 + r) / a.T : 0;
            const uint4 *f = static_cast<const uint4 *>(a.fq) +
                             ((long long)hq * a.P + (real ? new_position(a, g.b, s, tok_all) : 0)) * (a.RP / 4);
            bool over = false;
#pragma unroll 1
            for (int i = 0; i < a.RP / 8; i += 2) {  // sixteen ranks; eight are 16 bytes of hi and 16 of lo
              uint4 u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) u[k] = real ? __ldg(f + 2 * i + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t hw[4] = {u[2 * k].x, u[2 * k].y, u[2 * k + 1].x, u[2 * k + 1].y};
                const uint32_t lw[4] = {u[2 * k].z, u[2 * k].w, u[2 * k + 1].z, u[2 * k + 1].w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                  const float2 h2 = __half22float2(*reinterpret_cast<const __half2 *>(&hw[w]));
                  const float2 l2 = __half22float2(*reinterpret_cast<const __half2 *>(&lw[w]));
                  float x0 = (h2.x + l2.x) * inv, x1 = (h2.y + l2.y) * inv;
                  over |= !(fabsf(x0) <= 65504.f) || !(fabsf(x1) <= 65504.f);
                  if (fabsf(x0) > 65504.f) x0 = copysignf(65504.f, x0);  // NaN stays
                  if (fabsf(x1) > 65504.f) x1 = copysignf(65504.f, x1);
                  const __half2 hh = __floats2half2_rn(x0, x1);
                  const float2 hf = __half22float2(hh);
                  const __half2 ll = __floats2half2_rn(x0 - hf.x, x1 - hf.y);
                  hi[w] = *reinterpret_cast<const uint32_t *>(&hh);
                  lo[w] = *reinterpret_cast<const uint32_t *>(&ll);
                }
                sts16(ft + tile_at<128>(l, i + k), hi[0], hi[1], hi[2], hi[3]);
                sts16(ft + tile_at<128>(l, p.rpb / 8 + i + k), lo[0], lo[1], lo[2], lo[3]);
              }
            }
            if (over) atomicOr(a.flags, kFlagRange);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&c.q_full);
      }
      for (int kt = g.k0; kt < g.k1; ++kt, ++tile) {
        const int j0 = kt * kTileKeys, left = s.len - j0;
        const bool tail = j0 + kTileKeys > s.prefix;
        const unsigned alive = pages.alive(a);
        const int slot = slots == 2 ? int(tile & 1u) : 0;
        const uint32_t dst = dst0 + slot * kTile;
        if (tile >= unsigned(slots)) wait_for(&empty[slot], (slots == 2 ? (tile >> 1) - 1 : tile - 1) & 1u, abort);
        if (!is_v) {
          if (l == 0) c.alive[tile & 3] = alive;
          if (alive != (1u << kGroups) - 1u && l == 0) atomicOr(a.flags, kFlagRange);
          if constexpr (BIAS != 0) {
            const int hk = a.fk_heads > 1 ? h : 0;
            const bool plain = j0 + kTileKeys <= min(s.prefix, a.P);  // positions are j0, j0 + 1, ...
            auto position = [&](int row) {
              const int j = j0 + row;
              if (plain) return j;
              if (j >= s.len) return 0;
              if (j >= s.prefix) return new_position(a, g.b, s, j - s.prefix);
              if (j < a.P) return j;
              atomicOr(a.flags, kFlagRange);
              return a.P - 1;
            };
            if constexpr (BIAS == 1) {
              if (l < kTileKeys) {
                const float4 f = __ldg(static_cast<const float4 *>(a.fk) + (long long)hk * a.P + position(l));
                float(*pl)[kTileKeys] = planes[tile & 3];
                pl[0][l] = f.x, pl[1][l] = f.y, pl[2][l] = f.z, pl[3][l] = f.w;
              }
            } else {
              // The keys' factors, (4 hi, 4 lo) groups of 16 bytes, go to the hi and lo columns of the slot's factor tile
              // by asynchronous copies of 8 bytes.
              const uint32_t ft = base + p.fk + slot * fk_tile;
              const int groups = a.RP / 4, total = kTileKeys * groups;
              const uint4 *fbase = static_cast<const uint4 *>(a.fk) + (long long)hk * a.P * groups;
              // lo columns: four chunks on in the same 64 columns, or in the blocks behind the hi ones
              const uint32_t lo_flip = p.rpb == 32 ? 64u : 0u, lo_skip = (p.rpb >> 6) * (kTileKeys * 128);
              auto copy = [&](const uint4 *src, int row, int q) {
                const uint32_t hi = ft + tile_at<kTileKeys>(row, q >> 1) + (q & 1) * 8;
                copy8(hi, src);
                copy8((hi ^ lo_flip) + lo_skip, reinterpret_cast<const uint2 *>(src) + 1);
              };
              int row = l / groups, q = l - row * groups;
              const int rstep = 128 / groups, qstep = 128 - rstep * groups;
              if (plain) {
                const uint4 *src = fbase + (long long)j0 * groups + l;
#pragma unroll 1
                for (int e = l; e < total; e += 128) {
                  copy(src, row, q);
                  src += 128, row += rstep, q += qstep;
                  if (q >= groups) q -= groups, ++row;
                }
              } else {
#pragma unroll 1
                for (int e = l; e < total; e += 128) {
                  copy(fbase + (long long)position(row) * groups + q, row, q);
                  row += rstep, q += qstep;
                  if (q >= groups) q -= groups, ++row;
                }
              }
            }
          }
        }
        const bool more = kt + 1 < g.k1;
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
          if (i >= mine) break;
          const int row = row0 + i * stride;
          const uint4 was = raw[i];
          Chunks out;
          out.x = out.y = was;
          if constexpr (E4M3) {
            const float f = scale_value(sc[E4M3 ? i : 0]);
            out.x = make_uint4(e4m3_to_bf16(was.x, false, f), e4m3_to_bf16(was.x, true, f),
                               e4m3_to_bf16(was.y, false, f), e4m3_to_bf16(was.y, true, f));
            out.y = make_uint4(e4m3_to_bf16(was.z, false, f), e4m3_to_bf16(was.z, true, f),
                               e4m3_to_bf16(was.w, false, f), e4m3_to_bf16(was.w, true, f));
          }
          if (more) load(i, pages.next, j0 + kTileKeys);
          if (!inside || row >= left || !((alive >> (row >> 4)) & 1u)) out.x = out.y = make_uint4(0u, 0u, 0u, 0u);
          if (__builtin_expect(is_v && tail, 0)) out = clear_odd(out, &c.odd[tile & 7], int(tile) + 1);
          const uint32_t to = dst + tile_at<kTileKeys>(row, E4M3 ? 2 * ch : ch);
          sts16(to, out.x.x, out.x.y, out.x.z, out.x.w);
          if constexpr (E4M3) sts16(to ^ 16u, out.y.x, out.y.y, out.y.z, out.y.w);  // the next chunk, an odd one
        }
        pages.now = pages.next;
        pages.next = pages.fetch(a, g.b, j0 + 2 * kTileKeys, s.len, lane);
        if (BIAS == 2 && !is_v) copies_wait_all();
        fence_proxy_async_smem();
        mbar_arrive(&full[slot]);
      }
    }
  } else {
    // ---------------------------------------------------------- MMA issuer
    // One lane issues. The tensor cores take 48 clocks a product and wait for whatever it does between two: a loop that
    // finds each step's addresses anew took 133, without anything else running, so four steps at a time are unrolled,
    // with immediate offsets, and the slots are counters that run on. Both streams share one copy of the code.
    constexpr uint32_t kQK = make_idesc_f16(true, true, 128, kTileKeys, false);
    constexpr uint32_t kF = make_idesc_f16(false, false, 128, kTileKeys, false);
    constexpr uint32_t kPV = make_idesc_f16(true, true, 128, DP, true);
    const uint32_t q0 = low_k(base + p.q), fq0 = low_k(base + p.fq), k0 = low_k(base + p.k), fk0 = low_k(base + p.fk);
    const uint32_t v0 = low_v(base + p.v);
    const uint32_t fq_low = BIAS == 2 ? step_k<128>(p.rpb / 16) : 0u, fk_low = BIAS == 2 ? step_k<kTileKeys>(p.rpb / 16) : 0u;
    const bool split = p.split, ks2 = p.ks == 2;
    const int factor_steps = BIAS == 2 ? a.RP / 16 : 0;
    unsigned ktile = 0, vtile = 0;  // tiles whose K and V the products to come read
    uint32_t qphase = 0, pphase = 0;  // bit t of pphase: stream t's
    if (elect_one()) {
    while (walk.next(a, g)) {
      const int n = g.k1 - g.k0, h = g.item / a.chunks;
      const int rows = min(p.tiles * 128, a.rows - (g.item - h * a.chunks) * p.tiles * 128);
      const int n0 = steps_of(0, n, rows), n1 = nstreams == 2 ? steps_of(1, n, rows) : 0;
      const bool alone = split || n1 == 0;  // a tile is one stream's
      wait_for(&c.q_full, qphase & 1u, abort);
      ++qphase;
      auto score = [&](uint32_t t) {
        const uint32_t slot = ks2 ? ktile & 1u : 0u;
        if (t == 0 || split) wait_for(&c.k_full[slot], (ks2 ? ktile >> 1 : ktile) & 1u, abort);
        tc_fence_after();
        const uint32_t d = tmem + 128u * t, row_tile = t == 1 && !split ? 1u : 0u;
        uint32_t k = k0 + slot * (kTile >> 4), q = q0 + row_tile * (kQTile >> 4);
#pragma unroll 1
        for (uint32_t more = 0; more < DP / 64; ++more) {  // 64 columns, four products
          mma_ss_one(d, desc(q), desc(k), kQK, more);
#pragma unroll
          for (int kk = 1; kk < 4; ++kk) mma_ss_one(d, desc(q + 2 * kk), desc(k + 2 * kk), kQK, 1u);
          q += 128 * 128 >> 4, k += kTileKeys * 128 >> 4;
        }
        if constexpr (BIAS == 2) {
          uint32_t fq = fq0 + row_tile * (fq_tile >> 4), fk = fk0 + slot * (fk_tile >> 4);
#pragma unroll 1
          for (int kk = 0; kk < factor_steps; ++kk) {
            mma_ss_one(d, desc(fq), desc(fk), kF, 1u);
            mma_ss_one(d, desc(fq + fq_low), desc(fk), kF, 1u);
            mma_ss_one(d, desc(fq), desc(fk + fk_low), kF, 1u);
            fq += kk == 3 ? (128 * 128 >> 4) - 6 : 2, fk += kk == 3 ? (kTileKeys * 128 >> 4) - 6 : 2;
          }
        }
        tc_commit(&c.s_full[t]);
        if (alone || t == 1) {
          tc_commit(&c.k_empty[slot]);
          ++ktile;
        }
      };
      auto product = [&](uint32_t t, bool first, bool final) {
        const uint32_t slot = vtile & 1u;
        if (t == 0 || split) wait_for(&c.v_full[slot], (vtile >> 1) & 1u, abort);
        wait_for(&c.p_full[t], (pphase >> t) & 1u, abort);
        pphase ^= 1u << t;
        tc_fence_after();
        const uint32_t d = tmem + 256u + 128u * t, pt = tmem + 128u * t, v = v0 + slot * (kTile >> 4);
        mma_ts_one(d, pt, desc(v), kPV, first ? 0u : 1u);
#pragma unroll
        for (int kk = 1; kk < kTileKeys / 16; ++kk) mma_ts_one(d, pt + uint32_t(kk * 8), desc(v + step_v(kk)), kPV, 1u);
        if (alone || t == 1) {
          tc_commit(&c.v_empty[slot]);
          ++vtile;
        }
        if (final) tc_commit(&c.o_final[t]);
      };
      // S_0(0), S_1(0), PV_0(0), S_0(1), PV_1(0), S_1(1), PV_0(1), ...
#pragma unroll 1
      for (int half = 0; half <= 2 * n0; ++half) {
        const uint32_t t = half & 1;
        const int i = half >> 1, pi = t ? i : i - 1, pn = t ? n0 : n1;
        if (i < (t ? n1 : n0)) score(t);
        if (pi >= 0 && pi < pn) product(1 - t, pi == 0, pi == pn - 1);
      }
    }
      tc_commit(&c.drain);
      if (!mbar_wait_for(&c.drain, 0, 1000000000ull)) c.abort = 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && c.abort) atomicOr(a.flags, kFlagTimeout);
}

// The shared-memory plan, or smem = 0 where none fits.
TilePlan make_plan(int d, int R, int rows) {
  const int DP = d <= 64 ? 64 : 128;
  const int RP = (R + 15) / 16 * 16;
  const uint32_t tile = kTileKeys * DP * 2, qtile = 128 * DP * 2;
  TilePlan best{};
  // One or two row tiles, then slots of K. One of these fits at every head dim and rank: two row tiles up to rank 64
  // (with one slot of K at head dim 128 and rank 64), and beyond it one, with one slot of K at head dim 128.
  static const int kOptions[4][2] = {{2, 2}, {2, 1}, {1, 2}, {1, 1}};
  for (const auto &o : kOptions) {
    TilePlan p{};
    p.tiles = o[0], p.ks = o[1];
    if (p.tiles == 2 && rows <= 128) continue;
    p.rpb = R <= kCacheBiasExact ? 0 : (RP <= 32 ? 32 : (RP <= 64 ? 64 : 128));
    const uint32_t f = kTileKeys * 4 * p.rpb;
    p.q = 0;
    p.fq = p.q + p.tiles * qtile;
    p.k = p.fq + p.tiles * 128 * 4 * p.rpb;
    p.fk = p.k + p.ks * tile;
    p.v = p.fk + p.ks * f;
    p.planes = p.v + 2 * tile;
    p.ctrl = p.planes + (R > 0 && R <= kCacheBiasExact ? 4 * 4 * kTileKeys * 4 : 0);
    p.smem = p.ctrl + uint32_t(sizeof(Ctrl)) + 1024;
    p.split = p.tiles == 1 && p.ks == 2;
    if (p.smem <= 227u * 1024u) {
      best = p;
      break;
    }
  }
  // more than half of the SM's shared memory: one CTA an SM, which takes all of the SM's TMEM
  if (best.smem) best.smem = std::max(best.smem, 120u * 1024u);
  return best;
}

template <int DP, bool E4M3, int BIAS>
cudaError_t launch_bias(const CacheAttnArgs &a, const TilePlan &p, int grid, cudaStream_t st) {
  auto *k = attn_cache_tile_kernel<DP, E4M3, BIAS>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_all_shared_memory(reinterpret_cast<const void *>(k), done);
  if (e != cudaSuccess) return e;
  return launch_programmatic(k, dim3(unsigned(grid)), dim3(kThreads), size_t(p.smem), st, a, p);
}

template <int DP, bool E4M3>
cudaError_t launch_tile(const CacheAttnArgs &a, const TilePlan &p, int grid, cudaStream_t st) {
  if (a.R == 0) return launch_bias<DP, E4M3, 0>(a, p, grid, st);
  return a.R <= kCacheBiasExact ? launch_bias<DP, E4M3, 1>(a, p, grid, st) : launch_bias<DP, E4M3, 2>(a, p, grid, st);
}

}  // namespace

size_t cache_tile_part_floats(int d, int sms) { return size_t(2) * sms * 256 * ((d <= 64 ? 64 : 128) + 2); }

cudaError_t launch_attn_cache_tile(CacheAttnArgs a, int e4m3, int sms, cudaStream_t st) {
  const TilePlan p = make_plan(a.d, a.R, a.rows);
  if (!p.smem) return cudaErrorInvalidValue;
  a.chunks = (a.rows + p.tiles * 128 - 1) / (p.tiles * 128);
  const long long blocks = std::max<long long>(1, (((long long)a.max_pages << a.page_shift) + kTileKeys - 1) / kTileKeys);
  const int grid = int(std::min<long long>((long long)a.B * a.H * a.chunks * blocks, sms));
  if (a.d <= 64) return e4m3 ? launch_tile<64, true>(a, p, grid, st) : launch_tile<64, false>(a, p, grid, st);
  return e4m3 ? launch_tile<128, true>(a, p, grid, st) : launch_tile<128, false>(a, p, grid, st);
}

}  // namespace fb
