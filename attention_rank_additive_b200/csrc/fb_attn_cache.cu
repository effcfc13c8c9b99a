// fb_attn_cache.cu -- attention of new tokens (one, or a tree of drafted ones)
// over a paged key/value cache, with a low-rank additive bias:
//
//   x_tj = scale q_t.k_j + phi_q[pos t].phi_k[pos j],
//   O_t  = sum_j softmax_j(x_tj) v_j,   LSE_t = ln sum_j exp x_tj,
//
// over the context (every row sees it) and the drafted tokens that row t's mask
// names. The G query heads of a key/value head and the T tokens of a sequence
// are the rows of one tile, so the cache is read once per key/value head.
//
// What bounds it: the cache's bytes. So the products are laid out for loads:
// the keys are the 16 rows of the matrix instruction and the (few) query rows
// its 8 columns, S^T = K Q^T and O^T = V^T P^T. Both operands that come from
// memory then take d in any order as long as the query side (or the output)
// uses the same one, so a lane's operand registers are 16 neighbouring bytes of
// a row, and every sector of a row is read whole by one instruction. The same
// swap halves the idle rows for a single token (8 columns, not 16 rows). P^T is
// S^T's accumulator after one 8x8 transpose (movmatrix).
//
// Each warp walks over 16-key groups of its own, one or two a step. A group lies
// in one page, so its K, V, scales and (in the context) factors are one run of
// bytes each: one lane fetches them with bulk copies into the warp's ring in
// shared memory, a few steps ahead, and the other lanes do no address work.
//
// 8-bit keys and values become fp16 in registers, exactly. (Given codes as they
// are, the 8-bit mma.sync instruction of this architecture takes twice the
// matrix instructions and 50 additions a group more: a decode step of 16 ragged
// contexts up to 8191 tokens, 16 heads of 128, took 130 us with it.) Measured:
// that step 90 us, 4.7 TB/s; two contexts of 131071 tokens in bf16, 32 query and
// 8 key/value heads, 190 us, 5.5 TB/s. What bounds them is the latency of each
// warp's chain of instructions: 12 and 8 warps are all that an SM's shared
// memory feeds. With one group a step the first took 112 us, with two CTAs of an
// SM in place of three 104 us.
//
// Work is dealt out by keys: all blocks of keys of all (sequence, head) items,
// as the lengths on the device say, are numbered through and each CTA takes an
// equal run of them. An item that crosses CTAs leaves partial (O, max, sum)
// rows in the workspace; the last of its CTAs to arrive adds them up in CTA
// order, so the result does not depend on who arrives last.
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "fb_attn_cache.cuh"
#include "fb_internal.h"

namespace fb {
namespace {

constexpr int kWarps = 4;

// 16-key groups that a warp takes in one step: two where rows are short, which gives its chains of dependent
// instructions something to overlap with.
constexpr int groups_per_step(int D, bool E4M3, int NB) { return NB == 1 && D * (E4M3 ? 1 : 2) <= 128 ? 2 : 1; }

// CTAs of 128 threads on an SM at most, by blocks of 8 query rows: the registers of O and Q allow no more.
constexpr int cta_per_sm(int NB) { return NB == 1 ? 4 : 3; }
// And what their rings leave room for (head dim 128 in 8 bits with two groups a step: three).
constexpr int most_ctas(int D, bool E4M3, int NB) { return std::min(cta_per_sm(NB), D == 128 ? (E4M3 ? 3 : 2) : 4); }

__device__ __forceinline__ void mma_bf16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two e4m3 codes (the low or high half of w) as fp16; exact.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(y) : "r"(w));
  return y;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(y) : "r"(w));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}
// N words of shared memory: plain loads, which the compiler may start early and order among the products as it likes.
template <int N>
__device__ __forceinline__ void read_words(const uint8_t *src, uint32_t *w) {
  if constexpr (N == 4) {
    const uint4 u = *reinterpret_cast<const uint4 *>(src);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2 *>(src);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(src);
  }
}

// How a lane's share of a row lies, for head dims padded to D (32, 64, 96, 128).
template <int D, bool E4M3>
struct Lay {
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int KW = D * ES / 16;  // words of one key row per lane (a quarter of the row)
  static constexpr int VW = D * ES / 32;  // words of one value row per lane (an eighth of the row)
  // K: loads of KL words; the four lanes of a row take neighbouring KL-word pieces
  static constexpr int KL = E4M3 && D % 64 != 0 ? 2 : 4;
  // V: a piece of 64 values (of 128 for e4m3 at D = 128) is spread over eight lanes, then one of 32
  static constexpr int VL0 = D == 32 ? VW : (E4M3 ? (D == 128 ? 4 : 2) : 4);
  // d of value v (0 .. D/8 - 1) of lane group g
  static __device__ __forceinline__ int vd(int g, int v) {
    constexpr int per0 = VL0 * 4 / ES;  // values of a piece per lane
    if constexpr (D == 96) return v < per0 ? g * per0 + v : 64 + g * (per0 / 2) + (v - per0);
    return (v / per0) * (8 * per0) + g * per0 + v % per0;
  }
};

constexpr int kMaxStages = 8;

template <int D, int NB>
struct Join {  // over the ring, once a segment's keys are done
  float o[kWarps][8 * NB][D];
  float m[kWarps][8 * NB], l[kWarps][8 * NB], e[kWarps][8 * NB];
};

template <int NB, int BIAS>
struct Smem {
  uint4 fq[BIAS == 2 ? NB * 8 * 32 : 1];  // phi_q as matrix operands: [block][16 ranks][lane]
  uint64_t full[kWarps][kMaxStages];      // a ring slot's copies have landed
  int last;
  int odd;  // a non-finite value left the products of this segment
  int abort;
  int pad;
};

// What a group takes in the ring: 16 rows of K, of V, 16 scale bytes of each (e4m3), 16 rows of factors. A slot holds a
// step's groups, all of their K first, then V, the scales and the factors; 16-byte multiples.
__host__ __device__ __forceinline__ int stage_bytes(int d, bool e4m3, int bias, int RP) {
  return 32 * d * (e4m3 ? 1 : 2) + (e4m3 ? 32 : 0) + (bias == 1 ? 256 : (bias == 2 ? 64 * RP : 0));
}

template <int D, bool E4M3, int NB, int BIAS>
__global__ void __launch_bounds__(kWarps * 32, most_ctas(D, E4M3, NB)) attn_cache_kernel(const __grid_constant__ CacheAttnArgs a, const int stages) {
  using L = Lay<D, E4M3>;
  constexpr int KS = D / 16, ROWS = 8 * NB, KM = groups_per_step(D, E4M3, NB);
  constexpr int BK = 16 * KM * kWarps;  // a block of keys: a step of each warp
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto &sm = *reinterpret_cast<Smem<NB, BIAS> *>(smem_raw);
  auto &join = *reinterpret_cast<Join<D, NB> *>(smem_raw + sizeof(sm));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  griddep_wait();

  // ---- this CTA's run of blocks of all items
  Walk walk(a, BK, 0, lane);
  if (blockIdx.x >= walk.ctas) return;
  if (threadIdx.x == 0) sm.abort = 0;
  if (lane < stages) mbar_init(&sm.full[warp][lane], 1);
  fence_mbar_init();
  int slot = 0;         // of the next group to use
  uint32_t parity = 0;  // of its barrier
  Segment seg;
  while (walk.next(a, seg)) {
    const Seq &s = seg.s;
    const int b = seg.b, nb = seg.blocks, k0 = seg.k0, k1 = seg.k1;
    const int h = seg.item / a.chunks, r0 = (seg.item - h * a.chunks) * ROWS;
    const long long qrow0 = ((long long)b * a.Hq + (long long)h * a.G) * a.T;  // row r of the item is output row qrow0 + r

    // ---- queries as the matrix operand: lane (g, t4) holds row g's values at the d that its key loads have. 8-bit keys
    // become fp16, exactly, and the queries too: a power of two is taken out of a row so that its largest value lies in
    // [2^14, 2^15). Values from 2^-28 of that on are exact, smaller ones off by 2^-39 of it at most.
    uint32_t qf[NB][KS][2];  // bf16 or fp16 pairs
    float mult[NB][2];       // scale, and the power of two taken out of a query row
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int r = r0 + n * 8 + g;
      const bool in = r < a.rows;
      const __nv_bfloat16 *q = a.Q + (qrow0 + (in ? r : 0)) * a.d;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        constexpr int per = L::KL * 4 / L::ES;  // values per load and lane
        const int d0 = (k * 4 / per) * (4 * per) + t4 * per + (k * 4) % per;
        uint2 v = make_uint2(0u, 0u);
        if (in && d0 < a.d) v = __ldg(reinterpret_cast<const uint2 *>(q + d0));
        qf[n][k][0] = v.x, qf[n][k][1] = v.y;
      }
      mult[n][0] = mult[n][1] = a.scale;
      if constexpr (E4M3) {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x0 = fabsf(__uint_as_float(qf[n][k][i] << 16)), x1 = fabsf(__uint_as_float(qf[n][k][i] & 0xffff0000u));
            top = fmaxf(top, fmaxf(x0 < INFINITY ? x0 : 0.f, x1 < INFINITY ? x1 : 0.f));
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(int(__float_as_uint(top) >> 23) - 141, -126);  // top = 1.m 2^(e + 14)
        const float down = pow2i(-e), up = pow2i(e);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[n][k][i] = pack_f16x2(__uint_as_float(qf[n][k][i] << 16) * down,
                                     __uint_as_float(qf[n][k][i] & 0xffff0000u) * down);
        mult[n][0] *= __shfl_sync(0xffffffffu, up, t4 * 8);
        mult[n][1] *= __shfl_sync(0xffffffffu, up, t4 * 8 + 4);
      }
    }
    // ---- the rows' tokens and factors (lane's score columns: rows 2 t4, 2 t4 + 1 of each block)
    int tok[NB][2];
    float fq[NB][2][BIAS == 1 ? 4 : 1];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + n * 8 + 2 * t4 + i;
        const int t = r < a.rows ? r % a.T : a.T;
        tok[n][i] = t < s.count ? t : -1;
        if constexpr (BIAS == 1) {
          float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
          if (tok[n][i] >= 0) {
            const int hq = a.fq_heads > 1 ? h * a.G + r / a.T : 0;
            f = __ldg(static_cast<const float4 *>(a.fq) + (long long)hq * a.P + new_position(a, b, s, t));
          }
          fq[n][i][0] = f.x, fq[n][i][1] = f.y, fq[n][i][2] = f.z, fq[n][i][3] = f.w;
        }
      }
    if constexpr (BIAS == 2) {
      __syncthreads();  // the last item's readers are done
      for (int i = threadIdx.x; i < NB * (a.RP / 16) * 32; i += kWarps * 32) {
        const int ln = i & 31, c = (i >> 5) % (a.RP / 16), n = (i >> 5) / (a.RP / 16);
        const int r = r0 + n * 8 + (ln >> 2), t = r < a.rows ? r % a.T : a.T;
        uint4 f = make_uint4(0u, 0u, 0u, 0u);
        if (t < s.count) {
          const int hq = a.fq_heads > 1 ? h * a.G + r / a.T : 0;
          f = __ldg(static_cast<const uint4 *>(a.fq) + ((long long)hq * a.P + new_position(a, b, s, t)) * (a.RP / 4) +
                    c * 4 + (ln & 3));
        }
        sm.fq[(n * 8 + c) * 32 + ln] = f;
      }
      __syncthreads();
    }

    float o[KS][NB][4];
    float m[NB][2], l[NB][2], ex[NB][2];  // running maximum, this lane's sum, exponent of O's unit 2^ex (e4m3)
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[k][n][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) m[n][i] = -INFINITY, l[n][i] = 0.f, ex[n][i] = -INFINITY;
    }

    if (threadIdx.x == 0) sm.odd = 0;
    fence_proxy_async_smem();  // the ring's bulk copies come after what was written and read there
    __syncthreads();           // sm.odd; and the last segment's readers of shared memory are done
    fence_proxy_async_smem();
    const int *table = a.table + (long long)b * a.max_pages;
    const int jend = min(s.len, k1 * BK), jstart = k0 * BK + warp * 16 * KM;
    const int hk = BIAS ? (a.fk_heads > 1 ? h : 0) : 0;
    const int rb = a.d * L::ES;  // bytes of a row
    const int slot_bytes = KM * stage_bytes(a.d, E4M3, BIAS, a.RP);
    const int v_at = KM * 16 * rb, ks_at = 2 * v_at, vs_at = ks_at + KM * 16, f_at = ks_at + (E4M3 ? KM * 32 : 0);
    const int fk_row = BIAS == 1 ? 16 : 4 * a.RP;
    const uint8_t *fk_head = static_cast<const uint8_t *>(a.fk) + (BIAS ? (long long)hk * a.P * fk_row : 0ll);
    uint8_t *ring = smem_raw + sizeof(sm) + warp * stages * slot_bytes;
    // The page of lane i's group (i < KM) of the step at j, and one that is not there.
    auto page_of = [&](int j) {
      j += 16 * lane;
      return lane < KM && j < jend ? __ldg(table + (j >> a.page_shift)) : -1;
    };
    auto page_ok = [&](int page) { return page >= 0 && page < a.num_pages; };
    // Fetch the step at j into ring slot `to`. What the copies take is the same in all lanes, found by reductions, which
    // leave it in uniform registers: a copy by a lane with values of its own costs a loop over the lanes.
    auto fetch = [&](int j, int page, int to) {
      if (j >= jend) return;
      int pages[KM];
      bool ok[KM];
      int there = 0;
#pragma unroll
      for (int i = 0; i < KM; ++i) {
        pages[i] = __reduce_max_sync(0xffffffffu, lane == i ? page : INT_MIN);
        ok[i] = page_ok(pages[i]);
        there += ok[i];
        if (!ok[i] && j + 16 * i < jend && lane == 0) atomicOr(a.flags, kFlagRange);
      }
      // the step's factors, where all are of the context; else they are read where they are used
      const bool factors = BIAS != 0 && j + 16 * KM <= min(s.prefix, a.P);
      const bool one = KM == 1 || (a.page_shift > 4 && there == KM);  // its groups are neighbours in one page
      if (elect_one()) {
        uint64_t *bar = &sm.full[warp][to];
        uint8_t *dst = ring + to * slot_bytes;
        mbar_arrive_expect_tx(bar, there * (32 * rb + (E4M3 ? 32 : 0)) + (factors ? KM * 16 * fk_row : 0));
#pragma unroll
        for (int i = 0; i < KM; ++i) {
          if (!ok[i] || (one && i > 0)) continue;
          const long long prow = (((long long)pages[i] * a.H + h) << a.page_shift) + ((j + 16 * i) & ((1 << a.page_shift) - 1));
          const int rows = one ? 16 * KM : 16;
          bulk_load(dst + 16 * i * rb, static_cast<const uint8_t *>(a.kp) + prow * rb, rows * rb, bar);
          bulk_load(dst + v_at + 16 * i * rb, static_cast<const uint8_t *>(a.vp) + prow * rb, rows * rb, bar);
          if constexpr (E4M3) {
            bulk_load(dst + ks_at + 16 * i, a.ks + prow, rows, bar);
            bulk_load(dst + vs_at + 16 * i, a.vs + prow, rows, bar);
          }
        }
        if (factors) bulk_load(dst + f_at, fk_head + (long long)j * fk_row, KM * 16 * fk_row, bar);
      }
      __syncwarp();
    };
    // Lanes whose d lies past the row (two of a key row's four, in its last piece) read its first bytes instead: the
    // queries are 0 there, and O is not written. Key values of 16 bits, which may be infinite, become 0 too; an 8-bit one
    // is finite or NaN, and NaN is the score in any case.
    const bool past = !E4M3 && a.d < D && t4 >= 2;
    int kat[L::KW / L::KL], vat[L::VW / L::VL0 + (D == 96 ? 1 : 0)];
#pragma unroll
    for (int c = 0; c < L::KW / L::KL; ++c) {
      const int at = (c * 4 + t4) * (L::KL * 4);
      kat[c] = g * rb + (at < rb ? at : 0);
    }
#pragma unroll
    for (int c = 0; c < L::VW / L::VL0 + (D == 96 ? 1 : 0); ++c) {
      const int at = D == 96 && c == 1 ? 64 * L::ES + g * (L::VL0 * 2) : (c * 8 + g) * (L::VL0 * 4);
      vat[c] = v_at + 2 * t4 * rb + (at < rb ? at : 0);
    }
    // page numbers one step ahead of their fetch
    int fill = slot;
    for (int i = 0; i < stages - 1; ++i) {
      fetch(jstart + i * BK, page_of(jstart + i * BK), fill);
      fill = fill + 1 == stages ? 0 : fill + 1;
    }
    int page_fill = page_of(jstart + (stages - 1) * BK);
    int page_use = page_of(jstart);
    for (int j0 = jstart; j0 < jend; j0 += BK) {
      fetch(j0 + (stages - 1) * BK, page_fill, fill);
      fill = fill + 1 == stages ? 0 : fill + 1;
      page_fill = page_of(j0 + stages * BK);
      const unsigned alive = __ballot_sync(0xffffffffu, page_ok(page_use));  // bit mb: group mb has a page
      page_use = page_of(j0 + BK);
      mbar_wait(&sm.full[warp][slot], parity, &sm.abort);
      const uint8_t *src = ring + slot * slot_bytes;
      const bool tail = j0 + 16 * KM > s.prefix || alive != (1u << KM) - 1u;  // new tokens, rows past the end, or no page

      // ---- scores: S^T = K Q^T (16 keys x 8 rows per block)
      float x[KM][NB][4];
#pragma unroll
      for (int mb = 0; mb < KM; ++mb) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[mb][n][i] = 0.f;
#pragma unroll
        for (int c = 0; c < L::KW / L::KL; ++c) {
          uint32_t kr[2][L::KL];
#pragma unroll
          for (int i = 0; i < 2; ++i) read_words<L::KL>(src + (mb * 16 + 8 * i) * rb + kat[c], kr[i]);
          if (!E4M3 && c == L::KW / L::KL - 1 && past) {
#pragma unroll
            for (int w = 0; w < L::KL; ++w) kr[0][w] = kr[1][w] = 0u;
          }
          // a product takes four values of each row: two words of bf16, or one word of codes
          constexpr int products = E4M3 ? L::KL : L::KL / 2;
#pragma unroll
          for (int kk = 0; kk < products; ++kk) {
            const int k = c * products + kk;
            uint32_t a0, a1, a2, a3;
            if constexpr (E4M3) {
              a0 = e4m3_lo(kr[0][kk]), a1 = e4m3_lo(kr[1][kk]), a2 = e4m3_hi(kr[0][kk]), a3 = e4m3_hi(kr[1][kk]);
            } else {
              a0 = kr[0][2 * kk], a1 = kr[1][2 * kk], a2 = kr[0][2 * kk + 1], a3 = kr[1][2 * kk + 1];
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              if constexpr (E4M3)
                mma_f16(x[mb][n], a0, a1, a2, a3, qf[n][k][0], qf[n][k][1]);
              else
                mma_bf16(x[mb][n], a0, a1, a2, a3, qf[n][k][0], qf[n][k][1]);
            }
          }
        }
      }
      // ---- scale and bias
      float svf[KM][2];
#pragma unroll
      for (int mb = 0; mb < KM; ++mb) {
        const int j1 = j0 + 16 * mb;
        const bool in_ring = BIAS != 0 && j0 + 16 * KM <= min(s.prefix, a.P);
        const uint8_t *fsrc = src + f_at + mb * 16 * fk_row;
        int kpos[2] = {0, 0};
        if (BIAS != 0 && !in_ring) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int jk = j1 + g + 8 * i;
            if (jk >= s.len) continue;
            kpos[i] = jk >= s.prefix ? new_position(a, b, s, jk - s.prefix) : jk;
            if (kpos[i] >= a.P) {
              atomicOr(a.flags, kFlagRange);
              kpos[i] = a.P - 1;
            }
          }
        }
        float bias[NB][4];
        if constexpr (BIAS == 2) {
          float low[NB][4];  // the two small products
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) bias[n][i] = low[n][i] = 0.f;
          for (int c = 0; c < a.RP / 16; ++c) {
            uint32_t f[2][4];  // 4 hi, 4 lo
            if (in_ring) {
#pragma unroll
              for (int i = 0; i < 2; ++i) read_words<4>(fsrc + (g + 8 * i) * fk_row + c * 64 + t4 * 16, f[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(fk_head + (long long)kpos[i] * fk_row + c * 64 + t4 * 16));
                f[i][0] = u.x, f[i][1] = u.y, f[i][2] = u.z, f[i][3] = u.w;
              }
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              const uint4 q = sm.fq[(n * 8 + c) * 32 + lane];
              // (kh + kl)(qh + ql) without the last 2^-22
              mma_f16(low[n], f[0][2], f[1][2], f[0][3], f[1][3], q.x, q.y);
              mma_f16(bias[n], f[0][0], f[1][0], f[0][1], f[1][1], q.x, q.y);
              mma_f16(low[n], f[0][0], f[1][0], f[0][1], f[1][1], q.z, q.w);
            }
          }
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) bias[n][i] += low[n][i];
        }
        float fk[2][4], skf[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (BIAS == 1) {
            const float4 f = in_ring ? *reinterpret_cast<const float4 *>(fsrc + (g + 8 * i) * 16)
                                     : __ldg(reinterpret_cast<const float4 *>(fk_head) + kpos[i]);
            fk[i][0] = f.x, fk[i][1] = f.y, fk[i][2] = f.z, fk[i][3] = f.w;
          }
          skf[i] = svf[mb][i] = 0.f;
          if constexpr (E4M3) {
            const uint32_t k8 = src[ks_at + mb * 16 + g + 8 * i], v8 = src[vs_at + mb * 16 + g + 8 * i];
            skf[i] = scale_value(k8);
            svf[mb][i] = v8 == 255u ? __uint_as_float(0x7fffffffu) : float(int(v8) - 127);
          }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kk = i >> 1, rr = i & 1;
            float f = mult[n][rr];
            if constexpr (E4M3) f *= skf[kk];
            if constexpr (BIAS == 1) {
              float y = fk[kk][0] * fq[n][rr][0];
#pragma unroll
              for (int r = 1; r < 4; ++r) y = fmaf(fk[kk][r], fq[n][rr][r], y);
              x[mb][n][i] = fmaf(x[mb][n][i], f, y);
            } else if constexpr (BIAS == 2) {
              x[mb][n][i] = fmaf(x[mb][n][i], f, bias[n][i]);
            } else {
              x[mb][n][i] *= f;
            }
          }
        if (tail) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j1 + g + 8 * (i >> 1), u = j - s.prefix, t = tok[n][i & 1];
              const bool see = ((alive >> mb) & 1u) && j < s.len && (u < 0 || (t >= 0 && drafted_visible(a, b, t, u)));
              if (!see) x[mb][n][i] = -INFINITY;
            }
        }
      }
      // ---- running maximum, raised only when a score passes it by more than 8 (exp stays below e^8)
      float top[NB][2];
      bool need = false;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[n][i] = fmaxf(x[0][n][i], x[0][n][i + 2]);
#pragma unroll
          for (int mb = 1; mb < KM; ++mb) top[n][i] = fmax3(top[n][i], x[mb][n][i], x[mb][n][i + 2]);
          need |= top[n][i] > m[n][i] + 8.f;
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v = top[n][i];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, w));
            const float mn = fmaxf(m[n][i], v);
            if (mn > m[n][i]) {
              const float down = (m[n][i] - mn) * kCacheLog2e;  // -inf at the first
              const float alpha = ex2_approx(down);
              l[n][i] *= alpha;
              if constexpr (E4M3) {
                ex[n][i] += down;  // O is kept and counts in a smaller unit
              } else {
#pragma unroll
                for (int k = 0; k < KS; ++k) o[k][n][i] *= alpha, o[k][n][i + 2] *= alpha;
              }
              m[n][i] = mn;
            }
          }
      }
      // ---- probabilities; e4m3 values: each key's weight takes the value row's power of two, fp16 in O's unit
      uint32_t pf[KM][NB][2];
      if constexpr (E4M3) {
        bool grow = false;
        float ytop[NB][2];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mu = m[n][i] == -INFINITY ? 0.f : m[n][i];
            ytop[n][i] = -INFINITY;
#pragma unroll
            for (int mb = 0; mb < KM; ++mb)
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) {
                const float y = (x[mb][n][2 * kk + i] - mu) * kCacheLog2e;
                x[mb][n][2 * kk + i] = y;
                l[n][i] += ex2_approx(y);
                ytop[n][i] = fmaxf(ytop[n][i], y + svf[mb][kk]);
              }
            grow |= ytop[n][i] - 15.f > ex[n][i];  // the largest weight is kept below 2^15
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float v = ytop[n][i];
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, w));
              const float en = fmaxf(ex[n][i], v - 8.f);
              if (en > ex[n][i]) {
                const float alpha = ex2_approx(ex[n][i] - en);
#pragma unroll
                for (int k = 0; k < KS; ++k) o[k][n][i] *= alpha, o[k][n][i + 2] *= alpha;
                ex[n][i] = en;
              }
            }
        }
#pragma unroll
        for (int mb = 0; mb < KM; ++mb)
#pragma unroll
          for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float y = x[mb][n][i];
              x[mb][n][i] = y == -INFINITY ? 0.f : ex2_approx(y + (svf[mb][i >> 1] - ex[n][i & 1]));
            }
            pf[mb][n][0] = transpose8x8(pack_f16x2(x[mb][n][0], x[mb][n][1]));
            pf[mb][n][1] = transpose8x8(pack_f16x2(x[mb][n][2], x[mb][n][3]));
          }
      } else {
        // weights rounded to bf16 (2^-8 at most, each its own, next to O's own rounding); their sum stays fp32
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
          for (int mb = 0; mb < KM; ++mb) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[mb][n][i] = ex2_approx((x[mb][n][i] - (i & 1 ? m1 : m0)) * kCacheLog2e);
              l[n][i & 1] += x[mb][n][i];
            }
            pf[mb][n][0] = transpose8x8(pack_bf16x2(x[mb][n][0], x[mb][n][1]));
            pf[mb][n][1] = transpose8x8(pack_bf16x2(x[mb][n][2], x[mb][n][3]));
          }
        }
      }
      // ---- O^T += V^T P^T
      constexpr int VP = L::VL0;
      constexpr int pieces = L::VW / VP + (D == 96 ? 1 : 0);
#pragma unroll
      for (int mb = 0; mb < KM; ++mb)
#pragma unroll
        for (int c = 0; c < pieces; ++c) {
          constexpr int full = D == 96 ? 1 : pieces;
          const bool last = c >= full;  // the half piece of D = 96
          uint32_t vr[4][VP];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint8_t *p = src + (mb * 16 + (i & 1) + 8 * (i >> 1)) * rb + vat[c];
            if (!last)
              read_words<VP>(p, vr[i]);
            else
              read_words<(VP + 1) / 2>(p, vr[i]);
          }
          // an infinite or NaN value must not reach the rows that do not see its key (0 * inf): where new tokens are
          // among the step's keys it leaves the product, and the rows that see it get it back when the segment is joined
          // (a step wholly of the context keeps it: all rows see it); rows behind the last token, and those of no page,
          // are nothing at all
          if (tail) {
            const bool fresh = j0 + 16 * KM > s.prefix;
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool real = ((alive >> mb) & 1u) && j0 + 16 * mb + 2 * t4 + (i & 1) + 8 * (i >> 1) < s.len;
#pragma unroll
              for (int w = 0; w < VP; ++w) {
                if (last && w >= VP / 2) continue;
                const uint32_t was = real ? vr[i][w] : 0u, even = fresh ? even_word<E4M3>(was) : was;
                odd |= even != was;
                vr[i][w] = even;
              }
            }
            if (odd) sm.odd = 1;
          }
          constexpr int per = E4M3 ? VP * 2 : VP;  // products per piece
#pragma unroll
          for (int kk = 0; kk < per; ++kk) {
            if (last && kk >= per / 2) continue;
            const int k = c * per + kk;
            uint32_t a0, a1, a2, a3;
            if constexpr (E4M3) {
              const int w = kk / 2;
              const uint32_t sel = kk & 1 ? 0x7362u : 0x5140u;  // the two keys' bytes side by side
              const uint32_t u = __byte_perm(vr[0][w], vr[1][w], sel);
              const uint32_t v = __byte_perm(vr[2][w], vr[3][w], sel);
              a0 = e4m3_lo(u), a1 = e4m3_hi(u), a2 = e4m3_lo(v), a3 = e4m3_hi(v);
            } else {
              a0 = __byte_perm(vr[0][kk], vr[1][kk], 0x5410), a1 = __byte_perm(vr[0][kk], vr[1][kk], 0x7632);
              a2 = __byte_perm(vr[2][kk], vr[3][kk], 0x5410), a3 = __byte_perm(vr[2][kk], vr[3][kk], 0x7632);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              if constexpr (E4M3)
                mma_f16(o[k][n], a0, a1, a2, a3, pf[mb][n][0], pf[mb][n][1]);
              else
                mma_bf16(o[k][n], a0, a1, a2, a3, pf[mb][n][0], pf[mb][n][1]);
            }
          }
        }
      if (++slot == stages) slot = 0, parity ^= 1u;
      __syncwarp();  // the slot's readers are done before it is filled again
    }

    __syncthreads();  // the ring becomes the join's memory
    const bool odd = sm.odd;  // read by all before the next barrier, behind which thread 0 may clear it for the next segment
    // ---- the warps' parts of the segment
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[n][i];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        const int row = n * 8 + 2 * t4 + i;
        if (g == 0) join.m[warp][row] = m[n][i], join.l[warp][row] = sum, join.e[warp][row] = E4M3 ? ex[n][i] : 0.f;
#pragma unroll
        for (int v = 0; v < D / 8; ++v) join.o[warp][row][L::vd(g, v)] = o[v / 2][n][(v & 1) * 2 + i];
      }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == nb;
    const int nrows = min(ROWS, a.rows - r0);
    constexpr long long kSlot = ROWS * (D + 2);
    float *mine = a.part + (2ll * blockIdx.x + (k0 == 0)) * kSlot;
    for (int i = threadIdx.x; i < nrows * D; i += kWarps * 32) {
      const int row = i / D, dd = i % D;
      float top = join.m[0][row];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, join.m[w][row]);
      float sum = 0.f, val = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (saw_none(join.m[w][row], join.l[w][row])) continue;
        const float y = (join.m[w][row] - top) * kCacheLog2e;
        sum += join.l[w][row] * ex2_approx(y);
        val += join.o[w][row][dd] * ex2_approx(y + join.e[w][row]);
      }
      if (odd && dd < a.d) val += odd_sum<E4M3, false>(a, s, b, h, (r0 + row) % a.T, dd, max(k0 * BK, s.prefix / (16 * KM) * (16 * KM)), jend);
      if (whole) {
        write_row(a, s, qrow0 + r0 + row, (r0 + row) % a.T, dd, top, sum, val);
      } else {
        mine[row * (D + 2) + dd] = val;
        if (dd == 0) mine[row * (D + 2) + D] = top, mine[row * (D + 2) + D + 1] = sum;
      }
    }
    if (!whole) {
      const int c0 = walk.owner(seg.start), c1 = walk.owner(seg.start + nb - 1);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) sm.last = atomicAdd(a.counters + c0, 1u) == unsigned(c1 - c0);
      __syncthreads();
      if (sm.last) {
        __threadfence();
        for (int i = threadIdx.x; i < nrows * D; i += kWarps * 32) {
          const int row = i / D, dd = i % D;
          float top = -INFINITY, sum = 0.f, val = 0.f;
          for (int c = c0; c <= c1; ++c) {
            const float *p = a.part + (2ll * c + (c == c0)) * kSlot + row * (D + 2);
            const float mc = __ldcg(p + D);
            const float sc = __ldcg(p + D + 1), vc = __ldcg(p + dd);
            if (saw_none(mc, sc)) continue;
            const float mn = fmaxf(top, mc);
            const float f0 = ex2_approx((top - mn) * kCacheLog2e), f1 = ex2_approx((mc - mn) * kCacheLog2e);
            sum = sum * f0 + sc * f1;
            val = val * f0 + vc * f1;
            top = mn;
          }
          write_row(a, s, qrow0 + r0 + row, (r0 + row) % a.T, dd, top, sum, val);
        }
        if (threadIdx.x == 0) a.counters[c0] = 0u;  // for the next call
      }
    }
  }
  if (threadIdx.x == 0 && sm.abort) atomicOr(a.flags, kFlagTimeout);
}

template <int D, bool E4M3, int NB, int BIAS>
cudaError_t launch_bias(const CacheAttnArgs &a, int sms, cudaStream_t st) {
  auto *k = attn_cache_kernel<D, E4M3, NB, BIAS>;
  constexpr int keys = 16 * groups_per_step(D, E4M3, NB) * kWarps;  // a block's
  const int stage = keys / 16 * stage_bytes(a.d, E4M3, BIAS, a.RP);
  const int fixed = sizeof(Smem<NB, BIAS>), join = sizeof(Join<D, NB>);
  // CTAs on an SM: as many as leave each a ring of four groups a warp (three, of one group a step) in the 227 KB (1 KB
  // a CTA is the system's); every CTA of the grid is resident, so the equal runs of keys also end together
  constexpr int least = groups_per_step(D, E4M3, NB) == 2 ? 2 : 3;
  int ctas = most_ctas(D, E4M3, NB) + 1, stages = 0;
  while (stages < least && ctas > 1) {
    --ctas;
    stages = std::min(kMaxStages, (227 * 1024 / ctas - 1024 - fixed) / stage);
  }
  stages = std::max(2, stages);
  const int smem = fixed + std::max(join, stages * stage);
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_all_shared_memory(reinterpret_cast<const void *>(k), done);
  if (e != cudaSuccess) return e;
  const long long blocks = std::max<long long>(1, (((long long)a.max_pages << a.page_shift) + keys - 1) / keys);
  const int grid = int(std::min<long long>((long long)a.B * a.H * a.chunks * blocks, (long long)sms * ctas));
  return launch_programmatic(k, dim3(unsigned(grid)), dim3(kWarps * 32), size_t(smem), st, a, stages);
}

template <int D, bool E4M3, int NB>
cudaError_t launch_nb(CacheAttnArgs &a, int sms, cudaStream_t st) {
  a.chunks = (a.rows + 8 * NB - 1) / (8 * NB);
  if (a.R == 0) return launch_bias<D, E4M3, NB, 0>(a, sms, st);
  return a.R <= kCacheBiasExact ? launch_bias<D, E4M3, NB, 1>(a, sms, st) : launch_bias<D, E4M3, NB, 2>(a, sms, st);
}

template <int D, bool E4M3>
cudaError_t launch_d(CacheAttnArgs &a, int sms, cudaStream_t st) {
  return a.rows <= 8 ? launch_nb<D, E4M3, 1>(a, sms, st) : launch_nb<D, E4M3, 2>(a, sms, st);
}

}  // namespace

size_t cache_attn_part_floats(int d, int T, int G, int sms) {
  const int nb = (long long)T * G <= 8 ? 1 : 2;
  const int D = (d + 31) / 32 * 32;
  return size_t(2) * sms * cta_per_sm(nb) * (8 * nb) * (D + 2);
}

cudaError_t launch_attn_cache(CacheAttnArgs a, int e4m3, int sms, cudaStream_t st) {
  const int D = (a.d + 31) / 32;
  if (e4m3)
    return D == 1 ? launch_d<32, true>(a, sms, st)
                  : (D == 2 ? launch_d<64, true>(a, sms, st)
                            : (D == 3 ? launch_d<96, true>(a, sms, st) : launch_d<128, true>(a, sms, st)));
  return D == 1 ? launch_d<32, false>(a, sms, st)
                : (D == 2 ? launch_d<64, false>(a, sms, st)
                          : (D == 3 ? launch_d<96, false>(a, sms, st) : launch_d<128, false>(a, sms, st)));
}

}  // namespace fb
