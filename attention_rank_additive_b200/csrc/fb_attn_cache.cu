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
// uses the same one, so each lane loads 16 neighbouring bytes of a row straight
// into the registers that feed the tensor cores: no shared memory, no barrier
// between warps, and every sector of a row is read whole by one instruction.
// The same swap halves the idle rows for a single token (8 columns, not 16
// rows). P^T is S^T's accumulator after one 8x8 transpose (movmatrix).
//
// Work is dealt out by keys: all blocks of keys of all (sequence, head) items,
// as the lengths on the device say, are numbered through and each CTA takes an
// equal run of them. An item that crosses CTAs leaves partial (O, max, sum)
// rows in the workspace; the last of its CTAs to arrive adds them up in CTA
// order, so the result does not depend on who arrives last.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "fb_attn_cache.h"
#include "fb_internal.h"
#include "fb_ptx.cuh"

namespace fb {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 4;

__device__ __forceinline__ void mma_bf16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
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
// 2^e for an integer e, clamped to the normal range.
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(uint32_t(min(max(e, -126), 127) + 127) << 23); }

// N words (1, 2, 4 or a sum of those) from an address aligned to the widest of them.
template <int N>
__device__ __forceinline__ void load_words(const void *p, uint32_t *w) {
  if constexpr (N == 4) {
    const uint4 u = __ldg(static_cast<const uint4 *>(p));
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = __ldg(static_cast<const uint2 *>(p));
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = __ldg(static_cast<const uint32_t *>(p));
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
  // 16-key blocks per warp and step: about 8 KB of loads in flight per warp
  static constexpr int KM = D * ES >= 192 ? 1 : (D * ES >= 96 ? 2 : 4);
  // d of value v (0 .. D/8 - 1) of lane group g
  static __device__ __forceinline__ int vd(int g, int v) {
    constexpr int per0 = VL0 * 4 / ES;  // values of a piece per lane
    if constexpr (D == 96) return v < per0 ? g * per0 + v : 64 + g * (per0 / 2) + (v - per0);
    return (v / per0) * (8 * per0) + g * per0 + v % per0;
  }
};

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

// Non-finite values in a word of value codes, the word without them, and one such value (0 for a finite one).
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
template <bool E4M3>
__device__ __forceinline__ bool odd_word(uint32_t w) {
  return even_word<E4M3>(w) != w;
}
template <bool E4M3>
__device__ __forceinline__ float odd_value(const uint8_t *row, int at) {
  if constexpr (E4M3) {
    return (row[at] & 0x7fu) == 0x7fu ? __uint_as_float(0x7fffffffu) : 0.f;
  } else {
    const uint32_t v = reinterpret_cast<const uint16_t *>(row)[at];
    return (v & 0x7f80u) == 0x7f80u ? __uint_as_float(v << 16) : 0.f;
  }
}

// Value dd of one output row, from the sums relative to exp(top); row t of a sequence that brings fewer tokens is 0.
__device__ __forceinline__ void write_row(const CacheAttnArgs &a, const Seq &s, long long row, int t, int dd, float top,
                                          float sum, float val) {
  const bool none = t >= s.count || top == -INFINITY;
  if (dd < a.d) a.O[row * a.d + dd] = __float2bfloat16_rn(none ? 0.f : val / sum);
  if (dd == 0) a.LSE[row] = none ? -INFINITY : top + logf(sum);
}

template <int D, bool E4M3, int NB, int BIAS>
struct Smem {
  float o[kWarps][8 * NB][D];
  float m[kWarps][8 * NB], l[kWarps][8 * NB], e[kWarps][8 * NB];
  uint4 fq[BIAS == 2 ? NB * 8 * 32 : 1];  // phi_q as matrix operands: [block][16 ranks][lane]
  int last;
};

template <int D, bool E4M3, int NB, int BIAS>
__global__ void __launch_bounds__(kWarps * 32, NB == 1 ? 3 : 2) attn_cache_kernel(const CacheAttnArgs a) {
  using L = Lay<D, E4M3>;
  constexpr int KM = L::KM, KS = D / 16, ROWS = 8 * NB;
  constexpr int BK = kWarps * 16 * KM;  // keys per block
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto &sm = *reinterpret_cast<Smem<D, E4M3, NB, BIAS> *>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  griddep_wait();

  // ---- this CTA's run of blocks, [lo, hi) of all blocks of all items
  const int HC = a.H * a.chunks;
  auto blocks_of = [&](int b) {
    const Seq s = sequence(a, b, false);
    return max(1, (s.len + BK - 1) / BK);
  };
  long long total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) total += __reduce_add_sync(0xffffffffu, b0 + lane < a.B ? blocks_of(b0 + lane) : 0);
  total *= HC;
  const long long N = min((long long)gridDim.x, total);  // CTAs with work
  if (blockIdx.x >= N) return;
  auto first_block = [&](long long c) { return c * total / N; };
  auto owner = [&](long long x) {  // the CTA whose run holds block x
    long long c = x * N / total;
    while (c + 1 < N && first_block(c + 1) <= x) ++c;
    while (c > 0 && first_block(c) > x) --c;
    return int(c);
  };
  const long long lo = first_block(blockIdx.x), hi = first_block(blockIdx.x + 1);
  int b = 0;
  long long bstart = 0;  // the first block of sequence b
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int mine = b0 + lane < a.B ? blocks_of(b0 + lane) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const bool past = b0 + lane >= a.B || bstart + (long long)incl * HC > lo;
    const unsigned vote = __ballot_sync(0xffffffffu, past);
    if (vote) {
      const int f = __ffs(vote) - 1;
      b = b0 + f;
      bstart += (long long)(__shfl_sync(0xffffffffu, incl, f) - __shfl_sync(0xffffffffu, mine, f)) * HC;
      break;
    }
    bstart += (long long)__shfl_sync(0xffffffffu, incl, 31) * HC;
  }

  long long pos = lo;
  while (pos < hi && b < a.B) {
    Seq s = sequence(a, b, true);
    const int nb = max(1, (s.len + BK - 1) / BK);
    if (pos >= bstart + (long long)nb * HC) {
      bstart += (long long)nb * HC;
      ++b;
      continue;
    }
    const int item = int((pos - bstart) / nb);
    const int k0 = int((pos - bstart) - (long long)item * nb);
    const int k1 = int(min((long long)nb, k0 + (hi - pos)));
    const int h = item / a.chunks, r0 = (item - h * a.chunks) * ROWS;
    const long long qrow0 = ((long long)b * a.Hq + (long long)h * a.G) * a.T;  // row r of the item is output row qrow0 + r

    // ---- queries as the matrix operand: lane (g, t4) holds row g's values at the d that its key loads have
    uint32_t qf[NB][KS][2];
    float mult[NB][2];  // scale, and the power of two taken out of an fp16 query row
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int r = r0 + n * 8 + g;
      const bool in = r < a.rows;
      const __nv_bfloat16 *q = a.Q + (qrow0 + (in ? r : 0)) * a.d;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        constexpr int per = L::KL * 4 / L::ES;  // values per load and lane
        const int d0 = (k * 4 / per) * (4 * per) + t4 * per + (k * 4) % per;
        uint2 u = make_uint2(0u, 0u);
        if (in && d0 < a.d) u = __ldg(reinterpret_cast<const uint2 *>(q + d0));
        qf[n][k][0] = u.x, qf[n][k][1] = u.y;
      }
      mult[n][0] = mult[n][1] = a.scale;
      if constexpr (E4M3) {
        // fp16 queries: each row times a power of two that brings its largest value to [2^14, 2^15), so that
        // values down to 2^-38 of it keep a bit; bf16's 8 bits fit fp16's 11.
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
        const int e = int(__float_as_uint(top) >> 23) - 127 - 14;
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

    const int *table = a.table + (long long)b * a.max_pages;
    const int jend = min(s.len, k1 * BK);
    const int hk = BIAS ? (a.fk_heads > 1 ? h : 0) : 0;
    int pages[KM];
    auto fetch_pages = [&](int j0) {
#pragma unroll
      for (int mb = 0; mb < KM; ++mb) {
        const int j = j0 + mb * 16;
        pages[mb] = j < jend ? __ldg(table + (j >> a.page_shift)) : 0;
      }
    };
    int j0 = k0 * BK + warp * 16 * KM;
    fetch_pages(j0);
    for (; j0 < jend; j0 += BK) {
      // ---- loads
      uint32_t kr[KM][2][L::KW], vr[KM][4][L::VW];
      uint32_t sk[KM][2], sv[KM][2];
      float fk[KM][2][BIAS == 1 ? 4 : 1];
      int kpos[KM][2];
      bool alive[KM];
      long long prow[KM];
#pragma unroll
      for (int mb = 0; mb < KM; ++mb) {
        alive[mb] = j0 + mb * 16 < jend;
        if (alive[mb] && (pages[mb] < 0 || pages[mb] >= a.num_pages)) {
          if (lane == 0) atomicOr(a.flags, kFlagRange);
          alive[mb] = false;
        }
        prow[mb] = (((long long)pages[mb] * a.H + h) << a.page_shift) + ((j0 + mb * 16) & ((1 << a.page_shift) - 1));
        const uint8_t *kb = static_cast<const uint8_t *>(a.kp) + prow[mb] * (a.d * L::ES);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int jj = g + 8 * i;
          const bool in = alive[mb] && j0 + mb * 16 + jj < s.len;
#pragma unroll
          for (int c = 0; c < L::KW / L::KL; ++c) {
            constexpr int per = L::KL * 4 / L::ES;
            const int d0 = c * 4 * per + t4 * per;
#pragma unroll
            for (int w = 0; w < L::KL; ++w) kr[mb][i][c * L::KL + w] = 0u;
            if (in && d0 < a.d) load_words<L::KL>(kb + (jj * a.d + d0) * L::ES, &kr[mb][i][c * L::KL]);
          }
          if constexpr (E4M3) {
            sk[mb][i] = in ? __ldg(a.ks + prow[mb] + jj) : 127u;
            sv[mb][i] = in ? __ldg(a.vs + prow[mb] + jj) : 127u;
          }
        }
      }
#pragma unroll
      for (int mb = 0; mb < KM; ++mb) {
        const uint8_t *vb = static_cast<const uint8_t *>(a.vp) + prow[mb] * (a.d * L::ES);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int jj = 2 * t4 + (i & 1) + 8 * (i >> 1);
          const bool in = alive[mb] && j0 + mb * 16 + jj < s.len;
#pragma unroll
          for (int w = 0; w < L::VW; ++w) vr[mb][i][w] = 0u;
          constexpr int per = L::VL0 * 4 / L::ES;
          constexpr int pieces = D == 96 ? 1 : L::VW / L::VL0;
#pragma unroll
          for (int c = 0; c < pieces; ++c) {
            const int d0 = c * 8 * per + g * per;
            if (in && d0 < a.d) load_words<L::VL0>(vb + (jj * a.d + d0) * L::ES, &vr[mb][i][c * L::VL0]);
          }
          if constexpr (D == 96) {
            const int d0 = 64 + g * (per / 2);
            if (in && d0 < a.d) load_words<L::VL0 / 2>(vb + (jj * a.d + d0) * L::ES, &vr[mb][i][L::VL0]);
          }
        }
      }
      const bool tail = j0 + 16 * KM > s.prefix;  // drafted keys, or rows past the end
#pragma unroll
      for (int mb = 0; mb < KM; ++mb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = j0 + mb * 16 + g + 8 * i;
          kpos[mb][i] = j;
          if constexpr (BIAS != 0) {
            if (j >= s.prefix) kpos[mb][i] = j < s.len ? new_position(a, b, s, j - s.prefix) : 0;
            if (kpos[mb][i] >= a.P) {
              atomicOr(a.flags, kFlagRange);
              kpos[mb][i] = a.P - 1;
            }
          }
          if constexpr (BIAS == 1) {
            const float4 f = __ldg(static_cast<const float4 *>(a.fk) + (long long)hk * a.P + kpos[mb][i]);
            fk[mb][i][0] = f.x, fk[mb][i][1] = f.y, fk[mb][i][2] = f.z, fk[mb][i][3] = f.w;
          }
        }
      fetch_pages(j0 + BK);

      // ---- scores: S^T = K Q^T (16 keys x 8 rows per block)
      float x[KM][NB][4];
#pragma unroll
      for (int mb = 0; mb < KM; ++mb) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[mb][n][i] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t a0, a1, a2, a3;
          if constexpr (E4M3) {
            a0 = e4m3_lo(kr[mb][0][k]), a2 = e4m3_hi(kr[mb][0][k]);
            a1 = e4m3_lo(kr[mb][1][k]), a3 = e4m3_hi(kr[mb][1][k]);
          } else {
            a0 = kr[mb][0][2 * k], a2 = kr[mb][0][2 * k + 1];
            a1 = kr[mb][1][2 * k], a3 = kr[mb][1][2 * k + 1];
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
      // ---- scale and bias
      float bias[KM][NB][BIAS == 2 ? 4 : 1];
      if constexpr (BIAS == 2) {
#pragma unroll
        for (int mb = 0; mb < KM; ++mb)
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) bias[mb][n][i] = 0.f;
        const uint4 *fb = static_cast<const uint4 *>(a.fk) + (long long)hk * a.P * (a.RP / 4) + t4;
        for (int c = 0; c < a.RP / 16; ++c) {
          uint4 f[KM][2];
#pragma unroll
          for (int mb = 0; mb < KM; ++mb)
#pragma unroll
            for (int i = 0; i < 2; ++i) f[mb][i] = __ldg(fb + (long long)kpos[mb][i] * (a.RP / 4) + c * 4);
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            const uint4 q = sm.fq[(n * 8 + c) * 32 + lane];
            // (kh + kl)(qh + ql) without the last 2^-22
#pragma unroll
            for (int mb = 0; mb < KM; ++mb) {
              mma_f16(bias[mb][n], f[mb][0].z, f[mb][1].z, f[mb][0].w, f[mb][1].w, q.x, q.y);
              mma_f16(bias[mb][n], f[mb][0].x, f[mb][1].x, f[mb][0].y, f[mb][1].y, q.z, q.w);
              mma_f16(bias[mb][n], f[mb][0].x, f[mb][1].x, f[mb][0].y, f[mb][1].y, q.x, q.y);
            }
          }
        }
      }
      uint32_t need = 0;
#pragma unroll
      for (int mb = 0; mb < KM; ++mb)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kk = i >> 1, rr = i & 1;
            float f = mult[n][rr];
            if constexpr (E4M3) f *= sk[mb][kk] == 255u ? __uint_as_float(0x7fffffffu) : pow2i(int(sk[mb][kk]) - 127);
            if constexpr (BIAS == 1) {
              float y = fk[mb][kk][0] * fq[n][rr][0];
#pragma unroll
              for (int r = 1; r < 4; ++r) y = fmaf(fk[mb][kk][r], fq[n][rr][r], y);
              x[mb][n][i] = fmaf(x[mb][n][i], f, y);
            } else if constexpr (BIAS == 2) {
              x[mb][n][i] = fmaf(x[mb][n][i], f, bias[mb][n][i]);
            } else {
              x[mb][n][i] *= f;
            }
          }
      if (tail) {
#pragma unroll
        for (int mb = 0; mb < KM; ++mb)
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + mb * 16 + g + 8 * (i >> 1), u = j - s.prefix, t = tok[n][i & 1];
              const bool see = alive[mb] && j < s.len && (u < 0 || (t >= 0 && drafted_visible(a, b, t, u)));
              if (!see) x[mb][n][i] = -INFINITY;
            }
      } else {
#pragma unroll
        for (int mb = 0; mb < KM; ++mb)
          if (!alive[mb]) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) x[mb][n][i] = -INFINITY;
          }
      }
      // ---- running maximum, raised only when a score passes it by more than 8 (exp stays below e^8)
      float top[NB][2];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[n][i] = -INFINITY;
#pragma unroll
          for (int mb = 0; mb < KM; ++mb) top[n][i] = fmaxf(top[n][i], fmaxf(x[mb][n][i], x[mb][n][i + 2]));
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
              const float down = (m[n][i] - mn) * kLog2e;  // -inf at the first
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
        float svf[KM][2];
#pragma unroll
        for (int mb = 0; mb < KM; ++mb)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            svf[mb][i] = sv[mb][i] == 255u ? __uint_as_float(0x7fffffffu) : float(int(sv[mb][i]) - 127);
        uint32_t grow = 0;
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
                const float y = (x[mb][n][2 * kk + i] - mu) * kLog2e;
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
        // weights rounded to bf16 (2^-9 each, independent, next to O's own rounding); their sum stays fp32
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
          for (int mb = 0; mb < KM; ++mb) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[mb][n][i] = ex2_approx((x[mb][n][i] - (i & 1 ? m1 : m0)) * kLog2e);
              l[n][i & 1] += x[mb][n][i];
            }
            pf[mb][n][0] = transpose8x8(pack_bf16x2(x[mb][n][0], x[mb][n][1]));
            pf[mb][n][1] = transpose8x8(pack_bf16x2(x[mb][n][2], x[mb][n][3]));
          }
        }
      }
      // ---- a drafted value that is infinite or NaN must not reach the rows that do not see it (0 * inf): it
      // leaves the product and is added to the rows that do
      if (tail) {
        bool odd = false;
#pragma unroll
        for (int mb = 0; mb < KM; ++mb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int w = 0; w < L::VW; ++w) odd |= odd_word<E4M3>(vr[mb][i][w]);
        if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
          for (int mb = 0; mb < KM; ++mb) {
            if (!alive[mb]) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int w = 0; w < L::VW; ++w) vr[mb][i][w] = even_word<E4M3>(vr[mb][i][w]);
            const uint8_t *vb = static_cast<const uint8_t *>(a.vp) + prow[mb] * (a.d * L::ES);
            for (int jj = 0; jj < 16; ++jj) {
              const int j = j0 + mb * 16 + jj, u = j - s.prefix;
              if (j >= s.len) break;
#pragma unroll
              for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int t = tok[n][i];
                  if (!(u < 0 || (t >= 0 && drafted_visible(a, b, t, u)))) continue;
#pragma unroll
                  for (int v = 0; v < D / 8; ++v) {
                    const int dd = L::vd(g, v);
                    const float bad = dd < a.d ? odd_value<E4M3>(vb, jj * a.d + dd) : 0.f;
                    o[v / 2][n][(v & 1) * 2 + i] += bad;
                  }
                }
            }
          }
        }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int mb = 0; mb < KM; ++mb)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t a0, a1, a2, a3;
          if constexpr (E4M3) {
            const int w = k / 2;
            const uint32_t sel = k & 1 ? 0x7362u : 0x5140u;  // the two keys' bytes side by side
            const uint32_t u = __byte_perm(vr[mb][0][w], vr[mb][1][w], sel);
            const uint32_t v = __byte_perm(vr[mb][2][w], vr[mb][3][w], sel);
            a0 = e4m3_lo(u), a1 = e4m3_hi(u), a2 = e4m3_lo(v), a3 = e4m3_hi(v);
          } else {
            a0 = __byte_perm(vr[mb][0][k], vr[mb][1][k], 0x5410), a1 = __byte_perm(vr[mb][0][k], vr[mb][1][k], 0x7632);
            a2 = __byte_perm(vr[mb][2][k], vr[mb][3][k], 0x5410), a3 = __byte_perm(vr[mb][2][k], vr[mb][3][k], 0x7632);
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

    // ---- the warps' parts of the segment
    __syncthreads();  // the last segment's readers of shared memory are done
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[n][i];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        const int row = n * 8 + 2 * t4 + i;
        if (g == 0) sm.m[warp][row] = m[n][i], sm.l[warp][row] = sum, sm.e[warp][row] = E4M3 ? ex[n][i] : 0.f;
#pragma unroll
        for (int v = 0; v < D / 8; ++v) sm.o[warp][row][L::vd(g, v)] = o[v / 2][n][(v & 1) * 2 + i];
      }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == nb;
    const int nrows = min(ROWS, a.rows - r0);
    constexpr long long kSlot = ROWS * (D + 2);
    float *slot = a.part + (2ll * blockIdx.x + (k0 == 0)) * kSlot;
    for (int i = threadIdx.x; i < nrows * D; i += kWarps * 32) {
      const int row = i / D, dd = i % D;
      float top = sm.m[0][row];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm.m[w][row]);
      float sum = 0.f, val = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (sm.m[w][row] == -INFINITY) continue;
        const float y = (sm.m[w][row] - top) * kLog2e;
        sum += sm.l[w][row] * ex2_approx(y);
        val += sm.o[w][row][dd] * ex2_approx(y + sm.e[w][row]);
      }
      if (whole) {
        write_row(a, s, qrow0 + r0 + row, (r0 + row) % a.T, dd, top, sum, val);
      } else {
        slot[row * (D + 2) + dd] = val;
        if (dd == 0) slot[row * (D + 2) + D] = top, slot[row * (D + 2) + D + 1] = sum;
      }
    }
    if (!whole) {
      const long long start = bstart + (long long)item * nb;
      const int c0 = owner(start), c1 = owner(start + nb - 1);
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
            if (mc == -INFINITY) continue;
            const float sc = __ldcg(p + D + 1), vc = __ldcg(p + dd);
            const float mn = fmaxf(top, mc);
            const float f0 = ex2_approx((top - mn) * kLog2e), f1 = ex2_approx((mc - mn) * kLog2e);
            sum = sum * f0 + sc * f1;
            val = val * f0 + vc * f1;
            top = mn;
          }
          write_row(a, s, qrow0 + r0 + row, (r0 + row) % a.T, dd, top, sum, val);
        }
        if (threadIdx.x == 0) a.counters[c0] = 0u;  // for the next call
      }
    }
    pos += k1 - k0;
  }
}

template <int D, bool E4M3, int NB>
cudaError_t launch_nb(const CacheAttnArgs &a, int grid, cudaStream_t st) {
  const int bias = a.R == 0 ? 0 : (a.R <= kCacheBiasExact ? 1 : 2);
  void (*k)(const CacheAttnArgs) = bias == 0 ? attn_cache_kernel<D, E4M3, NB, 0>
                                             : (bias == 1 ? attn_cache_kernel<D, E4M3, NB, 1> : attn_cache_kernel<D, E4M3, NB, 2>);
  const size_t smem = bias == 2 ? sizeof(Smem<D, E4M3, NB, 2>) : sizeof(Smem<D, E4M3, NB, 0>);
  static_assert(sizeof(Smem<D, E4M3, NB, 2>) <= 48 * 1024, "shared memory without opting in");
  return launch_programmatic(k, dim3(unsigned(grid)), dim3(kWarps * 32), smem, st, a);
}

template <int D, bool E4M3>
cudaError_t launch_d(CacheAttnArgs &a, int sms, cudaStream_t st) {
  constexpr int BK = kWarps * 16 * Lay<D, E4M3>::KM;
  const int nb = a.rows <= 8 ? 1 : 2;
  a.chunks = (a.rows + 8 * nb - 1) / (8 * nb);
  const long long most = (long long)a.B * a.H * a.chunks * ((((long long)a.max_pages << a.page_shift) + BK - 1) / BK);
  const int grid = int(std::min<long long>(most, (long long)sms * (nb == 1 ? 3 : 2)));
  return nb == 1 ? launch_nb<D, E4M3, 1>(a, grid, st) : launch_nb<D, E4M3, 2>(a, grid, st);
}

}  // namespace

size_t cache_attn_part_floats(int d, int T, int G, int sms) {
  const int nb = (long long)T * G <= 8 ? 1 : 2;
  const int D = (d + 31) / 32 * 32;
  return size_t(2) * sms * (nb == 1 ? 3 : 2) * (8 * nb) * (D + 2);
}

cudaError_t launch_attn_cache(CacheAttnArgs a, int e4m3, int sms, cudaStream_t st) {
  const int D = (a.d + 31) / 32;
  if (e4m3)
    return D == 1 ? launch_d<32, true>(a, sms, st)
                  : (D == 2 ? launch_d<64, true>(a, sms, st) : (D == 3 ? launch_d<96, true>(a, sms, st) : launch_d<128, true>(a, sms, st)));
  return D == 1 ? launch_d<32, false>(a, sms, st)
                : (D == 2 ? launch_d<64, false>(a, sms, st) : (D == 3 ? launch_d<96, false>(a, sms, st) : launch_d<128, false>(a, sms, st)));
}

}  // namespace fb
