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
// Each warp walks over 16-key groups of its own. A lane copies the very bytes
// that it will use itself into a ring in shared memory with cp.async, several
// groups ahead: the ring needs no barrier and has no bank conflicts, and the
// loads in flight cost no registers (held in registers, 32 keys a step, the
// 16-head ALiBi decode step took 142 us, 45 % of the copy rate).
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

#include "fb_attn_cache.cuh"
#include "fb_internal.h"

namespace fb {
namespace {

constexpr int kWarps = 4;
constexpr int kBlockKeys = 16 * kWarps;  // a block: a 16-key group per warp

// CTAs of 128 threads on an SM at most, by blocks of 8 query rows: the registers of O and Q allow no more.
constexpr int cta_per_sm(int NB) { return NB == 1 ? 4 : (NB == 2 ? 3 : 2); }

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
__device__ __forceinline__ void mma_e4m3(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
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
// Wait until at most `left` (0 to 7) of this thread's latest groups are in flight.
__device__ __forceinline__ void copies_wait(int left) {
  switch (left) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
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

__device__ __forceinline__ uint32_t e4m3_codes(const float *x) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3) |
         uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3)) << 16;
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
  // a stage of the ring: K pieces, V pieces, then 32 scale bytes (e4m3) and the keys' factors
  static constexpr int KBYTES = 2 * KW * 4 * 32, VBYTES = 4 * VW * 4 * 32, SBYTES = E4M3 ? 32 : 0;
  static constexpr int BASE = KBYTES + VBYTES + SBYTES;
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
  int last;
  int odd;  // a non-finite value left the products of this segment
  int pad[2];
};

template <int D, bool E4M3, int BIAS>
constexpr int stage_bytes(int RP) {
  return Lay<D, E4M3>::BASE + (BIAS == 1 ? 256 : (BIAS == 2 ? RP / 16 * 2 * 512 : 0));
}

template <int D, bool E4M3, int NB, int BIAS>
__global__ void __launch_bounds__(kWarps * 32, cta_per_sm(NB)) attn_cache_kernel(const CacheAttnArgs a, const int stages) {
  using L = Lay<D, E4M3>;
  constexpr int KS = D / 16, ROWS = 8 * NB;
  constexpr int BK = kBlockKeys;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto &sm = *reinterpret_cast<Smem<NB, BIAS> *>(smem_raw);
  auto &join = *reinterpret_cast<Join<D, NB> *>(smem_raw + sizeof(sm));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  griddep_wait();

  // ---- this CTA's run of blocks of all items
  Walk walk(a, BK, lane);
  if (blockIdx.x >= walk.ctas) return;
  Segment seg;
  while (walk.next(a, seg)) {
    const Seq &s = seg.s;
    const int b = seg.b, nb = seg.blocks, k0 = seg.k0, k1 = seg.k1;
    const int h = seg.item / a.chunks, r0 = (seg.item - h * a.chunks) * ROWS;
    const long long qrow0 = ((long long)b * a.Hq + (long long)h * a.G) * a.T;  // row r of the item is output row qrow0 + r

    // ---- queries as the matrix operand: lane (g, t4) holds row g's values at the d that its key loads have. For an
    // 8-bit cache each row is a power of two times two e4m3 parts, hi + lo / 16: with the row's largest value in
    // (224, 448] hi holds four bits of every value and lo the four that are left of a bf16, so the sum is exact, or
    // off by 2^-23 of the largest value where lo is subnormal. The keys' codes then are operands as they are.
    uint32_t qf[NB][KS][2];  // bf16 pairs; e4m3: [32 d][hi words], then [32 d][lo words]
    float mult[NB][2];       // scale, and the power of two taken out of a query row
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int r = r0 + n * 8 + g;
      const bool in = r < a.rows;
      const __nv_bfloat16 *q = a.Q + (qrow0 + (in ? r : 0)) * a.d;
      uint32_t u[KS][2];
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        constexpr int per = L::KL * 4 / L::ES;  // values per load and lane
        const int d0 = (k * 4 / per) * (4 * per) + t4 * per + (k * 4) % per;
        uint2 v = make_uint2(0u, 0u);
        if (in && d0 < a.d) v = __ldg(reinterpret_cast<const uint2 *>(q + d0));
        u[k][0] = v.x, u[k][1] = v.y;
      }
      mult[n][0] = mult[n][1] = a.scale;
      if constexpr (!E4M3) {
#pragma unroll
        for (int k = 0; k < KS; ++k) qf[n][k][0] = u[k][0], qf[n][k][1] = u[k][1];
      } else {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x0 = fabsf(__uint_as_float(u[k][i] << 16)), x1 = fabsf(__uint_as_float(u[k][i] & 0xffff0000u));
            top = fmaxf(top, fmaxf(x0 < INFINITY ? x0 : 0.f, x1 < INFINITY ? x1 : 0.f));
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // top = 1.m 2^(f - 127), 448 = 1.75 2^8
        const uint32_t bits = __float_as_uint(top);
        const int e = int(bits >> 23) - 135 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
        const float down = pow2i(-e), up = pow2i(e);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          float x[4] = {__uint_as_float(u[k][0] << 16), __uint_as_float(u[k][0] & 0xffff0000u),
                        __uint_as_float(u[k][1] << 16), __uint_as_float(u[k][1] & 0xffff0000u)};
          float lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] *= down;
            if (!(fabsf(x[i]) < INFINITY)) x[i] = __uint_as_float(0x7fffffffu);
          }
          const uint32_t h = e4m3_codes(x);
          const uint32_t l0 = e4m3_lo(h), l1 = e4m3_hi(h);
          const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&l0));
          const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&l1));
          lo[0] = (x[0] - f0.x) * 16.f, lo[1] = (x[1] - f0.y) * 16.f, lo[2] = (x[2] - f1.x) * 16.f, lo[3] = (x[3] - f1.y) * 16.f;
          qf[n][k / 2][k & 1] = h;
          qf[n][KS / 2 + k / 2][k & 1] = e4m3_codes(lo);
        }
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
    __syncthreads();  // sm.odd; and the last segment's readers of shared memory are done
    const int *table = a.table + (long long)b * a.max_pages;
    const int jend = min(s.len, k1 * BK), jstart = k0 * BK + warp * 16;
    const int hk = BIAS ? (a.fk_heads > 1 ? h : 0) : 0;
    const int stage = stage_bytes<D, E4M3, BIAS>(a.RP);
    const uint8_t *ring = smem_raw + sizeof(sm) + warp * stages * stage;
    auto page_of = [&](int j) { return j < jend ? __ldg(table + (j >> a.page_shift)) : 0; };
    int next_page = page_of(jstart);
    // Copy the group at j into ring slot `slot`; false where the table leads nowhere (zeros are copied).
    auto fetch = [&](int j, int slot) {
      const int page = next_page;
      next_page = page_of(j + BK);
      bool alive = j < jend;
      if (alive && (page < 0 || page >= a.num_pages)) {
        if (lane == 0) atomicOr(a.flags, kFlagRange);
        alive = false;
      }
      const long long prow = (((long long)(alive ? page : 0) * a.H + h) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
      const uint32_t dst = smem_u32(ring + slot * stage);
      const uint8_t *kb = static_cast<const uint8_t *>(a.kp) + prow * (a.d * L::ES);
      const uint8_t *vb = static_cast<const uint8_t *>(a.vp) + prow * (a.d * L::ES);
      const int left = alive ? s.len - j : 0;  // keys of the group
      if (left >= 16 && a.d == D) {  // whole rows: fixed offsets from one address a side
        // K: the group's 16 rows lie one after the other, so the lanes take 16-byte chunks in order (a load of 64 bytes
        // of a row brings the whole 128-byte line, half of it twice) and put each where its user will look
        const uint8_t *vl = vb + t4 * (2 * D * L::ES) + g * (L::VL0 * 4);
        const uint32_t vd = dst + L::KBYTES + lane * (L::VL0 * 4);
        constexpr int cpr = D * L::ES / 16;  // chunks of a row
#pragma unroll
        for (int q = 0; q < cpr / 2; ++q) {
          const int at = q * 32 + lane, row = at / cpr, ch = at % cpr;
          const int piece = (row >> 3) * (L::KW / L::KL) + (L::KL == 4 ? ch >> 2 : ch >> 1);
          const int place = (row & 7) * 4 + (L::KL == 4 ? ch & 3 : (ch & 1) * 2);
          copy_whole<4>(dst + (piece * 32 + place) * (L::KL * 4), kb + at * 16);
        }
        constexpr int pieces = D == 96 ? 1 : L::VW / L::VL0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int off = ((i & 1) + 8 * (i >> 1)) * D * L::ES;
#pragma unroll
          for (int c = 0; c < pieces; ++c)
            copy_whole<L::VL0>(vd + i * (L::VW * 4 * 32) + c * (32 * L::VL0 * 4), vl + off + c * (8 * L::VL0 * 4));
          if constexpr (D == 96)
            copy_whole<L::VL0 / 2>(dst + L::KBYTES + i * (L::VW * 4 * 32) + 32 * (L::VL0 * 4) + lane * (L::VL0 * 2),
                                   vb + t4 * (2 * D * L::ES) + off + 64 * L::ES + g * (L::VL0 * 2));
        }
      } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int jj = g + 8 * i;
#pragma unroll
        for (int c = 0; c < L::KW / L::KL; ++c) {
          constexpr int per = L::KL * 4 / L::ES;
          const int d0 = c * 4 * per + t4 * per;
          const bool in = jj < left && d0 < a.d;
          copy_words<L::KL>(dst + ((i * (L::KW / L::KL) + c) * 32 + lane) * (L::KL * 4),
                            in ? kb + (jj * a.d + d0) * L::ES : kb, in);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int jj = 2 * t4 + (i & 1) + 8 * (i >> 1);
        constexpr int per = L::VL0 * 4 / L::ES;
        constexpr int pieces = D == 96 ? 1 : L::VW / L::VL0;
        const uint32_t vdst = dst + L::KBYTES + i * (L::VW * 4 * 32);
#pragma unroll
        for (int c = 0; c < pieces; ++c) {
          const int d0 = c * 8 * per + g * per;
          const bool in = jj < left && d0 < a.d;
          copy_words<L::VL0>(vdst + (c * 32 + lane) * (L::VL0 * 4), in ? vb + (jj * a.d + d0) * L::ES : vb, in);
        }
        if constexpr (D == 96) {
          const int d0 = 64 + g * (per / 2);
          const bool in = jj < left && d0 < a.d;
          copy_words<L::VL0 / 2>(vdst + 32 * (L::VL0 * 4) + lane * (L::VL0 * 2), in ? vb + (jj * a.d + d0) * L::ES : vb, in);
        }
      }
      }
      if constexpr (E4M3) {  // 16 scale bytes of either side: a group starts at a multiple of 16 rows
        if (lane < 2) copy_words<4>(dst + L::KBYTES + L::VBYTES + lane * 16, (lane ? a.vs : a.ks) + prow, alive);
      }
      if constexpr (BIAS != 0) {
        auto position = [&](int jj) {
          const int jk = j + jj;
          if (jj >= left) return 0;
          if (jk >= s.prefix) return new_position(a, b, s, jk - s.prefix);
          if (jk < a.P) return jk;
          atomicOr(a.flags, kFlagRange);
          return a.P - 1;
        };
        if constexpr (BIAS == 1) {
          if (lane < 16)
            copy_words<4>(dst + L::BASE + lane * 16, static_cast<const float4 *>(a.fk) + (long long)hk * a.P + position(lane),
                          lane < left);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 *f = static_cast<const uint4 *>(a.fk) + ((long long)hk * a.P + position(g + 8 * i)) * (a.RP / 4) + t4;
            for (int c = 0; c < a.RP / 16; ++c)
              copy_words<4>(dst + L::BASE + ((c * 2 + i) * 32 + lane) * 16, f + c * 4, g + 8 * i < left);
          }
        }
      }
      return alive;
    };
    unsigned alive_bits = 0;  // bit s: the group in ring slot s
    for (int i = 0; i < stages - 1; ++i) {
      alive_bits |= unsigned(fetch(jstart + i * BK, i)) << i;
      copies_commit();
    }
    int slot = 0;
    for (int j0 = jstart; j0 < jend; j0 += BK) {
      const int ahead = slot == 0 ? stages - 1 : slot - 1;
      const bool there = fetch(j0 + (stages - 1) * BK, ahead);
      copies_commit();
      alive_bits = (alive_bits & ~(1u << ahead)) | unsigned(there) << ahead;
      copies_wait(stages - 1);
      __syncwarp();  // scales and factors were copied by other lanes
      const bool alive = (alive_bits >> slot) & 1u;
      const uint8_t *src = ring + slot * stage;
      const bool tail = j0 + 16 > s.prefix;  // drafted keys, or rows past the end

      // ---- scores: S^T = K Q^T (16 keys x 8 rows per block)
      float x[NB][4], xl[NB][E4M3 ? 4 : 1];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = xl[n][E4M3 ? i : 0] = 0.f;
#pragma unroll
      for (int c = 0; c < L::KW / L::KL; ++c) {
        uint32_t kr[2][L::KL];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          read_words<L::KL>(src + ((i * (L::KW / L::KL) + c) * 32 + lane) * (L::KL * 4), kr[i]);
#pragma unroll
        for (int kk = 0; kk < L::KL / 2; ++kk) {
          const int k = c * (L::KL / 2) + kk;
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            if constexpr (E4M3) {
              mma_e4m3(x[n], kr[0][2 * kk], kr[1][2 * kk], kr[0][2 * kk + 1], kr[1][2 * kk + 1], qf[n][k][0], qf[n][k][1]);
              mma_e4m3(xl[n], kr[0][2 * kk], kr[1][2 * kk], kr[0][2 * kk + 1], kr[1][2 * kk + 1], qf[n][KS / 2 + k][0],
                       qf[n][KS / 2 + k][1]);
            } else {
              mma_bf16(x[n], kr[0][2 * kk], kr[1][2 * kk], kr[0][2 * kk + 1], kr[1][2 * kk + 1], qf[n][k][0], qf[n][k][1]);
            }
          }
        }
      }
      if constexpr (E4M3) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[n][i] = fmaf(xl[n][i], 0.0625f, x[n][i]);
      }
      // ---- scale and bias
      float bias[NB][BIAS == 2 ? 4 : 1];
      if constexpr (BIAS == 2) {
        float low[NB][4];  // the two small products
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) bias[n][i] = low[n][i] = 0.f;
        for (int c = 0; c < a.RP / 16; ++c) {
          uint32_t f[2][4];  // 4 hi, 4 lo
#pragma unroll
          for (int i = 0; i < 2; ++i) read_words<4>(src + L::BASE + ((c * 2 + i) * 32 + lane) * 16, f[i]);
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
      float fk[2][BIAS == 1 ? 4 : 1], skf[2], svf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (BIAS == 1) read_words<4>(src + L::BASE + (g + 8 * i) * 16, reinterpret_cast<uint32_t *>(fk[i]));
        skf[i] = svf[i] = 0.f;
        if constexpr (E4M3) {
          const uint32_t k8 = src[L::KBYTES + L::VBYTES + g + 8 * i], v8 = src[L::KBYTES + L::VBYTES + 16 + g + 8 * i];
          skf[i] = k8 == 255u ? __uint_as_float(0x7fffffffu) : pow2i(int(k8) - 127);
          svf[i] = v8 == 255u ? __uint_as_float(0x7fffffffu) : float(int(v8) - 127);
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
            x[n][i] = fmaf(x[n][i], f, y);
          } else if constexpr (BIAS == 2) {
            x[n][i] = fmaf(x[n][i], f, bias[n][i]);
          } else {
            x[n][i] *= f;
          }
        }
      if (tail || !alive) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j0 + g + 8 * (i >> 1), u = j - s.prefix, t = tok[n][i & 1];
            const bool see = alive && j < s.len && (u < 0 || (t >= 0 && drafted_visible(a, b, t, u)));
            if (!see) x[n][i] = -INFINITY;
          }
      }
      // ---- running maximum, raised only when a score passes it by more than 8 (exp stays below e^8)
      float top[NB][2];
      bool need = false;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[n][i] = fmaxf(x[n][i], x[n][i + 2]);
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
      uint32_t pf[NB][2];
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
            for (int kk = 0; kk < 2; ++kk) {
              const float y = (x[n][2 * kk + i] - mu) * kCacheLog2e;
              x[n][2 * kk + i] = y;
              l[n][i] += ex2_approx(y);
              ytop[n][i] = fmaxf(ytop[n][i], y + svf[kk]);
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
        for (int n = 0; n < NB; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float y = x[n][i];
            x[n][i] = y == -INFINITY ? 0.f : ex2_approx(y + (svf[i >> 1] - ex[n][i & 1]));
          }
          pf[n][0] = transpose8x8(pack_f16x2(x[n][0], x[n][1]));
          pf[n][1] = transpose8x8(pack_f16x2(x[n][2], x[n][3]));
        }
      } else {
        // weights rounded to bf16 (2^-8 at most, each its own, next to O's own rounding); their sum stays fp32
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[n][i] = ex2_approx((x[n][i] - (i & 1 ? m1 : m0)) * kCacheLog2e);
            l[n][i & 1] += x[n][i];
          }
          pf[n][0] = transpose8x8(pack_bf16x2(x[n][0], x[n][1]));
          pf[n][1] = transpose8x8(pack_bf16x2(x[n][2], x[n][3]));
        }
      }
      // ---- O^T += V^T P^T
      constexpr int VP = L::VL0;
      constexpr int pieces = L::VW / VP + (D == 96 ? 1 : 0);
#pragma unroll
      for (int c = 0; c < pieces; ++c) {
        constexpr int full = D == 96 ? 1 : pieces;
        const bool last = c >= full;  // the half piece of D = 96
        uint32_t vr[4][VP];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t *vsrc = src + L::KBYTES + i * (L::VW * 4 * 32);
          if (!last)
            read_words<VP>(vsrc + (c * 32 + lane) * (VP * 4), vr[i]);
          else
            read_words<(VP + 1) / 2>(vsrc + 32 * (VP * 4) + lane * (VP * 2), vr[i]);
        }
        // an infinite or NaN value must not reach the rows that do not see its key (0 * inf): where new tokens are
        // among the keys it leaves the product, and the rows that see it get it back when the segment is joined
        if (tail) {
          bool odd = false;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int w = 0; w < VP; ++w) {
              if (last && w >= VP / 2) continue;
              const uint32_t even = even_word<E4M3>(vr[i][w]);
              odd |= even != vr[i][w];
              vr[i][w] = even;
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
              mma_f16(o[k][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
            else
              mma_bf16(o[k][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
          }
        }
      }
      slot = slot + 1 == stages ? 0 : slot + 1;
      __syncwarp();  // the slot's readers are done before it is filled again
    }
    copies_wait(0);

    __syncthreads();  // the ring becomes the join's memory
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
        if (join.m[w][row] == -INFINITY) continue;
        const float y = (join.m[w][row] - top) * kCacheLog2e;
        sum += join.l[w][row] * ex2_approx(y);
        val += join.o[w][row][dd] * ex2_approx(y + join.e[w][row]);
      }
      if (sm.odd && dd < a.d) val += odd_sum<E4M3>(a, s, b, h, (r0 + row) % a.T, dd, max(k0 * BK, s.prefix / 16 * 16), jend);
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
            if (mc == -INFINITY) continue;
            const float sc = __ldcg(p + D + 1), vc = __ldcg(p + dd);
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
}

template <int D, bool E4M3, int NB, int BIAS>
cudaError_t launch_bias(const CacheAttnArgs &a, int sms, cudaStream_t st) {
  auto *k = attn_cache_kernel<D, E4M3, NB, BIAS>;
  const int stage = kWarps * stage_bytes<D, E4M3, BIAS>(a.RP);
  const int fixed = sizeof(Smem<NB, BIAS>), join = sizeof(Join<D, NB>);
  // CTAs on an SM: as many as leave each a ring of three stages in the 227 KB (1 KB a CTA is the system's); every
  // CTA of the grid is resident, so the equal runs of keys also end together
  int ctas = cta_per_sm(NB) + 1, stages = 0;
  while (stages < 3 && ctas > 1) {
    --ctas;
    stages = std::min(kMaxStages, (227 * 1024 / ctas - 1024 - fixed) / stage);
  }
  stages = std::max(2, stages);
  const int smem = fixed + std::max(join, stages * stage);
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long blocks = std::max<long long>(1, (((long long)a.max_pages << a.page_shift) + kBlockKeys - 1) / kBlockKeys);
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
