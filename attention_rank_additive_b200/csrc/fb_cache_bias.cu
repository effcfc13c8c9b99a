// fb_cache_bias.cu -- bias factors laid out once for attention over a cache,
// and the entry points of that attention (argument checks before any launch).
//
// Ranks up to 4 are kept in fp32, four values a position, and multiplied on the
// CUDA cores: a position factor such as ALiBi's (-m i, m)(1, j) cancels to a few
// units out of m i, which needs every bit of the products.
//
// Larger ranks go to the tensor cores as x = hi + lo in fp16 (22 bits) and three
// products, (qh + ql)(kh + kl) - ql kl. fp16's range is met by balancing each
// column first: q's column r times 2^-c and k's times 2^c with c half the
// difference of their largest exponents leaves the product alone and gives both
// the same size, so a column overflows only where the bias itself passes 2^30.
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "fb_attn_cache.h"
#include "fb_internal.h"
#include "fb_ptx.cuh"

namespace fb {
namespace {

constexpr int kMaxRank = 128;
constexpr size_t kTopBytes = 2 * kMaxRank * 4;     // largest magnitudes of q's and k's columns
constexpr size_t kCounterBytes = 4096;             // work-item counters of the attention kernel
constexpr int kMaxCtas = int(kCounterBytes / 4);

int padded(int R) { return (R + 15) / 16 * 16; }

__global__ void __launch_bounds__(256) bias_top_kernel(int R, long long rows_q, long long rows_k, const float *q,
                                                       const float *k, unsigned *top) {
  // thread: one column of a run of rows; both sides in turn
  griddep_wait();
  const int c = threadIdx.x % R, per = blockDim.x / R;
  const int rr = threadIdx.x / R;
  if (rr >= per) return;
  for (int side = 0; side < 2; ++side) {
    const float *x = side ? k : q;
    const long long rows = side ? rows_k : rows_q;
    float m = 0.f;
    for (long long i = blockIdx.x * (long long)per + rr; i < rows; i += (long long)gridDim.x * per) {
      const float v = fabsf(x[i * R + c]);
      if (v < INFINITY) m = fmaxf(m, v);
    }
    if (m > 0.f) atomicMax(top + side * kMaxRank + c, __float_as_uint(m));
  }
}

__device__ __forceinline__ int exponent(unsigned bits) { return max(int(bits >> 23), 1) - 127; }

// One thread: one group of four ranks of a row, written as 4 hi and 4 lo fp16 values (16 bytes).
__global__ void __launch_bounds__(256) bias_split_kernel(int R, int RP, long long rows_q, long long rows_k,
                                                         const float *q, const float *k, const unsigned *top,
                                                         uint4 *out, int *flags) {
  griddep_wait();
  const int groups = RP / 4;
  const long long i = blockIdx.x * 256ll + threadIdx.x;
  if (i >= (rows_q + rows_k) * groups) return;
  const long long row = i / groups;
  const int r0 = int(i - row * groups) * 4;
  const bool side = row >= rows_q;
  const float *x = side ? k + (row - rows_q) * R : q + row * R;
  uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
  bool over = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = r0 + j;
    if (r >= R) break;
    const unsigned tq = top[r], tk = top[kMaxRank + r];
    // a column that is zero on one side adds nothing: the other side is brought to 1, so that it does not overflow
    int c = tq && tk ? (exponent(tq) - exponent(tk)) / 2 : (tq ? exponent(tq) : (tk ? -exponent(tk) : 0));
    c = side ? c : -c;
    float v = ldexpf(x[r], c);
    if (!(fabsf(v) <= 65504.f)) {
      over = true;
      if (v == v) v = copysignf(65504.f, v);
    }
    const __half h = __float2half_rn(v);
    const __half l = __float2half_rn(v - __half2float(h));
    hi[j / 2] |= uint32_t(__half_as_ushort(h)) << (16 * (j & 1));
    lo[j / 2] |= uint32_t(__half_as_ushort(l)) << (16 * (j & 1));
  }
  if (over) atomicOr(flags, kFlagRange);
  out[i] = make_uint4(hi[0], hi[1], lo[0], lo[1]);
}

__global__ void __launch_bounds__(256) bias_exact_kernel(int R, long long rows_q, long long rows_k, const float *q,
                                                         const float *k, float4 *out) {
  griddep_wait();
  const long long row = blockIdx.x * 256ll + threadIdx.x;
  if (row >= rows_q + rows_k) return;
  const float *x = row >= rows_q ? k + (row - rows_q) * R : q + row * R;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (r < R) v[r] = x[r];
  out[row] = make_float4(v[0], v[1], v[2], v[3]);
}

int sm_count() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return std::min(n, kMaxCtas / 4);
}

bool sizes_ok(int B, int Hq, int H, int T, int d) {
  return B >= 1 && Hq >= 1 && H >= 1 && T >= 1 && Hq % H == 0 && d >= 16 && d <= 128 && d % 16 == 0 && T <= (1 << 16) &&
         Hq <= (1 << 14) && B <= (1 << 20) && (long long)Hq * T <= (1 << 24);
}

// Query rows of an item (heads of a group times tokens) above which the 128-row tiles are used: the other kernel holds two
// blocks of 8 in its registers. With four it took 62 us for 8 trees of 24 rows on contexts up to 2024, 12 heads of 64,
// rank 64, and the tiles 47.
constexpr int kTileRows = 16;

}  // namespace
}  // namespace fb

using namespace fb;

extern "C" {

size_t fb_cache_bias_bytes(int Hq, int H, int P, int R) {
  if (Hq < 1 || H < 1 || P < 1 || R < 1 || R > kMaxRank) return 0;
  const size_t rows = (size_t(Hq) + size_t(H)) * size_t(P);
  return R <= kCacheBiasExact ? rows * 16 : kTopBytes + rows * size_t(padded(R)) * 4;
}

int fb_cache_bias_prepare(int Hq, int H, int P, int R, const float *phi_q, const float *phi_k, void *prepared,
                          size_t prepared_bytes, void *stream) {
  if (Hq < 1 || H < 1 || P < 1 || R < 1) return FB_ERR_INVALID_ARG;
  if (R > kMaxRank || (long long)(Hq + (long long)H) * P > (1ll << 36)) return FB_ERR_UNSUPPORTED;
  if (!phi_q || !phi_k || ((reinterpret_cast<uintptr_t>(phi_q) | reinterpret_cast<uintptr_t>(phi_k)) & 3u) != 0)
    return FB_ERR_INVALID_ARG;
  if (!prepared || prepared_bytes < fb_cache_bias_bytes(Hq, H, P, R) || (reinterpret_cast<uintptr_t>(prepared) & 255u) != 0)
    return FB_ERR_WORKSPACE;
  int *flags = device_flags();
  if (!flags) return FB_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long rq = (long long)Hq * P, rk = (long long)H * P;
  cudaError_t e;
  if (R <= kCacheBiasExact) {
    e = launch_programmatic(bias_exact_kernel, dim3(unsigned((rq + rk + 255) / 256)), dim3(256), 0, st, R, rq, rk, phi_q,
                            phi_k, static_cast<float4 *>(prepared));
  } else {
    unsigned *top = static_cast<unsigned *>(prepared);
    if (cudaMemsetAsync(top, 0, kTopBytes, st) != cudaSuccess) return FB_ERR_CUDA;
    e = launch_programmatic(bias_top_kernel, dim3(592), dim3(256), 0, st, R, rq, rk, phi_q, phi_k, top);
    if (e == cudaSuccess) {
      const int RP = padded(R);
      const long long blocks = ((rq + rk) * (RP / 4) + 255) / 256;
      if (blocks > 0x7fffffffll) return FB_ERR_UNSUPPORTED;
      e = launch_programmatic(bias_split_kernel, dim3(unsigned(blocks)), dim3(256), 0, st, R, RP, rq, rk, phi_q, phi_k,
                              static_cast<const unsigned *>(top),
                              reinterpret_cast<uint4 *>(static_cast<uint8_t *>(prepared) + kTopBytes), flags);
    }
  }
  return e == cudaSuccess ? FB_OK : FB_ERR_CUDA;
}

size_t fb_attn_cache_workspace_bytes(int B, int Hq, int H, int T, int d) {
  if (!sizes_ok(B, Hq, H, T, d)) return 0;
  size_t part = cache_attn_part_floats(d, T, Hq / H, sm_count()) * 4;
  if (Hq / H * T > kTileRows) part = std::max(part, cache_tile_part_floats(d, sm_count()) * 4);
  return kCounterBytes + (part + 255) / 256 * 256;
}

int fb_attn_cache_fwd(int cache_dt, int B, int Hq, int H, int T, int d, const void *Q, const void *k_pages,
                      const void *v_pages, const uint8_t *k_scale, const uint8_t *v_scale, int num_pages, int page_size,
                      const int32_t *block_table, int max_pages, const int32_t *prefix, const int32_t *counts,
                      const uint32_t *tree_mask, int mask_words, const int32_t *depths, int R, int P, int phi_q_heads,
                      int phi_k_heads, const void *prepared_bias, float scale, void *O, float *LSE, void *workspace,
                      size_t workspace_bytes, void *stream) {
  if (cache_dt != FB_BF16 && cache_dt != FB_E4M3) return FB_ERR_UNSUPPORTED;
  if (B < 1 || Hq < 1 || H < 1 || T < 1 || num_pages < 1 || max_pages < 1) return FB_ERR_INVALID_ARG;
  if (Hq % H != 0) return FB_ERR_INVALID_ARG;
  if (!cache_dims_ok(d, page_size) || !sizes_ok(B, Hq, H, T, d)) return FB_ERR_UNSUPPORTED;
  if (!Q || !k_pages || !v_pages || !block_table || !prefix || !O || !LSE) return FB_ERR_INVALID_ARG;
  if (cache_dt == FB_E4M3 && (!k_scale || !v_scale)) return FB_ERR_INVALID_ARG;
  const uintptr_t wide = reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(k_pages) |
                         reinterpret_cast<uintptr_t>(v_pages) | reinterpret_cast<uintptr_t>(O) |
                         reinterpret_cast<uintptr_t>(prepared_bias) | reinterpret_cast<uintptr_t>(k_scale) |
                         reinterpret_cast<uintptr_t>(v_scale);
  const uintptr_t narrow = reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(prefix) |
                           reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(tree_mask) |
                           reinterpret_cast<uintptr_t>(depths) | reinterpret_cast<uintptr_t>(LSE);
  if (wide % 16 != 0 || narrow % 4 != 0) return FB_ERR_INVALID_ARG;
  if (tree_mask && (long long)mask_words * 32 < T) return FB_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FB_ERR_INVALID_ARG;
  if (R < 0 || R > kMaxRank) return FB_ERR_UNSUPPORTED;
  if (R > 0 && (!prepared_bias || P < 1 || (phi_q_heads != 1 && phi_q_heads != Hq) ||
                (phi_k_heads != 1 && phi_k_heads != H)))
    return FB_ERR_INVALID_ARG;
  if ((long long)max_pages * page_size > (1ll << 31) - 4096) return FB_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < fb_attn_cache_workspace_bytes(B, Hq, H, T, d) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return FB_ERR_WORKSPACE;
  int *flags = device_flags();
  if (!flags) return FB_ERR_CUDA;

  CacheAttnArgs a{};
  a.Q = static_cast<const __nv_bfloat16 *>(Q);
  a.kp = k_pages, a.vp = v_pages, a.ks = k_scale, a.vs = v_scale;
  a.table = block_table, a.prefix = prefix, a.counts = counts, a.depths = depths;
  a.mask = tree_mask, a.mask_words = mask_words;
  a.O = static_cast<__nv_bfloat16 *>(O), a.LSE = LSE;
  a.counters = static_cast<unsigned *>(workspace);
  a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kCounterBytes);
  a.B = B, a.Hq = Hq, a.H = H, a.G = Hq / H, a.T = T, a.d = d, a.rows = a.G * T;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  a.num_pages = num_pages, a.max_pages = max_pages;
  a.scale = scale;
  a.R = R, a.P = P, a.fq_heads = phi_q_heads, a.fk_heads = phi_k_heads;
  if (R > 0) {
    const uint8_t *base = static_cast<const uint8_t *>(prepared_bias);
    const size_t row = R <= kCacheBiasExact ? 16 : size_t(padded(R)) * 4;
    if (R > kCacheBiasExact) base += kTopBytes;
    a.RP = padded(R);
    a.fq = base;
    a.fk = base + size_t(phi_q_heads) * P * row;
  }
  a.flags = flags;
  const cudaError_t e = (a.rows > kTileRows ? launch_attn_cache_tile : launch_attn_cache)(
      a, cache_dt == FB_E4M3, sm_count(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FB_OK : FB_ERR_CUDA;
}

}  // extern "C"
