// fb_cache.cu -- the paged key/value cache: new rows quantised as they are
// written, and rows read back.
//
// A cache is two pools of pages, [pages, heads, page, d], of bf16 or of e4m3
// codes; an e4m3 row carries a power-of-two scale in one byte (E8M0),
//   x ~ code 2^(s - 127),  s - 127 = ceil(log2(amax |x| / 448)), at least -126.
// A power of two makes the division exact, so the one rounding is the code's
// (relative 2^-4, RN), two implementations agree to the bit, and a value read
// back has four significant bits and is exact in bf16, within that type's range.
//
// What should bound both kernels is HBM: each row is read once and written once. A
// long read comes near it (6.0 TB/s). A prompt's 8-bit write does not (3.9 TB/s):
// issue slots are 70 % busy with the maxima, exponents and codes, and what stalls
// most beside that is the latency of the loads. A row is the work of d / 8
// neighbouring lanes (16 bytes of bf16 each), rounded up to a power of two so that
// the row's maximum is a shuffle reduction; consecutive groups of lanes take
// consecutive tokens of one head, which are neighbours in a page, so a warp's
// stores form whole lines.
#include <cuda_fp8.h>

#include "fb_internal.h"
#include "fb_ptx_cache.cuh"

namespace fb {
namespace {

struct CacheArgs {
  const void *src[2];  // write: new K, V (element strides below); read: the pools
  void *dst[2];        // write: the pools; read: K, V [B, H, N, d]
  uint8_t *scale[2];
  long long xb, xh, xn, yb, yh, yn;  // write: strides of new K and new V
  int B, H, N, d, page, shift;       // N: tokens a sequence at most; page = 1 << shift
  int num_pages, max_pages;
  const int *table, *starts, *counts;
  int lanes, lanes_shift;            // lanes of a row, a power of two
  int tok_shift, head_shift;         // a block: 2^tok_shift tokens by 2^head_shift heads, and kSteps such blocks of tokens
  int *flags;
};

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *x) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                             pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float *p, const float *x) {
  *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Row of token (b, position) in head h of the pools, or -1 (flagged) where the
// block table does not lead to a page.
__device__ __forceinline__ long long pool_row(const CacheArgs &a, int b, int h, long long pos) {
  const long long i = pos >> a.shift;
  int page = -1;
  if (pos >= 0 && i < a.max_pages) page = a.table[(long long)b * a.max_pages + i];
  if (page < 0 || page >= a.num_pages) {
    atomicOr(a.flags, kFlagRange);
    return -1;
  }
  return ((long long)page * a.H + h) * a.page + (pos & (a.page - 1));
}

// Which rows this thread's group of lanes works on: n, n + step, ...
constexpr int kSteps = 2;
struct Row {
  int b, h, n, step, lane;
};
__device__ __forceinline__ Row row_of(const CacheArgs &a) {
  Row r;
  const int row = threadIdx.x >> a.lanes_shift;
  r.lane = threadIdx.x & (a.lanes - 1);
  r.b = blockIdx.x;
  r.h = (blockIdx.z << a.head_shift) + (row >> a.tok_shift);
  r.step = 1 << a.tok_shift;
  r.n = blockIdx.y * (kSteps << a.tok_shift) + (row & (r.step - 1));
  return r;
}

// Eight values of a new row as they are loaded.
template <typename T>
struct Eight {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float *x) const {
    if constexpr (sizeof(T) == 4) {
      const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    } else {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// All loads of a block's rows are issued before the first row's maximum is taken, so that a block costs one memory
// latency (one row after the other: 20 us for 8 prompts of up to 2048 tokens of 12 heads of 64 into pages of 16). Two
// rows a thread: with four the registers left fewer threads on an SM and the last wave was longer (18 us, and 133 us in
// place of 127 for the read of 4 x 32768 tokens, 8 heads of 128, whose kernel is laid out alike); now 15.5 us, 3.9 TB/s.
template <typename T, bool E4M3>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheArgs a) {
  const Row r = row_of(a);
  griddep_wait();
  const int count = r.h < a.H ? min(a.counts ? a.counts[r.b] : a.N, a.N) : 0;
  const long long start = a.starts[r.b];
  const bool lane_in = r.lane * 8 < a.d;
  const T *src[2] = {static_cast<const T *>(a.src[0]) + r.b * a.xb + r.h * a.xh + r.lane * 8,
                     static_cast<const T *>(a.src[1]) + r.b * a.yb + r.h * a.yh + r.lane * 8};
  Eight<T> in[kSteps][2];
  long long row[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int n = r.n + i * r.step;
    const bool have = n < count && lane_in;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      in[i][w].clear();
      if (have) in[i][w].load(src[w] + n * (w ? a.yn : a.xn));
    }
    row[i] = -1;
    if (n < count) row[i] = pool_row(a, r.b, r.h, start + n);
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const bool live = row[i] >= 0 && lane_in;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float x[8];
      in[i][w].get(x);
      if constexpr (!E4M3) {
        if (live) store8(static_cast<__nv_bfloat16 *>(a.dst[w]) + row[i] * a.d + r.lane * 8, x);
      } else {
        // the row's largest finite magnitude; infinities, which are rare, are left out in a second look
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 8; k += 2) top = fmax3(top, fabsf(x[k]), fabsf(x[k + 1]));
        if (__any_sync(0xffffffffu, top == INFINITY)) {
          top = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[k]) < INFINITY ? fabsf(x[k]) : 0.f);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
          if (o < a.lanes) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // top = 1.m 2^(f - 127); the scale's exponent is f - 127 - 8, one more where 1.m > 1.75 (448 = 1.75 2^8)
        const uint32_t bits = __float_as_uint(top);
        int e = int(bits >> 23) - 135 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = max(e, -126);
        const float inv = __uint_as_float(uint32_t(127 - e) << 23);
        if (live) {
          const uint32_t lo = e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16);
          const uint32_t hi = e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16);
          *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.dst[w]) + row[i] * a.d + r.lane * 8) = make_uint2(lo, hi);
          if (r.lane == 0) a.scale[w][row[i]] = uint8_t(e + 127);
        }
      }
    }
  }
}

// Eight values of a pool row.
template <bool E4M3>
struct Piece {
  uint4 v;  // bf16, or codes in x, y and the scale byte in z
};
template <bool E4M3>
__device__ __forceinline__ Piece<E4M3> fetch(const void *pool, const uint8_t *scale, long long row, int d, int lane) {
  Piece<E4M3> p;
  if constexpr (E4M3) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(pool) + row * d + lane * 8));
    p.v = make_uint4(u.x, u.y, __ldg(scale + row), 0u);
  } else {
    p.v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(pool) + row * d + lane * 8));
  }
  return p;
}
template <bool E4M3>
__device__ __forceinline__ void expand(const Piece<E4M3> &p, float *x) {
  if constexpr (E4M3) {
    const float scale = scale_value(p.v.z);
    const uint32_t v[2] = {p.v.x, p.v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(v[i / 2] >> (16 * (i % 2))), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      x[2 * i] = f.x * scale;
      x[2 * i + 1] = f.y * scale;
    }
  } else {
    const uint32_t w[4] = {p.v.x, p.v.y, p.v.z, p.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheArgs a) {
  const Row r = row_of(a);
  griddep_wait();
  if (r.h >= a.H || r.lane * 8 >= a.d) return;
  const int count = a.counts ? a.counts[r.b] : a.N;
  const long long start = a.starts ? a.starts[r.b] : 0;
  Piece<E4M3> p[kSteps][2];  // all loads before the first store: a step costs one memory latency
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int n = r.n + i * r.step;
    long long row = -1;
    if (n < count && n < a.N) row = pool_row(a, r.b, r.h, start + n);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      p[i][w].v = make_uint4(0u, 0u, 0u, 0u);
      if (row >= 0) p[i][w] = fetch<E4M3>(a.src[w], a.scale[w], row, a.d, r.lane);
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int n = r.n + i * r.step;
    if (n >= a.N) break;
    const long long out = (((long long)r.b * a.H + r.h) * a.N + n) * a.d + r.lane * 8;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float x[8];
      expand<E4M3>(p[i][w], x);
      store8(static_cast<T *>(a.dst[w]) + out, x);
    }
  }
}

int cache_status(int cache_dt, int B, int H, int N, int d, int num_pages, int page_size, int max_pages,
                 const void *k_pages, const void *v_pages, const void *k_scale, const void *v_scale,
                 const int32_t *table) {
  if (cache_dt != FB_BF16 && cache_dt != FB_E4M3) return FB_ERR_UNSUPPORTED;
  if (B < 1 || H < 1 || N < 1 || num_pages < 1 || max_pages < 1) return FB_ERR_INVALID_ARG;
  if (!cache_dims_ok(d, page_size)) return FB_ERR_UNSUPPORTED;
  if (!k_pages || !v_pages || !table || (cache_dt == FB_E4M3 && (!k_scale || !v_scale))) return FB_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 15u) != 0 ||
      (reinterpret_cast<uintptr_t>(table) & 3u) != 0)
    return FB_ERR_INVALID_ARG;
  return FB_OK;
}

cudaError_t launch_rows(void (*k)(const CacheArgs), CacheArgs &a, cudaStream_t st) {
  a.shift = 0;
  while ((1 << a.shift) < a.page) ++a.shift;
  a.lanes = 1, a.lanes_shift = 0;
  while (a.lanes * 8 < a.d) a.lanes *= 2, ++a.lanes_shift;
  const int rows_shift = 8 - a.lanes_shift;  // rows of a block of 256 threads
  a.tok_shift = 0;
  while (a.tok_shift < rows_shift && (1 << a.tok_shift) < a.N) ++a.tok_shift;
  a.head_shift = rows_shift - a.tok_shift;
  const long long toks = (long long)kSteps << a.tok_shift, heads = 1ll << a.head_shift;
  const long long by = (a.N + toks - 1) / toks, bz = (a.H + heads - 1) / heads;
  if (by > 65535 || bz > 65535) return cudaErrorInvalidValue;
  return launch_programmatic(k, dim3(unsigned(a.B), unsigned(by), unsigned(bz)), dim3(256), 0, st, a);
}

int status_of(cudaError_t e) {
  return e == cudaSuccess ? FB_OK : (e == cudaErrorInvalidValue ? FB_ERR_UNSUPPORTED : FB_ERR_CUDA);
}

}  // namespace

bool cache_dims_ok(int d, int page_size) {
  if (d < 16 || d > 128 || d % 16 != 0) return false;
  return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128 || page_size == 256;
}

}  // namespace fb

using namespace fb;

extern "C" {

int fb_cache_write(int dt, int cache_dt, int B, int H, int T, int d, const void *K, int64_t k_bstride,
                   int64_t k_hstride, int64_t k_tstride, const void *V, int64_t v_bstride, int64_t v_hstride,
                   int64_t v_tstride, void *k_pages, void *v_pages, uint8_t *k_scale, uint8_t *v_scale, int num_pages,
                   int page_size, const int32_t *block_table, int max_pages, const int32_t *starts,
                   const int32_t *counts, void *stream) {
  if (dt != FB_BF16 && dt != FB_F32) return FB_ERR_UNSUPPORTED;
  if (const int s = cache_status(cache_dt, B, H, T, d, num_pages, page_size, max_pages, k_pages, v_pages, k_scale,
                                 v_scale, block_table))
    return s;
  if (!K || !V || !starts) return FB_ERR_INVALID_ARG;
  const int64_t strides[6] = {k_bstride, k_hstride, k_tstride, v_bstride, v_hstride, v_tstride};
  const int vec = dt == FB_BF16 ? 8 : 4;  // 16-byte loads
  for (int64_t s : strides) {
    if (s < 0) return FB_ERR_INVALID_ARG;
    if (s % vec != 0) return FB_ERR_UNSUPPORTED;
  }
  if (((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V)) & 15u) != 0 ||
      ((reinterpret_cast<uintptr_t>(starts) | reinterpret_cast<uintptr_t>(counts)) & 3u) != 0)
    return FB_ERR_INVALID_ARG;
  int *flags = device_flags();
  if (!flags) return FB_ERR_CUDA;
  CacheArgs a{};
  a.src[0] = K, a.src[1] = V, a.dst[0] = k_pages, a.dst[1] = v_pages, a.scale[0] = k_scale, a.scale[1] = v_scale;
  a.xb = k_bstride, a.xh = k_hstride, a.xn = k_tstride, a.yb = v_bstride, a.yh = v_hstride, a.yn = v_tstride;
  a.B = B, a.H = H, a.N = T, a.d = d, a.page = page_size, a.num_pages = num_pages, a.max_pages = max_pages;
  a.table = block_table, a.starts = starts, a.counts = counts, a.flags = flags;
  void (*k)(const CacheArgs) =
      dt == FB_BF16 ? (cache_dt == FB_E4M3 ? cache_write_kernel<__nv_bfloat16, true> : cache_write_kernel<__nv_bfloat16, false>)
                    : (cache_dt == FB_E4M3 ? cache_write_kernel<float, true> : cache_write_kernel<float, false>);
  return status_of(launch_rows(k, a, static_cast<cudaStream_t>(stream)));
}

int fb_cache_read(int dt, int cache_dt, int B, int H, int N, int d, const void *k_pages, const void *v_pages,
                  const uint8_t *k_scale, const uint8_t *v_scale, int num_pages, int page_size,
                  const int32_t *block_table, int max_pages, const int32_t *starts, const int32_t *counts, void *K,
                  void *V, void *stream) {
  if (dt != FB_BF16 && dt != FB_F32) return FB_ERR_UNSUPPORTED;
  if (const int s = cache_status(cache_dt, B, H, N, d, num_pages, page_size, max_pages, k_pages, v_pages, k_scale,
                                 v_scale, block_table))
    return s;
  if (!K || !V) return FB_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V)) & 15u) != 0 ||
      ((reinterpret_cast<uintptr_t>(starts) | reinterpret_cast<uintptr_t>(counts)) & 3u) != 0)
    return FB_ERR_INVALID_ARG;
  int *flags = device_flags();
  if (!flags) return FB_ERR_CUDA;
  CacheArgs a{};
  a.src[0] = k_pages, a.src[1] = v_pages, a.dst[0] = K, a.dst[1] = V;
  a.scale[0] = const_cast<uint8_t *>(k_scale), a.scale[1] = const_cast<uint8_t *>(v_scale);
  a.B = B, a.H = H, a.N = N, a.d = d, a.page = page_size, a.num_pages = num_pages, a.max_pages = max_pages;
  a.table = block_table, a.starts = starts, a.counts = counts, a.flags = flags;
  void (*k)(const CacheArgs) =
      dt == FB_BF16 ? (cache_dt == FB_E4M3 ? cache_read_kernel<__nv_bfloat16, true> : cache_read_kernel<__nv_bfloat16, false>)
                    : (cache_dt == FB_E4M3 ? cache_read_kernel<float, true> : cache_read_kernel<float, false>);
  return status_of(launch_rows(k, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
