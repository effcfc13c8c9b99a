// fb_rope.cu -- rotary positions: queries and keys turned by angles that grow
// with the token's position, their gradient, and the frequency tables.
//
// Pair p of a token at position n turns by the angle n w_p:
//   y_a = f (x_a cos - x_b sin),  y_b = f (x_a sin + x_b cos),
// with (a, b) = (2p, 2p + 1) (interleaved) or (p, p + rot/2) (halves); values
// past the first `rot` of a head are copied. The gradient is the same turn by
// the opposite angle (the transpose of a rotation), times f.
//
// Angles: w_p is kept as 64-bit fixed-point turns, t_p = 2^64 w_p / 2 pi from a
// product of doubles, off by 2^-52 of w_p at most. The low 64 bits of n t_p are
// then the fraction of a turn that the angle has passed, off by n w_p 2^-52 radians
// (2^-21 at position 2^31 for w = 1), and its upper 32 bits go through sincospi in
// fp32, which rounds them to 2^-25 turns: one integer multiply in place of a
// product and a range reduction in fp64.
//
// What bounds it: each value is read and written once (HBM) and costs about
// three operations, while a sine and cosine cost about 40 instructions. So a
// thread computes the V sine/cosine pairs of one token and walks over several
// heads with them; V pairs are two 16-byte loads and two 16-byte stores. The two
// lie half the rotated part apart in either layout (interleaved: V / 2 pairs
// each), so that neighbouring lanes read neighbouring 16 bytes. Measured: prompts of
// 8 x 2048 tokens, 12 + 12 heads of 64, bf16, 21.8 us, 4.6 TB/s. Its 48 registers a
// thread leave 5 blocks on an SM, so 768 blocks are 1.04 waves: 32 warps an SM, which
// wait for their loads most of the time (9 of 15 stall cycles an instruction), not
// HBM's rate, and the last blocks alone.
#include <cmath>

#include "fb_internal.h"
#include "fb_ptx.cuh"

namespace fb {
namespace {

struct RopeTensor {
  const void *x;
  void *y;
  long long xb, xh, xn, yb, yh, yn;  // element strides of batch, head, token
};

struct RopeArgs {
  RopeTensor t[2];  // queries, keys
  int heads[2];
  int B, N, d, rot;
  int units, turn_units;  // work units of a head: those that turn, then those that copy
  int hpt, hgroups;       // heads per thread, groups of heads of a token
  float factor, sign;
  const unsigned long long *turns;
  const int *positions;  // [B or 1][N], or null: 0 .. N - 1
  long long pos_bs;
  int copy;  // values past rot are copied (the output is not the input)
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// One thread: one unit (V pairs, or 2V values to copy) of one token, for up to
// hpt heads. Consecutive threads take the units of a token, then the next
// token's, so that a warp reads whole rows.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
  const unsigned id = blockIdx.x * 256u + threadIdx.x;
  const unsigned tok = id / unsigned(a.units);
  if (tok >= unsigned(a.B) * unsigned(a.N)) return;
  const int hg = blockIdx.y;
  const int u = int(id - tok * unsigned(a.units));
  const int b = int(tok / unsigned(a.N));
  const int n = int(tok - unsigned(b) * unsigned(a.N));
  const bool turn = u < a.turn_units;

  int o0, o1;  // offsets of the unit's two vectors in a head
  int nv = 2 * V;  // values to copy (units past the rotated ones)
  float c[V], s[V];
  griddep_wait();
  if (turn) {
    o0 = INTERLEAVED && V == 1 ? 2 * u : u * V;
    o1 = INTERLEAVED && V == 1 ? o0 + 1 : a.rot / 2 + u * V;
    const long long pos = a.positions ? (long long)a.positions[b * a.pos_bs + n] : n;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // interleaved: V / 2 pairs in each vector
      const int p = INTERLEAVED && V > 1 ? (i < V / 2 ? o0 / 2 + i : o1 / 2 + i - V / 2) : u * V + i;
      const unsigned long long frac = a.turns[p] * (unsigned long long)pos;
      // signed upper half, in units of half turns
      const float half_turns = float(int(frac >> 32)) * 4.656612873077393e-10f;
      sincospif(half_turns, &s[i], &c[i]);
      c[i] *= a.factor;
      s[i] *= a.factor * a.sign;
    }
  } else {
    const int c = u - a.turn_units, half = (a.d - a.rot) / 2;
    if (2 * half == a.d - a.rot && half % V == 0) {
      o0 = a.rot + c * V;
      o1 = o0 + half;
    } else {
      o0 = a.rot + c * 2 * V;
      o1 = o0 + V;
      nv = min(2 * V, a.d - o0);
    }
  }
  const int h0 = hg * a.hpt, h1 = min(h0 + a.hpt, a.heads[0] + a.heads[1]);
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const int w = h < a.heads[0] ? 0 : 1;
    const int hh = w ? h - a.heads[0] : h;
    const RopeTensor &t = a.t[w];
    const T *x = static_cast<const T *>(t.x) + b * t.xb + hh * t.xh + n * t.xn;
    T *y = static_cast<T *>(t.y) + b * t.yb + hh * t.yh + n * t.yn;
    if (turn) {
      Vec<T, V> v0 = *reinterpret_cast<const Vec<T, V> *>(x + o0);
      Vec<T, V> v1 = *reinterpret_cast<const Vec<T, V> *>(x + o1);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        T &xa = INTERLEAVED ? (2 * i < V ? v0.v[2 * i] : v1.v[2 * i - V]) : v0.v[i];
        T &xb = INTERLEAVED ? (2 * i + 1 < V ? v0.v[2 * i + 1] : v1.v[2 * i + 1 - V]) : v1.v[i];
        const float fa = to_f32(xa), fb = to_f32(xb);
        xa = from_f32<T>(fa * c[i] - fb * s[i]);
        xb = from_f32<T>(fa * s[i] + fb * c[i]);
      }
      *reinterpret_cast<Vec<T, V> *>(y + o0) = v0;
      *reinterpret_cast<Vec<T, V> *>(y + o1) = v1;
    } else if (nv == 2 * V) {
      const Vec<T, V> v0 = *reinterpret_cast<const Vec<T, V> *>(x + o0);
      const Vec<T, V> v1 = *reinterpret_cast<const Vec<T, V> *>(x + o1);
      *reinterpret_cast<Vec<T, V> *>(y + o0) = v0;
      *reinterpret_cast<Vec<T, V> *>(y + o1) = v1;
    } else {
      for (int i = 0; i < nv; ++i) y[o0 + i] = x[o0 + i];
    }
  }
}

template <typename T, int V>
cudaError_t launch_v(RopeArgs a, int interleaved, cudaStream_t st) {
  a.turn_units = a.rot / 2 / V;
  const int copy_units = a.copy ? (a.d - a.rot + 2 * V - 1) / (2 * V) : 0;
  a.units = a.turn_units + copy_units;
  const long long tokens_units = (long long)a.B * a.N * a.units;
  const int H = a.heads[0] + a.heads[1];
  // Heads per thread, which share one set of sines and cosines (320 instructions for V = 8): as many as leave 148
  // SMs 1024 threads each, at most 16; a single token gets one head per thread. With four full waves of threads asked
  // for instead, a prompt of 8 x 2048 tokens and 24 heads got one head each and took 31 us.
  long long hpt = tokens_units * H / (148ll * 1024);
  a.hpt = int(hpt < 1 ? 1 : (hpt > 16 ? 16 : hpt));
  if (a.hpt > H) a.hpt = H;
  a.hgroups = (H + a.hpt - 1) / a.hpt;
  if (tokens_units > 0xffffff00ll || a.hgroups > 65535) return cudaErrorInvalidValue;
  const long long blocks = (tokens_units + 255) / 256;
  void (*k)(const RopeArgs) = interleaved ? rope_kernel<T, V, true> : rope_kernel<T, V, false>;
  return launch_programmatic(k, dim3(unsigned(blocks), unsigned(a.hgroups)), dim3(256), 0, st, a);
}

// The widest vectors that every address of the call allows.
int vector_width(const RopeArgs &a, int esize) {
  int v = 16 / esize;
  for (; v > 1; v /= 2) {
    bool ok = (a.rot / 2) % v == 0;
    for (int w = 0; w < 2 && ok; ++w) {
      if (a.heads[w] == 0) continue;
      const RopeTensor &t = a.t[w];
      const uintptr_t p = reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y);
      const long long s = t.xb | t.xh | t.xn | t.yb | t.yh | t.yn;
      ok = p % (uintptr_t(v) * esize) == 0 && s % v == 0;
    }
    if (ok) break;
  }
  return v;
}

int rope_call(int dt, int B, int N, int d, int rot, int interleaved, const uint64_t *turns, float factor, float sign,
              const int32_t *positions, int64_t pos_bstride, int Hq, const void *Q, int64_t q_bs, int64_t q_hs,
              int64_t q_ns, void *Qo, int64_t qo_bs, int64_t qo_hs, int64_t qo_ns, int Hk, const void *K,
              int64_t k_bs, int64_t k_hs, int64_t k_ns, void *Ko, int64_t ko_bs, int64_t ko_hs, int64_t ko_ns,
              void *stream) {
  if (dt != FB_BF16 && dt != FB_F32) return FB_ERR_UNSUPPORTED;
  if (B < 1 || N < 1 || d < 1 || Hq < 1 || Hk < 0) return FB_ERR_INVALID_ARG;
  if (rot < 2 || rot > d || rot % 2 != 0) return FB_ERR_INVALID_ARG;
  if (d > 4096 || Hq > 65536 || Hk > 65536) return FB_ERR_UNSUPPORTED;
  if (!turns || !Q || !Qo || (Hk > 0 && (!K || !Ko))) return FB_ERR_INVALID_ARG;
  if (!std::isfinite(factor) || factor == 0.f) return FB_ERR_INVALID_ARG;
  if (pos_bstride < 0 || q_bs < 0 || q_hs < 0 || q_ns < 0 || qo_bs < 0 || qo_hs < 0 || qo_ns < 0)
    return FB_ERR_INVALID_ARG;
  if (Hk > 0 && (k_bs < 0 || k_hs < 0 || k_ns < 0 || ko_bs < 0 || ko_hs < 0 || ko_ns < 0)) return FB_ERR_INVALID_ARG;
  if (Q == Qo && (q_bs != qo_bs || q_hs != qo_hs || q_ns != qo_ns)) return FB_ERR_INVALID_ARG;
  if (Hk > 0 && K == Ko && (k_bs != ko_bs || k_hs != ko_hs || k_ns != ko_ns)) return FB_ERR_INVALID_ARG;
  const unsigned es = dt == FB_BF16 ? 2 : 4;
  uintptr_t al = reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(Qo);
  if (Hk > 0) al |= reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(Ko);
  if (al % es != 0 || reinterpret_cast<uintptr_t>(turns) % 8 != 0 || reinterpret_cast<uintptr_t>(positions) % 4 != 0)
    return FB_ERR_INVALID_ARG;
  RopeArgs a;
  a.t[0] = RopeTensor{Q, Qo, q_bs, q_hs, q_ns, qo_bs, qo_hs, qo_ns};
  a.t[1] = RopeTensor{K, Ko, k_bs, k_hs, k_ns, ko_bs, ko_hs, ko_ns};
  a.heads[0] = Hq, a.heads[1] = Hk;
  a.B = B, a.N = N, a.d = d, a.rot = rot;
  a.factor = factor, a.sign = sign;
  a.turns = reinterpret_cast<const unsigned long long *>(turns);
  a.positions = positions, a.pos_bs = pos_bstride;
  a.copy = rot < d && (Q != Qo || (Hk > 0 && K != Ko));
  a.units = a.turn_units = a.hpt = a.hgroups = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dt == FB_BF16) {
    switch (vector_width(a, 2)) {
      case 8: e = launch_v<__nv_bfloat16, 8>(a, interleaved, st); break;
      case 4: e = launch_v<__nv_bfloat16, 4>(a, interleaved, st); break;
      case 2: e = launch_v<__nv_bfloat16, 2>(a, interleaved, st); break;
      default: e = launch_v<__nv_bfloat16, 1>(a, interleaved, st); break;
    }
  } else {
    switch (vector_width(a, 4)) {
      case 4: e = launch_v<float, 4>(a, interleaved, st); break;
      case 2: e = launch_v<float, 2>(a, interleaved, st); break;
      default: e = launch_v<float, 1>(a, interleaved, st); break;
    }
  }
  return e == cudaSuccess ? FB_OK : (e == cudaErrorInvalidValue ? FB_ERR_UNSUPPORTED : FB_ERR_CUDA);
}

}  // namespace
}  // namespace fb

extern "C" {

int fb_rope_fwd(int dt, int B, int N, int d, int rot, int interleaved, const uint64_t *turns, float factor,
                const int32_t *positions, int64_t pos_bstride, int Hq, const void *Q, int64_t q_bstride,
                int64_t q_hstride, int64_t q_nstride, void *Q_out, int64_t qo_bstride, int64_t qo_hstride,
                int64_t qo_nstride, int Hk, const void *K, int64_t k_bstride, int64_t k_hstride, int64_t k_nstride,
                void *K_out, int64_t ko_bstride, int64_t ko_hstride, int64_t ko_nstride, void *stream) {
  return fb::rope_call(dt, B, N, d, rot, interleaved, turns, factor, 1.f, positions, pos_bstride, Hq, Q, q_bstride,
                       q_hstride, q_nstride, Q_out, qo_bstride, qo_hstride, qo_nstride, Hk, K, k_bstride, k_hstride,
                       k_nstride, K_out, ko_bstride, ko_hstride, ko_nstride, stream);
}

int fb_rope_bwd(int dt, int B, int N, int d, int rot, int interleaved, const uint64_t *turns, float factor,
                const int32_t *positions, int64_t pos_bstride, int Hq, const void *dQ_out, int64_t q_bstride,
                int64_t q_hstride, int64_t q_nstride, void *dQ, int64_t qo_bstride, int64_t qo_hstride,
                int64_t qo_nstride, int Hk, const void *dK_out, int64_t k_bstride, int64_t k_hstride,
                int64_t k_nstride, void *dK, int64_t ko_bstride, int64_t ko_hstride, int64_t ko_nstride,
                void *stream) {
  return fb::rope_call(dt, B, N, d, rot, interleaved, turns, factor, -1.f, positions, pos_bstride, Hq, dQ_out,
                       q_bstride, q_hstride, q_nstride, dQ, qo_bstride, qo_hstride, qo_nstride, Hk, dK_out, k_bstride,
                       k_hstride, k_nstride, dK, ko_bstride, ko_hstride, ko_nstride, stream);
}

int fb_rope_turns_host(int pairs, const double *freq_host, uint64_t *turns_host) {
  if (pairs < 1 || !freq_host || !turns_host) return FB_ERR_INVALID_ARG;
  for (int p = 0; p < pairs; ++p)
    if (!std::isfinite(freq_host[p])) return FB_ERR_INVALID_ARG;
  const double inv_2pi = 0.15915494309189535;
  for (int p = 0; p < pairs; ++p) {
    double t = freq_host[p] * inv_2pi;
    t -= std::floor(t);  // whole turns per position do nothing
    const double scaled = std::ldexp(t, 64);
    turns_host[p] = scaled >= 18446744073709551615.0 ? 0ull : uint64_t(scaled);
  }
  return FB_OK;
}

int fb_rope_frequencies_host(int rot, double base, int scaling, double factor, double trained, double fast,
                             double slow, double *freq_host, double *out_factor_host) {
  if (rot < 2 || rot % 2 != 0 || rot > 4096 || !freq_host) return FB_ERR_INVALID_ARG;
  if (!std::isfinite(base) || base <= 1.0) return FB_ERR_INVALID_ARG;
  if (scaling < FB_ROPE_PLAIN || scaling > FB_ROPE_BANDS) return FB_ERR_UNSUPPORTED;
  if (scaling != FB_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0)) return FB_ERR_INVALID_ARG;
  if (scaling == FB_ROPE_BASE && rot < 4) return FB_ERR_INVALID_ARG;  // the exponent rot / (rot - 2)
  if (scaling == FB_ROPE_YARN || scaling == FB_ROPE_BANDS) {
    if (!std::isfinite(trained) || trained <= 0.0 || !std::isfinite(fast) || !std::isfinite(slow) || slow <= 0.0 ||
        fast <= slow)
      return FB_ERR_INVALID_ARG;
  }
  const double two_pi = 6.283185307179586476925;
  const int pairs = rot / 2;
  double b = base;
  if (scaling == FB_ROPE_BASE) b = base * std::pow(factor, double(rot) / double(rot - 2));
  double lo = 0, hi = 0;
  if (scaling == FB_ROPE_YARN) {
    // the pair whose angle makes `turns` turns over the trained length
    auto pair_of = [&](double turns) {
      return rot * std::log(trained / (turns * two_pi)) / (2.0 * std::log(base));
    };
    lo = std::floor(pair_of(fast));
    hi = std::ceil(pair_of(slow));
    if (lo < 0) lo = 0;
    if (hi > rot - 1) hi = rot - 1;
  }
  for (int p = 0; p < pairs; ++p) {
    const double w = std::pow(b, -2.0 * p / rot);
    double r = w;
    if (scaling == FB_ROPE_LINEAR) {
      r = w / factor;
    } else if (scaling == FB_ROPE_YARN) {
      double ramp = (p - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
      ramp = ramp < 0 ? 0 : (ramp > 1 ? 1 : ramp);
      r = w / factor * ramp + w * (1.0 - ramp);
    } else if (scaling == FB_ROPE_BANDS) {
      const double turns = trained * w / two_pi;  // turns over the trained length
      double keep = (turns - slow) / (fast - slow);
      keep = keep < 0 ? 0 : (keep > 1 ? 1 : keep);
      r = w / factor * (1.0 - keep) + w * keep;
    }
    freq_host[p] = r;
  }
  if (out_factor_host) *out_factor_host = scaling == FB_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return FB_OK;
}

}  // extern "C"
