// fb_call.cpp -- the serving entry points with their arguments as an array of
// 8-byte words: a decode step's calls take a few microseconds in all, half of
// which a foreign-function interface spends on converting 30 arguments singly.
#include <cstring>

#include "../../include/flashbias.h"

namespace {

struct Words {
  const uint64_t *w;
  int i = 0;
  int num() { return static_cast<int>(static_cast<int64_t>(w[i++])); }
  int64_t wide() { return static_cast<int64_t>(w[i++]); }
  float real() {
    double d;
    std::memcpy(&d, &w[i++], sizeof d);
    return static_cast<float>(d);
  }
  template <typename T>
  T *ptr() {
    return reinterpret_cast<T *>(static_cast<uintptr_t>(w[i++]));
  }
};

struct RopeSide {
  int heads;
  const void *x;
  int64_t xb, xh, xn;
  void *y;
  int64_t yb, yh, yn;
  explicit RopeSide(Words &a)
      : heads(a.num()), x(a.ptr<const void>()), xb(a.wide()), xh(a.wide()), xn(a.wide()), y(a.ptr<void>()), yb(a.wide()),
        yh(a.wide()), yn(a.wide()) {}
};

int rope(Words a, bool back) {
  const int dt = a.num(), B = a.num(), N = a.num(), d = a.num(), rot = a.num(), inter = a.num();
  const uint64_t *turns = a.ptr<const uint64_t>();
  const float factor = a.real();
  const int32_t *pos = a.ptr<const int32_t>();
  const int64_t pos_bs = a.wide();
  const RopeSide q(a), k(a);
  void *stream = a.ptr<void>();
  return (back ? fb_rope_bwd : fb_rope_fwd)(dt, B, N, d, rot, inter, turns, factor, pos, pos_bs, q.heads, q.x, q.xb, q.xh,
                                            q.xn, q.y, q.yb, q.yh, q.yn, k.heads, k.x, k.xb, k.xh, k.xn, k.y, k.yb, k.yh,
                                            k.yn, stream);
}

int write(Words a) {
  const int dt = a.num(), cdt = a.num(), B = a.num(), H = a.num(), T = a.num(), d = a.num();
  const void *K = a.ptr<const void>();
  const int64_t kb = a.wide(), kh = a.wide(), kt = a.wide();
  const void *V = a.ptr<const void>();
  const int64_t vb = a.wide(), vh = a.wide(), vt = a.wide();
  void *kp = a.ptr<void>(), *vp = a.ptr<void>();
  uint8_t *ks = a.ptr<uint8_t>(), *vs = a.ptr<uint8_t>();
  const int pages = a.num(), page = a.num();
  const int32_t *table = a.ptr<const int32_t>();
  const int max_pages = a.num();
  const int32_t *starts = a.ptr<const int32_t>(), *counts = a.ptr<const int32_t>();
  return fb_cache_write(dt, cdt, B, H, T, d, K, kb, kh, kt, V, vb, vh, vt, kp, vp, ks, vs, pages, page, table, max_pages,
                        starts, counts, a.ptr<void>());
}

int read(Words a) {
  const int dt = a.num(), cdt = a.num(), B = a.num(), H = a.num(), N = a.num(), d = a.num();
  const void *kp = a.ptr<const void>(), *vp = a.ptr<const void>();
  const uint8_t *ks = a.ptr<const uint8_t>(), *vs = a.ptr<const uint8_t>();
  const int pages = a.num(), page = a.num();
  const int32_t *table = a.ptr<const int32_t>();
  const int max_pages = a.num();
  const int32_t *starts = a.ptr<const int32_t>(), *counts = a.ptr<const int32_t>();
  void *K = a.ptr<void>(), *V = a.ptr<void>();
  return fb_cache_read(dt, cdt, B, H, N, d, kp, vp, ks, vs, pages, page, table, max_pages, starts, counts, K, V,
                       a.ptr<void>());
}

int attend(Words a) {
  const int cdt = a.num(), B = a.num(), Hq = a.num(), H = a.num(), T = a.num(), d = a.num();
  const void *Q = a.ptr<const void>(), *kp = a.ptr<const void>(), *vp = a.ptr<const void>();
  const uint8_t *ks = a.ptr<const uint8_t>(), *vs = a.ptr<const uint8_t>();
  const int pages = a.num(), page = a.num();
  const int32_t *table = a.ptr<const int32_t>();
  const int max_pages = a.num();
  const int32_t *prefix = a.ptr<const int32_t>(), *counts = a.ptr<const int32_t>();
  const uint32_t *mask = a.ptr<const uint32_t>();
  const int words = a.num();
  const int32_t *depths = a.ptr<const int32_t>();
  const int R = a.num(), P = a.num(), fq = a.num(), fk = a.num();
  const void *bias = a.ptr<const void>();
  const float scale = a.real();
  void *O = a.ptr<void>();
  float *LSE = a.ptr<float>();
  void *ws = a.ptr<void>();
  const size_t ws_bytes = static_cast<size_t>(a.wide());
  return fb_attn_cache_fwd(cdt, B, Hq, H, T, d, Q, kp, vp, ks, vs, pages, page, table, max_pages, prefix, counts, mask,
                           words, depths, R, P, fq, fk, bias, scale, O, LSE, ws, ws_bytes, a.ptr<void>());
}

}  // namespace

extern "C" int fb_call(int entry, const uint64_t *words, int count) {
  static const int kCounts[] = {29, 29, 25, 19, 31};  // by fb_entry
  if (entry < 0 || entry > FB_CALL_ATTN_CACHE_FWD) return FB_ERR_UNSUPPORTED;
  if (!words || count != kCounts[entry]) return FB_ERR_INVALID_ARG;
  const Words a{words};
  switch (entry) {
    case FB_CALL_ROPE_FWD: return rope(a, false);
    case FB_CALL_ROPE_BWD: return rope(a, true);
    case FB_CALL_CACHE_WRITE: return write(a);
    case FB_CALL_CACHE_READ: return read(a);
    default: return attend(a);
  }
}
