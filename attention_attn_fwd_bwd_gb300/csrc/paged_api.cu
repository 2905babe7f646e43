// C entry points of the paged cache: argument checks and launches. Declarations and the meaning
// of every argument are in include/attnfuse.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/attnfuse.h"
#include "launch.h"
#include "paged.cuh"

namespace afx {
namespace {

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return set_last_error(code, buf);
}

int done(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(ATTNFUSE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return set_last_error(ATTNFUSE_OK, "");
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Strides of a 16-byte-accessed tensor: innermost 1, the rest positive multiples of `mult`.
int check_strides(const void* p, const int64_t* st, int n, int mult, const char* name) {
  if (!p) return fail(ATTNFUSE_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, 16)) return fail(ATTNFUSE_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (!st) return fail(ATTNFUSE_ERR_INVALID_ARG, "%s strides are NULL", name);
  if (st[n - 1] != 1) return fail(ATTNFUSE_ERR_INVALID_ARG, "%s: innermost stride must be 1", name);
  for (int i = 0; i < n - 1; ++i)
    if (st[i] <= 0 || st[i] % mult)
      return fail(ATTNFUSE_ERR_INVALID_ARG, "%s: stride[%d] = %lld must be a positive multiple of %d elements",
                  name, i, (long long)st[i], mult);
  return ATTNFUSE_OK;
}

int check_rows(const void* p, const int64_t* st, int n, int mult, int64_t slot, const char* name) {
  int rc = check_strides(p, st, n, 1, name);
  if (rc) return rc;
  if (st[2] != slot)
    return fail(ATTNFUSE_ERR_INVALID_ARG, "%s: slots must be contiguous (stride[2] = %lld, need %lld)", name,
                (long long)st[2], (long long)slot);
  for (int i = 0; i < 2; ++i)
    if (st[i] % mult)
      return fail(ATTNFUSE_ERR_INVALID_ARG, "%s: stride[%d] = %lld must be a multiple of %d (16 bytes)", name, i,
                  (long long)st[i], mult);
  return ATTNFUSE_OK;
}

int check_cache(const attnfuse_paged_cache* c, PagedDev* out) {
  if (!c) return fail(ATTNFUSE_ERR_INVALID_ARG, "cache is NULL");
  if (c->format != ATTNFUSE_CACHE_BF16 && c->format != ATTNFUSE_CACHE_Q4)
    return fail(ATTNFUSE_ERR_INVALID_ARG, "cache format %d", c->format);
  if (c->num_pages <= 0 || c->Hkv <= 0 || c->B <= 0 || c->max_pages <= 0)
    return fail(ATTNFUSE_ERR_INVALID_ARG, "cache sizes must be positive (num_pages=%d Hkv=%d B=%d max_pages=%d)",
                c->num_pages, c->Hkv, c->B, c->max_pages);
  if (c->Hkv > 4096) return fail(ATTNFUSE_ERR_UNSUPPORTED, "Hkv=%d (at most 4096)", c->Hkv);
  if (c->d != 64 && c->d != 128) return fail(ATTNFUSE_ERR_UNSUPPORTED, "head dim %d (need 64 or 128)", c->d);
  if (c->page_size <= 0 || c->page_size % 16 || c->page_size > kPagedMaxPage)
    return fail(ATTNFUSE_ERR_UNSUPPORTED, "page_size %d (need a multiple of 16 up to %d)", c->page_size, kPagedMaxPage);
  if ((int64_t)c->max_pages * c->page_size > kPagedMaxPos)
    return fail(ATTNFUSE_ERR_UNSUPPORTED, "max_pages * page_size = %lld positions (at most %d)",
                (long long)c->max_pages * c->page_size, kPagedMaxPos);
  if (!c->page_table || !aligned(c->page_table, 4))
    return fail(ATTNFUSE_ERR_INVALID_ARG, "page_table NULL or misaligned");
  if (c->B > 1 && c->page_table_stride < 0)
    return fail(ATTNFUSE_ERR_INVALID_ARG, "negative page_table stride");
  memset(out, 0, sizeof(*out));
  int rc;
  if (c->format == ATTNFUSE_CACHE_BF16) {
    if ((rc = check_strides(c->k, c->k_strides, 4, 8, "cache k"))) return rc;
    if ((rc = check_strides(c->v, c->v_strides, 4, 8, "cache v"))) return rc;
  } else {
    if ((rc = check_rows(c->k, c->k_strides, 4, 16, c->d / 2, "cache k"))) return rc;
    if ((rc = check_rows(c->v, c->v_strides, 4, 16, c->d / 2, "cache v"))) return rc;
    if ((rc = check_rows(c->k_scales, c->k_scale_strides, 4, 8, c->d / 32, "cache k_scales"))) return rc;
    if ((rc = check_rows(c->v_scales, c->v_scale_strides, 4, 8, c->d / 32, "cache v_scales"))) return rc;
  }
  const int es = c->format == ATTNFUSE_CACHE_BF16 ? 2 : 1;
  out->k = static_cast<uint8_t*>(c->k);
  out->v = static_cast<uint8_t*>(c->v);
  out->k_sp = c->k_strides[0] * es, out->k_sh = c->k_strides[1] * es, out->k_st = c->k_strides[2] * es;
  out->v_sp = c->v_strides[0] * es, out->v_sh = c->v_strides[1] * es, out->v_st = c->v_strides[2] * es;
  if (c->format == ATTNFUSE_CACHE_Q4) {
    out->ks = static_cast<uint8_t*>(c->k_scales);
    out->vs = static_cast<uint8_t*>(c->v_scales);
    out->ks_sp = c->k_scale_strides[0] * 2, out->ks_sh = c->k_scale_strides[1] * 2;
    out->vs_sp = c->v_scale_strides[0] * 2, out->vs_sh = c->v_scale_strides[1] * 2;
  }
  out->table = c->page_table;
  out->table_stride = c->page_table_stride;
  out->num_pages = c->num_pages;
  out->page_size = c->page_size;
  out->max_pages = c->max_pages;
  out->cap = c->max_pages * c->page_size;
  out->div_mul = ((1ull << 40) + c->page_size - 1) / c->page_size;
  out->B = c->B;
  out->Hkv = c->Hkv;
  return ATTNFUSE_OK;
}

int check_rope(int* mode, float theta) {
  if (*mode == ATTNFUSE_ROPE_AUTO) *mode = ATTNFUSE_ROPE_FUSED;
  if (*mode != ATTNFUSE_ROPE_NONE && *mode != ATTNFUSE_ROPE_FUSED)
    return fail(ATTNFUSE_ERR_UNSUPPORTED, "paged caches rotate on the way: rope_mode NONE or FUSED");
  if (*mode == ATTNFUSE_ROPE_FUSED && (!(theta > 0.f) || !std::isfinite(theta)))
    return fail(ATTNFUSE_ERR_INVALID_ARG, "rope_theta must be positive");
  return ATTNFUSE_OK;
}

// A sum of two doubles, hi the nearest double to it (about 104 bits). Products and sums as in Dekker,
// "A floating-point technique for extending the available precision", 1971, with fused
// multiply-adds, which the compiler is not left to form by itself: all machines get the same bits.
struct Double2 {
  double hi, lo;
};
Double2 sum_of(double a, double b) {  // |a| >= |b| or a = 0
  const double s = a + b;
  return {s, b - (s - a)};
}
Double2 times(Double2 a, Double2 b) {
  const double p = a.hi * b.hi, e = std::fma(a.hi, b.hi, -p);
  return sum_of(p, std::fma(a.hi, b.lo, std::fma(a.lo, b.hi, e)));
}
Double2 inverse(double x) {
  const double q = 1.0 / x, e = std::fma(-q, x, 1.0), s = std::fma(e, q, q);
  return {s, std::fma(e, q, q - s)};
}
Double2 root(Double2 a) {
  const double s = std::sqrt(a.hi);
  return sum_of(s, (std::fma(-s, s, a.hi) + a.lo) / (2.0 * s));
}

// The frequencies of a theta; a thread keeps those of its last call (they cost as much as a launch).
// The kernels multiply them by positions up to 2^24, so a double's 53 bits would leave an angle
// 2^-29 off. Whole turns per position (theta < 0.16) drop out, positions being whole numbers.
const PagedFreqs& paged_freqs(int d, float theta) {
  static thread_local PagedFreqs f;
  static thread_local int have_d = 0;
  static thread_local float have_theta = 0.f;
  if (have_d != d || have_theta != theta) {
    memset(&f, 0, sizeof(f));
    Double2 step = inverse(theta);  // theta^(-2 / d)
    for (int n = d / 2; n > 1; n /= 2) step = root(step);
    Double2 turn = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / (2 pi)
    for (int i = 0; i < d / 2; ++i, turn = times(turn, step)) {
      const Double2 part = sum_of(turn.hi - std::rint(turn.hi), turn.lo);
      f.f[i].x = (float)part.hi;
      const double rest = (part.hi - f.f[i].x) + part.lo;
      f.f[i].y = (float)rest;
      f.f[i].z = (float)(rest - f.f[i].y);
    }
    have_d = d;
    have_theta = theta;
  }
  return f;
}

int check_index(const int32_t* p, bool need, const char* name) {
  if (!p && need) return fail(ATTNFUSE_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, 4)) return fail(ATTNFUSE_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
  return ATTNFUSE_OK;
}

// One thread block per 2 to 32 rows of the call and run of heads: B * N rows stay below 2^31.
int check_n(int B, int N) {
  if (N <= 0) return fail(ATTNFUSE_ERR_INVALID_ARG, "N=%d must be positive", N);
  if ((int64_t)B * N > 0x7fffffff) return fail(ATTNFUSE_ERR_UNSUPPORTED, "B * N too large");
  return ATTNFUSE_OK;
}

}  // namespace
}  // namespace afx

using namespace afx;

extern "C" {

attnfuse_status attnfuse_paged_append(const attnfuse_paged_cache* cache, const void* k,
                                      const int64_t k_strides[4], const void* v,
                                      const int64_t v_strides[4], const int32_t* start,
                                      const int32_t* count, int N, float rope_theta,
                                      attnfuse_rope_mode rope_mode, cudaStream_t stream) {
  PagedAppendParams p;
  memset(&p, 0, sizeof(p));
  int rc, mode = rope_mode;
  if ((rc = check_cache(cache, &p.cache))) return rc;
  if ((rc = check_n(cache->B, N))) return rc;
  if ((rc = check_strides(k, k_strides, 4, 8, "k"))) return rc;
  if ((rc = check_strides(v, v_strides, 4, 8, "v"))) return rc;
  if ((rc = check_index(start, true, "start")) || (rc = check_index(count, false, "count"))) return rc;
  if ((rc = check_rope(&mode, rope_theta))) return rc;
  if ((rc = current_status_word(&p.status))) return rc;
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.k_sb = k_strides[0] * 2, p.k_sh = k_strides[1] * 2, p.k_sn = k_strides[2] * 2;
  p.v_sb = v_strides[0] * 2, p.v_sh = v_strides[1] * 2, p.v_sn = v_strides[2] * 2;
  p.first = start;
  p.count = count;
  p.N = N;
  p.rows = (int64_t)cache->B * N;
  p.div_n = N > 1 ? ~0ull / N + 1 : 0;  // ceil(2^64 / N)
  if (mode == ATTNFUSE_ROPE_FUSED) p.freqs = paged_freqs(cache->d, rope_theta);
  return done(launch_paged_append(p, cache->d, cache->format, mode == ATTNFUSE_ROPE_FUSED, stream),
              "paged append launch");
}

attnfuse_status attnfuse_paged_gather(const attnfuse_paged_cache* cache, const int32_t* start,
                                      const int32_t* count, void* k, const int64_t k_strides[4],
                                      void* v, const int64_t v_strides[4], int N,
                                      cudaStream_t stream) {
  PagedGatherParams p;
  memset(&p, 0, sizeof(p));
  int rc;
  if ((rc = check_cache(cache, &p.cache))) return rc;
  if ((rc = check_n(cache->B, N))) return rc;
  if ((rc = check_strides(k, k_strides, 4, 8, "k"))) return rc;
  if ((rc = check_strides(v, v_strides, 4, 8, "v"))) return rc;
  if ((rc = check_index(start, false, "start")) || (rc = check_index(count, false, "count"))) return rc;
  if ((rc = current_status_word(&p.status))) return rc;
  p.k = static_cast<uint8_t*>(k);
  p.v = static_cast<uint8_t*>(v);
  p.k_sb = k_strides[0] * 2, p.k_sh = k_strides[1] * 2, p.k_sn = k_strides[2] * 2;
  p.v_sb = v_strides[0] * 2, p.v_sh = v_strides[1] * 2, p.v_sn = v_strides[2] * 2;
  p.first = start;
  p.count = count;
  p.N = N;
  p.rows = (int64_t)cache->B * N;
  p.div_n = N > 1 ? ~0ull / N + 1 : 0;  // ceil(2^64 / N)
  return done(launch_paged_gather(p, cache->d, cache->format, stream), "paged gather launch");
}

attnfuse_status attnfuse_paged_decode_workspace_size(int Hq, int Hkv, int d, int format, size_t* bytes) {
  if (!bytes) return fail(ATTNFUSE_ERR_INVALID_ARG, "bytes is NULL");
  if (Hq <= 0 || Hkv <= 0) return fail(ATTNFUSE_ERR_INVALID_ARG, "sizes must be positive (Hq=%d Hkv=%d)", Hq, Hkv);
  if (Hq % Hkv) return fail(ATTNFUSE_ERR_UNSUPPORTED, "Hq=%d not a multiple of Hkv=%d", Hq, Hkv);
  if (d != 64 && d != 128) return fail(ATTNFUSE_ERR_UNSUPPORTED, "head dim %d (need 64 or 128)", d);
  if (format != ATTNFUSE_CACHE_BF16 && format != ATTNFUSE_CACHE_Q4)
    return fail(ATTNFUSE_ERR_INVALID_ARG, "cache format %d", format);
  *bytes = paged_decode_workspace(d, Hq / Hkv, format);
  return set_last_error(ATTNFUSE_OK, "");
}

attnfuse_status attnfuse_paged_decode(const attnfuse_paged_cache* cache, const void* q,
                                      const int64_t q_strides[3], const int32_t* lens, void* out,
                                      const int64_t o_strides[3], float* lse, int Hq, float scale,
                                      float rope_theta, attnfuse_rope_mode rope_mode, int window,
                                      const float* alibi_slopes, void* workspace,
                                      size_t workspace_bytes, cudaStream_t stream) {
  PagedDecodeParams p;
  memset(&p, 0, sizeof(p));
  int rc, mode = rope_mode;
  if ((rc = check_cache(cache, &p.cache))) return rc;
  size_t need = 0;
  if ((rc = attnfuse_paged_decode_workspace_size(Hq, cache->Hkv, cache->d, cache->format, &need))) return rc;
  if ((rc = check_strides(q, q_strides, 3, 8, "q"))) return rc;
  if (!out || !aligned(out, 2) || !o_strides || o_strides[2] != 1 || o_strides[0] <= 0 || o_strides[1] <= 0)
    return fail(ATTNFUSE_ERR_INVALID_ARG, "out: NULL, misaligned or bad strides");
  if ((rc = check_index(lens, true, "lens"))) return rc;
  if (!aligned(lse, 4)) return fail(ATTNFUSE_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  if (!aligned(alibi_slopes, 4)) return fail(ATTNFUSE_ERR_INVALID_ARG, "alibi_slopes is not 4-byte aligned");
  if (!(scale > 0.f) || !std::isfinite(scale))
    return fail(ATTNFUSE_ERR_INVALID_ARG, "scale must be positive and finite");
  if (window < 0) return fail(ATTNFUSE_ERR_INVALID_ARG, "window %d < 0", window);
  if ((rc = check_rope(&mode, rope_theta))) return rc;
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return fail(ATTNFUSE_ERR_WORKSPACE_TOO_SMALL, "workspace needs %zu bytes (got %zu)", need, workspace_bytes);
  if ((int64_t)cache->B * Hq > 0x7fffffff || Hq > 4096 ||
      (int64_t)cache->B * Hq * (p.cache.cap / 64 + 1) > ((int64_t)1 << 36))
    return fail(ATTNFUSE_ERR_UNSUPPORTED, "B * Hq * max_pages * page_size too large (Hq at most 4096)");
  if ((rc = current_status_word(&p.status))) return rc;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_sb = q_strides[0], p.q_sh = q_strides[1];
  p.out = static_cast<__nv_bfloat16*>(out);
  p.o_sb = o_strides[0], p.o_sh = o_strides[1];
  p.lse = lse;
  p.lens = lens;
  p.Hq = Hq;
  p.g = Hq / cache->Hkv;
  p.window = window;
  p.slopes = alibi_slopes;
  p.rope = mode == ATTNFUSE_ROPE_FUSED;
  p.scale_log2 = scale * kLog2e;
  if (p.rope) p.freqs = paged_freqs(cache->d, rope_theta);
  p.workspace = workspace;
  p.frag_rows = paged_frag_rows(cache->page_size, cache->d, p.g, cache->format);
  if (cache->format == ATTNFUSE_CACHE_BF16) {
    if ((rc = encode_map_bhnd(&p.tmK, cache->k, cache->k_strides, cache->num_pages, cache->Hkv, cache->page_size,
                              cache->d, "cache k", p.frag_rows)))
      return rc;
    if ((rc = encode_map_bhnd(&p.tmV, cache->v, cache->v_strides, cache->num_pages, cache->Hkv, cache->page_size,
                              cache->d, "cache v", p.frag_rows)))
      return rc;
  }
  return done(launch_paged_decode(p, cache->d, cache->format, stream), "paged decode launch");
}

}  // extern "C"
