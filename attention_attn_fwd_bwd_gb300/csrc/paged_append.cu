// Writing rows into a paged cache (with the rotation of K and, for q4, the quantisation on the
// way) and reading them back out as dense bf16 rows.
//
// Both are bound by HBM: a row of K and V is read once and written once; prompts of 18.5k rows
// (Hkv = 8, d = 128) move 151 MB. A thread keeps its part of the row for a run of heads, so that
// the D/2 angles of a position are computed once per run and not once per head.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "paged.cuh"

namespace afx {

namespace {

constexpr int kThreads = 256;

// Row of this thread: sequence b, row n of the call, position pos; false if there is none.
struct RowAt {
  int b, n, page, slot;
  float pos;
};

__device__ __forceinline__ void raise_page(int* status) { atomicOr(status, kDevPageRange); }

// Count of live rows of sequence b (a count outside [0, N] is reported and clamped).
__device__ __forceinline__ int live_rows(const int32_t* count, int b, int N, int* status) {
  if (!count) return N;
  const int c = __ldg(count + b);
  if (c >= 0 && c <= N) return c;
  raise_page(status);
  return c < 0 ? 0 : N;
}

// Finds the page of row n of sequence b; false where nothing may be accessed.
__device__ __forceinline__ bool find_row(const PagedDev& c, int b, int n, int first, int* status, RowAt* r) {
  const int64_t p = static_cast<int64_t>(first) + n;
  if (first < 0 || p >= c.cap) {
    raise_page(status);
    return false;
  }
  r->b = b;
  r->n = n;
  r->pos = static_cast<float>(p);
  r->page = page_at(c, b, static_cast<int>(p), &r->slot);
  if (r->page < 0) raise_page(status);
  return r->page >= 0;
}

// ---------------------------------------------------------------------------------------------
// bf16: thread = 8 pairs (x_i, x_{i + D/2}) of a row, two 16-byte chunks
// ---------------------------------------------------------------------------------------------
template <int D, bool ROPE>
__global__ void __launch_bounds__(kThreads) append_bf16_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int CP = D / 16;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / CP) + threadIdx.x / CP;
  const int ch = threadIdx.x % CP;
  if (row >= p.rows) return;
  const int b = static_cast<int>(row / p.N), n = static_cast<int>(row - static_cast<int64_t>(b) * p.N);
  if (n >= live_rows(p.count, b, p.N, p.status)) return;
  RowAt r;
  if (!find_row(p.cache, b, n, __ldg(p.first + b), p.status, &r)) return;
  float c[8], s[8];
  if (ROPE) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      rope_cossin_fine(r.pos, p.freqs.hi[ch * 8 + e], p.freqs.lo[ch * 8 + e], &c[e], &s[e]);
  }
  const int h0 = blockIdx.y * p.heads_per_thread, h1 = min(p.cache.Hkv, h0 + p.heads_per_thread);
  const uint8_t* k = p.k + b * p.k_sb + n * p.k_sn + ch * 16;
  const uint8_t* v = p.v + b * p.v_sb + n * p.v_sn + ch * 16;
  uint8_t* kd = p.cache.k + r.page * p.cache.k_sp + r.slot * p.cache.k_st + ch * 16;
  uint8_t* vd = p.cache.v + r.page * p.cache.v_sp + r.slot * p.cache.v_st + ch * 16;
#pragma unroll 2
  for (int h = h0; h < h1; ++h) {
    uint4 lo = __ldg(reinterpret_cast<const uint4*>(k + h * p.k_sh));
    uint4 hi = __ldg(reinterpret_cast<const uint4*>(k + h * p.k_sh + D));
    const uint4 v0 = __ldg(reinterpret_cast<const uint4*>(v + h * p.v_sh));
    const uint4 v1 = __ldg(reinterpret_cast<const uint4*>(v + h * p.v_sh + D));
    if (ROPE) {
      uint32_t* L = reinterpret_cast<uint32_t*>(&lo);
      uint32_t* H = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float cw[2] = {c[2 * w], c[2 * w + 1]}, sw[2] = {s[2 * w], s[2 * w + 1]};
        rot_word_exact(L[w], H[w], cw, sw, r.pos, p.freqs, ch * 8 + 2 * w);
      }
    }
    *reinterpret_cast<uint4*>(kd + h * p.cache.k_sh) = lo;
    *reinterpret_cast<uint4*>(kd + h * p.cache.k_sh + D) = hi;
    *reinterpret_cast<uint4*>(vd + h * p.cache.v_sh) = v0;
    *reinterpret_cast<uint4*>(vd + h * p.cache.v_sh + D) = v1;
  }
}

// ---------------------------------------------------------------------------------------------
// q4: 8 threads per row; thread r holds elements 32g + 4r .. + 3 of every group g, which are
// whole pairs (group g with group g + G/2) and exactly chunk r of the stored row
// ---------------------------------------------------------------------------------------------

// 4 elements (two bf16x2 words) with reciprocal step inv -> 4 nibbles, lowest first.
// x and the step have 8 significant bits each, so |x| / s is a tie k + 1/2 or at least 2^-12
// (relative) away from one; the product with the reciprocal is within 2^-23, and the factor
// 1 + 2^-20 puts ties, and only them, on the far side.
__device__ __forceinline__ uint32_t q4_codes(uint32_t w0, uint32_t w1, float inv) {
  const float x[4] = {bf16lo_to_f32(w0), bf16hi_to_f32(w0), bf16lo_to_f32(w1), bf16hi_to_f32(w1)};
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float t = fminf(fabsf(x[i] * inv), 7.0f);
    const float z = __fadd_rd(__fmaf_rn(t, 1.00000095367431640625f, 0.5f), 8388608.0f);  // 2^23 + floor
    const int m = __float_as_int(z) & 7;
    out |= static_cast<uint32_t>(x[i] < 0.0f ? 8 - m : 8 + m) << (4 * i);
  }
  return out;
}

// Quantises one row: w[g] = this thread's two words of group g. Returns the chunk; thread 0 of
// the row also gets the scales.
template <int G>
__device__ __forceinline__ void q4_row(const uint2 (&w)[G], uint32_t (&chunk)[G / 2], uint32_t (&scales)[G / 2]) {
#pragma unroll
  for (int q = 0; q < G / 2; ++q) {
    // largest magnitudes of groups 2q and 2q + 1 as bf16 bits (their integers order like the
    // values, NaN above infinity), in one word
    uint32_t a = __vmaxu2(w[2 * q].x & 0x7FFF7FFFu, w[2 * q].y & 0x7FFF7FFFu);
    uint32_t b = __vmaxu2(w[2 * q + 1].x & 0x7FFF7FFFu, w[2 * q + 1].y & 0x7FFF7FFFu);
    a = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, o));
    chunk[q] = 0;
    scales[q] = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t bits = i ? a >> 16 : a & 0xFFFFu;
      const float amax = __uint_as_float(bits << 16);
      uint32_t s = __bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(amax, 7.0f)));
      float inv = __fdiv_rn(1.0f, __uint_as_float(s << 16));
      if (amax < 0x1p-96f) s = 0, inv = 0.0f;         // reads back as zeros
      if (bits >= 0x7F80u) s = 0x7FC0u, inv = 0.0f;   // an infinity or a NaN: reads back as NaN
      // (inf * 0 and NaN * 0 are NaN, which fminf turns into 7: harmless under a NaN scale)
      chunk[q] |= q4_codes(w[2 * q + i].x, w[2 * q + i].y, inv) << (16 * i);
      scales[q] |= s << (16 * i);
    }
  }
}

template <int D, bool ROPE>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int G = D / kQ4Group;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 8) + threadIdx.x / 8;
  const int t = threadIdx.x % 8;
  // rows without work stay for the shuffles
  const bool in = row < p.rows;
  const int b = in ? static_cast<int>(row / p.N) : 0;
  const int n = in ? static_cast<int>(row - static_cast<int64_t>(b) * p.N) : 0;
  RowAt r = {};
  const bool live = in && n < live_rows(p.count, b, p.N, p.status) &&
                    find_row(p.cache, b, n, __ldg(p.first + b), p.status, &r);
  if (!__any_sync(0xffffffffu, live)) return;
  float c[G / 2][4], s[G / 2][4];
  if (ROPE) {
#pragma unroll
    for (int g = 0; g < G / 2; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        rope_cossin_fine(r.pos, p.freqs.hi[32 * g + 4 * t + e], p.freqs.lo[32 * g + 4 * t + e], &c[g][e],
                         &s[g][e]);
  }
  const int h0 = blockIdx.y * p.heads_per_thread, h1 = min(p.cache.Hkv, h0 + p.heads_per_thread);
  const uint8_t* k = p.k + b * p.k_sb + n * p.k_sn + t * 8;
  const uint8_t* v = p.v + b * p.v_sb + n * p.v_sn + t * 8;
  const int64_t at = static_cast<int64_t>(r.slot) * (D / 2) + q4_place<D>(t, r.slot) * (D / 16);
  uint8_t* kd = p.cache.k + r.page * p.cache.k_sp + at;
  uint8_t* vd = p.cache.v + r.page * p.cache.v_sp + at;
  uint8_t* ksd = p.cache.ks + r.page * p.cache.ks_sp + r.slot * (D / 16);
  uint8_t* vsd = p.cache.vs + r.page * p.cache.vs_sp + r.slot * (D / 16);
  for (int h = h0; h < h1; ++h) {
    uint2 kw[G], vw[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      kw[g] = live ? __ldg(reinterpret_cast<const uint2*>(k + h * p.k_sh + g * 64)) : make_uint2(0, 0);
      vw[g] = live ? __ldg(reinterpret_cast<const uint2*>(v + h * p.v_sh + g * 64)) : make_uint2(0, 0);
    }
    if (ROPE) {
#pragma unroll
      for (int g = 0; g < G / 2; ++g) {
        const float c0[2] = {c[g][0], c[g][1]}, s0[2] = {s[g][0], s[g][1]};
        const float c1[2] = {c[g][2], c[g][3]}, s1[2] = {s[g][2], s[g][3]};
        rot_word_exact(kw[g].x, kw[g + G / 2].x, c0, s0, r.pos, p.freqs, 32 * g + 4 * t);
        rot_word_exact(kw[g].y, kw[g + G / 2].y, c1, s1, r.pos, p.freqs, 32 * g + 4 * t + 2);
      }
    }
    uint32_t chunk[G / 2], scales[G / 2];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      q4_row<G>(which ? vw : kw, chunk, scales);
      uint8_t* dst = which ? vd + h * p.cache.v_sh : kd + h * p.cache.k_sh;
      uint8_t* sd = which ? vsd + h * p.cache.vs_sh : ksd + h * p.cache.ks_sh;
      if (!live) continue;
      if constexpr (G == 4) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(chunk[0], chunk[1]);
        if (t == 0) *reinterpret_cast<uint2*>(sd) = make_uint2(scales[0], scales[1]);
      } else {
        *reinterpret_cast<uint32_t*>(dst) = chunk[0];
        if (t == 0) *reinterpret_cast<uint32_t*>(sd) = scales[0];
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Gather: cache rows first[b] .. first[b] + count[b] - 1 -> dense rows 0 .. N - 1, zeros behind
// ---------------------------------------------------------------------------------------------
template <int D, bool Q4>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ PagedGatherParams p) {
  constexpr int TPR = Q4 ? 8 : D / 8;  // threads per row: q4 chunks, or 16-byte pieces
  constexpr int G = D / kQ4Group;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  if (row >= p.rows) return;
  const int b = static_cast<int>(row / p.N), n = static_cast<int>(row - static_cast<int64_t>(b) * p.N);
  RowAt r;
  const bool live = n < live_rows(p.count, b, p.N, p.status) &&
                    find_row(p.cache, b, n, p.first ? __ldg(p.first + b) : 0, p.status, &r);
  const int h0 = blockIdx.y * p.heads_per_thread, h1 = min(p.cache.Hkv, h0 + p.heads_per_thread);
  uint8_t* ko = p.k + b * p.k_sb + n * p.k_sn;
  uint8_t* vo = p.v + b * p.v_sb + n * p.v_sn;
  for (int h = h0; h < h1; ++h) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      uint8_t* out = which ? vo + h * p.v_sh : ko + h * p.k_sh;
      if (!Q4) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (live) {
          const uint8_t* src = which ? p.cache.v + r.page * p.cache.v_sp + r.slot * p.cache.v_st + h * p.cache.v_sh
                                     : p.cache.k + r.page * p.cache.k_sp + r.slot * p.cache.k_st + h * p.cache.k_sh;
          x = *reinterpret_cast<const uint4*>(src + t * 16);
        }
        *reinterpret_cast<uint4*>(out + t * 16) = x;
      } else {
        uint32_t w[G / 2] = {}, sc[G / 2] = {};
        if (live) {
          const int64_t at = static_cast<int64_t>(r.slot) * (D / 2) + q4_place<D>(t, r.slot) * (D / 16);
          const uint8_t* src = which ? p.cache.v + r.page * p.cache.v_sp + h * p.cache.v_sh + at
                                     : p.cache.k + r.page * p.cache.k_sp + h * p.cache.k_sh + at;
          const uint8_t* ss = which ? p.cache.vs + r.page * p.cache.vs_sp + h * p.cache.vs_sh + r.slot * (D / 16)
                                    : p.cache.ks + r.page * p.cache.ks_sp + h * p.cache.ks_sh + r.slot * (D / 16);
#pragma unroll
          for (int q = 0; q < G / 2; ++q) {
            w[q] = reinterpret_cast<const uint32_t*>(src)[q];
            sc[q] = reinterpret_cast<const uint32_t*>(ss)[q];
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t h4 = (w[g / 2] >> (16 * (g & 1))) & 0xFFFFu;
          const float s = (g & 1) ? bf16hi_to_f32(sc[g / 2]) : bf16lo_to_f32(sc[g / 2]);
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)  // code times step: 12 significant bits, rounded once
            x[i] = s * static_cast<float>(static_cast<int>((h4 >> (4 * i)) & 15) - 8);
          *reinterpret_cast<uint2*>(out + g * 64 + t * 8) =
              live ? make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])) : make_uint2(0, 0);
        }
      }
    }
  }
}

// Heads per thread: a run of heads shares one row's lookup and angles (8 angles cost about as
// much as 4 heads), but the launch should still fill the GPU's thread slots.
int heads_per_thread(int64_t rows, int tpr, int Hkv) {
  const int64_t want = 152 * 1024;
  const int64_t h = rows * tpr * Hkv / want;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(h, std::min(Hkv, 8))));
}

}  // namespace

cudaError_t launch_paged_append(PagedAppendParams p, int d, int format, bool rope, cudaStream_t stream) {
  const int tpr = format == kPagedQ4 ? 8 : d / 16;
  p.heads_per_thread = heads_per_thread(p.rows, tpr, p.cache.Hkv);
  const int rpb = kThreads / tpr;
  const dim3 grid(static_cast<unsigned>((p.rows + rpb - 1) / rpb),
                  (p.cache.Hkv + p.heads_per_thread - 1) / p.heads_per_thread);
  void (*kern)(PagedAppendParams) = nullptr;
  if (format == kPagedQ4)
    kern = d == 128 ? (rope ? append_q4_kernel<128, true> : append_q4_kernel<128, false>)
                    : (rope ? append_q4_kernel<64, true> : append_q4_kernel<64, false>);
  else
    kern = d == 128 ? (rope ? append_bf16_kernel<128, true> : append_bf16_kernel<128, false>)
                    : (rope ? append_bf16_kernel<64, true> : append_bf16_kernel<64, false>);
  kern<<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_paged_gather(PagedGatherParams p, int d, int format, cudaStream_t stream) {
  const int tpr = format == kPagedQ4 ? 8 : d / 8;
  p.heads_per_thread = heads_per_thread(p.rows, tpr, p.cache.Hkv);
  const int rpb = kThreads / tpr;
  const dim3 grid(static_cast<unsigned>((p.rows + rpb - 1) / rpb),
                  (p.cache.Hkv + p.heads_per_thread - 1) / p.heads_per_thread);
  void (*kern)(PagedGatherParams) = nullptr;
  if (format == kPagedQ4) kern = d == 128 ? gather_kernel<128, true> : gather_kernel<64, true>;
  else kern = d == 128 ? gather_kernel<128, false> : gather_kernel<64, false>;
  kern<<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace afx
