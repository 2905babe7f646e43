// Attention of a chunk of new tokens over a paged cache.
//
//   O = sum_m p_m v_m,  p = softmax over m in (P - W, P] of  s_m = scale <R_P q, k_m> + slope_h (m - P)
//
// for query row n of sequence b at position P = first[b] + n. A warp takes one row of one head and
// walks its keys one at a time with a running maximum and sum.
#include <cuda_runtime.h>

#include "launch.h"
#include "paged.cuh"

namespace afx {

namespace {

constexpr int kThreads = 128;

// Elements C l .. C l + C - 1 (C = D / 32) of a cache row of one head.
template <int D, bool Q4>
__device__ __forceinline__ void row_piece(const uint8_t* pool, const uint8_t* steps, int64_t row, int64_t steps_row, int slot,
                                          int lane, float (&x)[D / 32]) {
  constexpr int C = D / 32;
  if constexpr (!Q4) {
    const uint16_t* at = reinterpret_cast<const uint16_t*>(pool + row) + C * lane;
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = __uint_as_float(static_cast<uint32_t>(at[c]) << 16);
  } else {
    const int e = C * lane, g = e / 32, r = e % 32 / 4;
    const uint16_t word = *reinterpret_cast<const uint16_t*>(pool + row + q4_place<D>(r, slot) * (D / 16) + 2 * g);
    const float step = __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(steps + steps_row + 2 * g)) << 16);
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = step * (static_cast<float>((word >> (4 * ((e + c) % 4))) & 15) - 8.0f);
  }
}

template <int D, bool Q4>
__global__ void __launch_bounds__(kThreads) attend_rows_kernel(const __grid_constant__ PagedAttendParams p) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x % 32;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / 32;
  if (w >= static_cast<int64_t>(p.cache.B) * p.Hq * p.N) return;
  const int n = static_cast<int>(w % p.N), h = static_cast<int>(w / p.N % p.Hq), b = static_cast<int>(w / p.N / p.Hq);
  int first = __ldg(p.first + b), count = p.count ? __ldg(p.count + b) : p.N;
  bool bad = count < 0 || count > p.N;
  count = min(max(count, 0), p.N);
  if (count > 0 && (first < 0 || static_cast<int64_t>(first) + count > p.cache.cap)) {
    bad = true;
    if (first < 0 || first >= p.cache.cap) first = 0, count = 0;
    else count = p.cache.cap - first;
  }
  if (bad && lane == 0) atomicOr(p.status, kDevPageRange);
  __nv_bfloat16* out = p.out + b * p.o_sb + h * p.o_sh + n * p.o_sn + C * lane;
  float m = kNegInf, l = 0.f, o[C] = {};
  if (n < count) {
    const int pos = first + n;
    float q[C];
    const __nv_bfloat16* at = p.q + b * p.q_sb + h * p.q_sh + n * p.q_sn + C * lane;
#pragma unroll
    for (int c = 0; c < C; ++c) q[c] = __bfloat162float(at[c]);
    if (p.rope) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float other = __shfl_xor_sync(0xffffffffu, q[c], 16);
        const float4 a = turn_cossin(static_cast<float>(pos), freq_at(p.freqs, (C * lane + c) % (D / 2)));
        q[c] = q[c] * (a.x + a.y) + (lane < 16 ? -other : other) * (a.z + a.w);
      }
    }
    const float slope = p.slopes ? __ldg(p.slopes + h) : 0.f;
    const int kvh = h / p.g;
    for (int i = p.window > 0 ? max(0, pos - p.window + 1) : 0; i <= pos; ++i) {
      int slot;
      const int page = page_at(p.cache, b, i, &slot);
      if (page < 0) {
        if (lane == 0) atomicOr(p.status, kDevPageRange);
        continue;
      }
      const int64_t st = Q4 ? D / 2 : 0;
      float k[C], v[C];
      row_piece<D, Q4>(p.cache.k, p.cache.ks, page * p.cache.k_sp + kvh * p.cache.k_sh + slot * (Q4 ? st : p.cache.k_st),
                       page * p.cache.ks_sp + kvh * p.cache.ks_sh + slot * (D / 16), slot, lane, k);
      row_piece<D, Q4>(p.cache.v, p.cache.vs, page * p.cache.v_sp + kvh * p.cache.v_sh + slot * (Q4 ? st : p.cache.v_st),
                       page * p.cache.vs_sp + kvh * p.cache.vs_sh + slot * (D / 16), slot, lane, v);
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) s = fmaf(q[c], k[c], s);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s = s * p.scale + slope * static_cast<float>(i - pos);
      if (s > m) {
        const float a = expf(m - s);
        m = s;
        l *= a;
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] *= a;
      }
      const float e = m == kNegInf ? 0.f : expf(s - m);
      l += e;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = fmaf(e, v[c], o[c]);
    }
  }
  const bool any = !(l == 0.f);
#pragma unroll
  for (int c = 0; c < C; ++c) out[c] = __float2bfloat16_rn(any ? o[c] / l : 0.f);
  if (p.lse && lane == 0) p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.N + n] = any ? m + logf(l) : kNegInf;
}

}  // namespace

size_t paged_attend_workspace(int, int, int, int, int, int, bool) { return 16; }

cudaError_t launch_paged_attend(PagedAttendParams p, int d, int format, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.cache.B) * p.Hq * p.N;
  void (*kern)(PagedAttendParams);
  if (format == kPagedQ4) kern = d == 128 ? attend_rows_kernel<128, true> : attend_rows_kernel<64, true>;
  else kern = d == 128 ? attend_rows_kernel<128, false> : attend_rows_kernel<64, false>;
  kern<<<static_cast<unsigned>((rows + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace afx
