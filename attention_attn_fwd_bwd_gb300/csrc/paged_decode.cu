// Decode over a paged cache: one query per sequence against that sequence's own length.
//
//   O_h = sum_n p_n v_n,  p = softmax over n in [max(0, L - W), L) of
//   s_n = scale <R_{L-1} q_h, k_n> + slope_h (n - (L - 1)),  L = lens[b].
//
// One CTA per (sequence, query head); warps take keys in turn, each keeps a running maximum,
// sum and accumulator (lane = d / 32 elements), and the warps' states are joined at the end.
#include <cuda_runtime.h>

#include "launch.h"
#include "paged.cuh"

namespace afx {

namespace {

constexpr int kWarps = 8;

// Element e of a cache row (any format).
template <int D, bool Q4>
__device__ __forceinline__ float row_elem(const uint8_t* row, const uint8_t* scales, int slot, int e) {
  if (!Q4) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[e]);
  const int g = e / 32, r = (e % 32) / 4, i = e % 4;
  const uint16_t w = reinterpret_cast<const uint16_t*>(row + q4_place<D>(r, slot) * (D / 16))[g];
  return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(scales)[g]) *
         static_cast<float>(((w >> (4 * i)) & 15) - 8);
}

template <int D, bool Q4>
__global__ void __launch_bounds__(kWarps * 32) paged_decode_kernel(const __grid_constant__ PagedDecodeParams p) {
  constexpr int E = D / 32;
  __shared__ float qs[D];
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq, kvh = h / p.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int L = __ldg(p.lens + b);
  if (L < 0 || L > p.cache.cap) {
    atomicOr(p.status, kDevPageRange);
    L = L < 0 ? 0 : p.cache.cap;
  }
  const int first = p.window > 0 && L > p.window ? L - p.window : 0;
  const __nv_bfloat16* q = p.q + b * p.q_sb + h * p.q_sh;
  if (threadIdx.x < D / 2) {
    const int i = threadIdx.x;
    float lo = __bfloat162float(q[i]), hi = __bfloat162float(q[i + D / 2]);
    if (p.rope && L > 0) {
      float c, s, yl, yh;
      rope_cossin_fine(static_cast<float>(L - 1), p.freqs.hi[i], p.freqs.lo[i], &c, &s);
      rot_pair(lo, hi, c, s, yl, yh);
      lo = yl;
      hi = yh;
    }
    qs[i] = lo;
    qs[i + D / 2] = hi;
  }
  __syncthreads();
  float qr[E], o[E] = {}, m = kNegInf, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) qr[e] = qs[lane + 32 * e];
  const float slope = p.slopes ? __ldg(p.slopes + h) * kLog2e : 0.f;
  for (int n = first + warp; n < L; n += kWarps) {
    int slot;
    const int page = page_at(p.cache, b, n, &slot);
    if (page < 0) {
      if (lane == 0) atomicOr(p.status, kDevPageRange);
      continue;
    }
    const uint8_t* kr = p.cache.k + page * p.cache.k_sp + kvh * p.cache.k_sh + slot * p.cache.k_st;
    const uint8_t* vr = p.cache.v + page * p.cache.v_sp + kvh * p.cache.v_sh + slot * p.cache.v_st;
    const uint8_t* ks = p.cache.ks + page * p.cache.ks_sp + kvh * p.cache.ks_sh + slot * (D / 16);
    const uint8_t* vs = p.cache.vs + page * p.cache.vs_sp + kvh * p.cache.vs_sh + slot * (D / 16);
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x = fmaf(qr[e], row_elem<D, Q4>(kr, ks, slot, lane + 32 * e), x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    x = x * p.scale_log2 + slope * static_cast<float>(n - (L - 1));
    const float mn = fmaxf(m, x);
    const float base = mn == kNegInf ? 0.f : mn;
    const float a = ex2_approx(m - base), w = ex2_approx(x - base);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * row_elem<D, Q4>(vr, vs, slot, lane + 32 * e);
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float M = kNegInf, total = 0.f, acc = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    const float base = M == kNegInf ? 0.f : M;
    for (int w = 0; w < kWarps; ++w) {
      const float a = ex2_approx(sm[w] - base);
      total += a * sl[w];
      acc += a * so[w][threadIdx.x];
    }
    const bool any = !(total == 0.f);  // a NaN goes to the output
    p.out[b * p.o_sb + h * p.o_sh + threadIdx.x] = __float2bfloat16_rn(any ? acc / total : 0.f);
    if (p.lse && threadIdx.x == 0) p.lse[blockIdx.x] = any ? (base + log2f(total)) * kLn2 : kNegInf;
  }
}

}  // namespace

size_t paged_decode_workspace(int, int) { return 0; }

cudaError_t launch_paged_decode(const PagedDecodeParams& p, int d, int format, cudaStream_t stream) {
  void (*kern)(PagedDecodeParams) = nullptr;
  if (format == kPagedQ4) kern = d == 128 ? paged_decode_kernel<128, true> : paged_decode_kernel<64, true>;
  else kern = d == 128 ? paged_decode_kernel<128, false> : paged_decode_kernel<64, false>;
  kern<<<p.cache.B * p.Hq, kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace afx
