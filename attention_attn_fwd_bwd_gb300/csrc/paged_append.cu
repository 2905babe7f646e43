// Writing rows into a paged cache (with the rotation of K and, for q4, the quantisation on the
// way) and reading them back out as dense bf16 rows.
//
// A row of K and V is read once and written once, and HBM bounds the gather (187 MB of bf16 rows,
// d = 64: 31 us, 89% of a copy's rate) and, with the launch's ragged end, the bf16 append (138 MB,
// 18.5k rows of 8 heads, d = 128, rotated: 28 us, 72%). Appending to 4 bits (12k rows of 8 heads,
// d = 128: 23 us, 38%) takes instructions: 564 per warp, the idle rows' included, keep the
// schedulers issuing 72% of the time.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "paged.cuh"

namespace afx {

namespace {

// The threads that a block's barrier and its slowest load hold up. Prompts to bf16 and to 4 bits
// (with their gather), one token: 128 threads 28.1, 33.5, 2.4 us; 64 (one row of 8 heads shares its
// angles) 36.6, 34.2, 2.4; 256 28.1, 34.6, 2.6; 512 32.9, 38.5, 2.9.
constexpr int kThreads = 128;

// Sequence and row of row number `row` < 2^31 of the call.
__device__ __forceinline__ int seq_of(uint64_t div_n, int64_t row) {
  return static_cast<int>(div_n ? __umul64hi(static_cast<uint64_t>(row), div_n) : row);
}

// Where a row lies in the cache.
struct RowAt {
  int page, slot;
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
  r->page = page_at(c, b, static_cast<int>(p), &r->slot);
  if (r->page < 0) raise_page(status);
  return r->page >= 0;
}

// A block covers rb rows x hb heads, tpr threads for each; the angles of its rows are computed
// once, by all threads, into shared memory: angle (k, t) of a row is that of thread t's k-th pair.
// Angles 2q and 2q + 1 of a thread lie as it uses them, packed: (cos hi, cos hi, cos lo, cos lo),
// then the sines.
struct Place {
  int64_t row;
  int t, rr, h;  // thread of the row, row of the block, head
};
template <int TPR>
__device__ __forceinline__ Place place_of(const PagedAppendParams& p) {
  const int lb = p.rb_log2, k = threadIdx.x / TPR;
  Place w;
  w.t = threadIdx.x % TPR;
  w.rr = k & ((1 << lb) - 1);
  w.row = (static_cast<int64_t>(blockIdx.x) << lb) + w.rr;
  w.h = blockIdx.y * p.hb + (k >> lb);
  return w;
}

// Pair that angle slot (k, t) of a row stands for.
template <int D, int TPR, bool Q4>
__device__ __forceinline__ int pair_of(int k, int t) {
  return Q4 ? 32 * (k / 4) + 4 * t + k % 4 : 8 * t + k;
}

template <int D, int TPR, bool Q4>
__device__ __forceinline__ void block_angles(const PagedAppendParams& p, float4* ang) {
  constexpr int K = D / 2 / TPR;  // pairs per thread of a row
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) << p.rb_log2;
  for (int i = threadIdx.x; i < (D / 2) << p.rb_log2; i += kThreads) {
    const int64_t row = row0 + i / (D / 2);
    if (row >= p.rows) break;
    const int j = i % (D / 2), b = seq_of(p.div_n, row), n = static_cast<int>(row - static_cast<int64_t>(b) * p.N);
    if (p.count && n >= __ldg(p.count + b)) continue;
    const int64_t pos = static_cast<int64_t>(__ldg(p.first + b)) + n;
    if (pos < 0 || pos >= p.cache.cap) continue;
    const int k = j / TPR, t = j % TPR;
    const float4 a = turn_cossin(static_cast<float>(pos), freq_at(p.freqs, pair_of<D, TPR, Q4>(k, t)));
    float* at = reinterpret_cast<float*>(ang + (i / (D / 2)) * (D / 2) + (k / 2) * 2 * TPR + t) + (k & 1);
    at[0] = a.x;
    at[2] = a.y;
    at[4 * TPR] = a.z;
    at[4 * TPR + 2] = a.w;
  }
  static_assert(K * TPR == D / 2, "pairs");
  __syncthreads();
}

// Rotates the words of pairs 2q, 2q + 1 of thread t of a row.
template <int D, int TPR>
__device__ __forceinline__ void rotate(uint32_t& lo, uint32_t& hi, const float4* ang, int rr, int q, int t) {
  const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(ang + rr * (D / 2) + q * 2 * TPR + t);
  const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(ang + rr * (D / 2) + (q * 2 + 1) * TPR + t);
  rot_word_exact(lo, hi, c.x, c.y, s.x, s.y);
}

// ---------------------------------------------------------------------------------------------
// bf16: thread = 8 pairs (x_i, x_{i + D/2}) of a row, two 16-byte chunks
// ---------------------------------------------------------------------------------------------
template <int D, bool ROPE>
__global__ void __launch_bounds__(kThreads) append_bf16_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int CP = D / 16;
  extern __shared__ float4 ang[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Place w = place_of<CP>(p);
  const bool in = w.row < p.rows && w.h < p.cache.Hkv;
  const int b = in ? seq_of(p.div_n, w.row) : 0;
  const int n = in ? static_cast<int>(w.row - static_cast<int64_t>(b) * p.N) : 0;
  RowAt r;
  const bool live = in && n < live_rows(p.count, b, p.N, p.status) &&
                    find_row(p.cache, b, n, __ldg(p.first + b), p.status, &r);
  uint4 lo, hi, v0, v1;
  if (live) {
    const uint8_t* k = p.k + b * p.k_sb + n * p.k_sn + w.h * p.k_sh + w.t * 16;
    const uint8_t* v = p.v + b * p.v_sb + n * p.v_sn + w.h * p.v_sh + w.t * 16;
    lo = __ldg(reinterpret_cast<const uint4*>(k));
    hi = __ldg(reinterpret_cast<const uint4*>(k + D));
    v0 = __ldg(reinterpret_cast<const uint4*>(v));
    v1 = __ldg(reinterpret_cast<const uint4*>(v + D));
  }
  if (ROPE) block_angles<D, CP, false>(p, ang);
  if (live) {
    if (ROPE) {
      uint32_t* L = reinterpret_cast<uint32_t*>(&lo);
      uint32_t* H = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
      for (int q = 0; q < 4; ++q) rotate<D, CP>(L[q], H[q], ang, w.rr, q, w.t);
    }
    uint8_t* kd = p.cache.k + r.page * p.cache.k_sp + r.slot * p.cache.k_st + w.h * p.cache.k_sh + w.t * 16;
    uint8_t* vd = p.cache.v + r.page * p.cache.v_sp + r.slot * p.cache.v_st + w.h * p.cache.v_sh + w.t * 16;
    *reinterpret_cast<uint4*>(kd) = lo;
    *reinterpret_cast<uint4*>(kd + D) = hi;
    *reinterpret_cast<uint4*>(vd) = v0;
    *reinterpret_cast<uint4*>(vd + D) = v1;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------------------------------------
// q4: 8 threads per row; thread t holds elements 32g + 4t .. + 3 of every group g, which are
// whole pairs (group g with group g + G/2) and exactly chunk t of the stored row
// ---------------------------------------------------------------------------------------------

// 4 elements (two bf16x2 words) -> 4 nibbles code + 8 in the low 16 bits, lowest first.
// inv = (1 + 2^-20) / s, twice. x and s have 8 significant bits each, so |x| / s is a tie k + 1/2
// or at least 2^-12 (relative) away from one; the reciprocal's error (1 ulp) and a rounding stay
// within 2^-22, so the factor puts ties, and only them, past the middle. |x| / s < 7.03: no clamp.
// Added to M + 8, M = 1.5 2^23, a quotient is rounded to an integer n in the sum's low bits, and
// sums M + n0 + 16 n1 (and M + a + 256 b of two such) are exact: 16 (M + n1) - 16 M is.
__device__ __forceinline__ uint32_t q4_codes(uint32_t w0, uint32_t w1, uint64_t inv) {
  constexpr float kM = 12582912.0f;
  const uint64_t at = f2_pack(kM + 8.0f, kM + 8.0f);
  const uint64_t even = fma2(f2_pack(bf16lo_to_f32(w0), bf16lo_to_f32(w1)), inv, at);
  const uint64_t odd = fma2(f2_pack(bf16hi_to_f32(w0), bf16hi_to_f32(w1)), inv, at);
  const uint64_t two = add2(even, fma2(odd, f2_pack(16.0f, 16.0f), f2_pack(-16.0f * kM, -16.0f * kM)));
  return __float_as_uint(__fadd_rn(f2_lo(two), __fmaf_rn(f2_hi(two), 256.0f, -256.0f * kM)));
}

// The largest magnitude of the group that thread t of a row answers for, group t % G of K
// (t % 2G < G) or V, as bf16 bits (their integers order like the values, NaN above infinity).
// Words of two groups each; a thread hands on half of its words at each step, so that 8 threads
// reduce 8 groups with 4 shuffles.
template <int G>
__device__ __forceinline__ uint32_t q4_amax(const uint2 (&x)[2][G], int t) {
  uint32_t a[2][G / 2];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int q = 0; q < G / 2; ++q) {
      const uint32_t e = __vmaxu2(x[w][2 * q].x & 0x7FFF7FFFu, x[w][2 * q].y & 0x7FFF7FFFu);
      const uint32_t o = __vmaxu2(x[w][2 * q + 1].x & 0x7FFF7FFFu, x[w][2 * q + 1].y & 0x7FFF7FFFu);
      a[w][q] = __vmaxu2(__byte_perm(e, o, 0x5410), __byte_perm(e, o, 0x7632));
    }
  uint32_t k0, k1;  // after the first step: words 0 and 1 of K or V; K's and V's word
  if constexpr (G == 4) {
    const bool up = t & 4;
    k0 = __vmaxu2(up ? a[1][0] : a[0][0], __shfl_xor_sync(0xffffffffu, up ? a[0][0] : a[1][0], 4));
    k1 = __vmaxu2(up ? a[1][1] : a[0][1], __shfl_xor_sync(0xffffffffu, up ? a[0][1] : a[1][1], 4));
  } else {
    k0 = __vmaxu2(a[0][0], __shfl_xor_sync(0xffffffffu, a[0][0], 4));
    k1 = __vmaxu2(a[1][0], __shfl_xor_sync(0xffffffffu, a[1][0], 4));
  }
  const bool up = t & 2;
  uint32_t k = __vmaxu2(up ? k1 : k0, __shfl_xor_sync(0xffffffffu, up ? k0 : k1, 2));
  k = __vmaxu2(k, __shfl_xor_sync(0xffffffffu, k, 1));
  return (t & 1) ? k >> 16 : k & 0xFFFFu;
}

template <int D, bool ROPE>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int G = D / kQ4Group;
  extern __shared__ float4 ang[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Place w = place_of<8>(p);
  const bool in = w.row < p.rows && w.h < p.cache.Hkv;
  const int b = in ? seq_of(p.div_n, w.row) : 0;
  const int n = in ? static_cast<int>(w.row - static_cast<int64_t>(b) * p.N) : 0;
  RowAt r = {};
  const bool live = in && n < live_rows(p.count, b, p.N, p.status) &&
                    find_row(p.cache, b, n, __ldg(p.first + b), p.status, &r);
  uint2 x[2][G];  // K, V
#pragma unroll
  for (int g = 0; g < G; ++g) x[0][g] = x[1][g] = make_uint2(0, 0);
  if (live) {
    const uint8_t* k = p.k + b * p.k_sb + n * p.k_sn + w.h * p.k_sh + w.t * 8;
    const uint8_t* v = p.v + b * p.v_sb + n * p.v_sn + w.h * p.v_sh + w.t * 8;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      x[0][g] = __ldg(reinterpret_cast<const uint2*>(k + g * 64));
      x[1][g] = __ldg(reinterpret_cast<const uint2*>(v + g * 64));
    }
  }
  if (ROPE) {
    block_angles<D, 8, true>(p, ang);
    if (live) {
#pragma unroll
      for (int g = 0; g < G / 2; ++g) {
        rotate<D, 8>(x[0][g].x, x[0][g + G / 2].x, ang, w.rr, 2 * g, w.t);
        rotate<D, 8>(x[0][g].y, x[0][g + G / 2].y, ang, w.rr, 2 * g + 1, w.t);
      }
    }
  }
  // Steps: thread t finds the step of group t % G, of K (t < G) or V, stores it, and hands its
  // reciprocal to the row's other threads. amax / 7 is never a tie of bf16 (or is exact), and at
  // least 2^-12 (relative) away from one, so the product with 1/7 rounds to the same step.
  const uint32_t bits = q4_amax<G>(x, w.t);
  const float amax = __uint_as_float(bits << 16);
  uint32_t s = __bfloat16_as_ushort(__float2bfloat16_rn(amax * (1.0f / 7.0f)));
  float inv;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(__uint_as_float(s << 16)));
  inv *= 1.00000095367431640625f;
  if (amax < 0x1p-96f) s = 0, inv = 0.0f;        // reads back as zeros
  if (bits >= 0x7F80u) s = 0x7FC0u, inv = 0.0f;  // an infinity or a NaN: reads back as NaN, whatever the codes
  uint32_t code[2][G];
  const int row0 = threadIdx.x & 24;  // the row's first lane
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int g = 0; g < G; ++g)
    {
      const float i = __shfl_sync(0xffffffffu, inv, row0 + which * G + g);
      code[which][g] = q4_codes(x[which][g].x, x[which][g].y, f2_pack(i, i));
    }
  if (live) {
    const int64_t at = static_cast<int64_t>(r.slot) * (D / 2) + q4_place<D>(w.t, r.slot) * (D / 16);
    uint8_t* kd = p.cache.k + r.page * p.cache.k_sp + w.h * p.cache.k_sh + at;
    uint8_t* vd = p.cache.v + r.page * p.cache.v_sp + w.h * p.cache.v_sh + at;
    if constexpr (G == 4) {
      *reinterpret_cast<uint2*>(kd) = make_uint2(__byte_perm(code[0][0], code[0][1], 0x5410), __byte_perm(code[0][2], code[0][3], 0x5410));
      *reinterpret_cast<uint2*>(vd) = make_uint2(__byte_perm(code[1][0], code[1][1], 0x5410), __byte_perm(code[1][2], code[1][3], 0x5410));
    } else {
      *reinterpret_cast<uint32_t*>(kd) = __byte_perm(code[0][0], code[0][1], 0x5410);
      *reinterpret_cast<uint32_t*>(vd) = __byte_perm(code[1][0], code[1][1], 0x5410);
    }
    if (w.t < 2 * G) {
      uint8_t* sd = w.t < G ? p.cache.ks + r.page * p.cache.ks_sp + w.h * p.cache.ks_sh
                            : p.cache.vs + r.page * p.cache.vs_sp + w.h * p.cache.vs_sh;
      *reinterpret_cast<uint16_t*>(sd + r.slot * (D / 16) + (w.t % G) * 2) = static_cast<uint16_t>(s);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------------------------------------
// Gather: cache rows first[b] .. first[b] + count[b] - 1 -> dense rows 0 .. N - 1, zeros behind
// ---------------------------------------------------------------------------------------------
// A thread moves its piece of K and V for up to two heads, all loads before the first store.
// Eight heads in turn, a load at a time: 34.6 us for 187 MB of bf16 rows; one head, two, or four
// at a time: 31 each. 343 MB from 4-bit rows: one head 61.0 us, two 54.8, four (64 registers) 55.7.
constexpr int kGatherHeads = 2;

template <int D, bool Q4>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ PagedGatherParams p) {
  constexpr int TPR = Q4 ? 8 : D / 8;  // threads per row: q4 chunks, or 16-byte pieces
  constexpr int G = D / kQ4Group;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  if (row >= p.rows) return;
  const int b = seq_of(p.div_n, row), n = static_cast<int>(row - static_cast<int64_t>(b) * p.N);
  RowAt r;
  const bool live = n < live_rows(p.count, b, p.N, p.status) &&
                    find_row(p.cache, b, n, p.first ? __ldg(p.first + b) : 0, p.status, &r);
  const int h0 = blockIdx.y * p.heads_per_thread, h1 = min(p.cache.Hkv, h0 + p.heads_per_thread);
  uint8_t* const out[2] = {p.k + b * p.k_sb + n * p.k_sn, p.v + b * p.v_sb + n * p.v_sn};
  const int64_t out_sh[2] = {p.k_sh, p.v_sh};
  const uint8_t *src[2] = {}, *steps[2] = {};
  const int64_t src_sh[2] = {p.cache.k_sh, p.cache.v_sh}, steps_sh[2] = {p.cache.ks_sh, p.cache.vs_sh};
  if (live) {
    const int64_t at = Q4 ? static_cast<int64_t>(r.slot) * (D / 2) + q4_place<D>(t, r.slot) * (D / 16) : t * 16;
    src[0] = p.cache.k + r.page * p.cache.k_sp + (Q4 ? at : r.slot * p.cache.k_st + at);
    src[1] = p.cache.v + r.page * p.cache.v_sp + (Q4 ? at : r.slot * p.cache.v_st + at);
    if (Q4) {
      steps[0] = p.cache.ks + r.page * p.cache.ks_sp + r.slot * (D / 16);
      steps[1] = p.cache.vs + r.page * p.cache.vs_sp + r.slot * (D / 16);
    }
  }
  if constexpr (!Q4) {
    uint4 x[2][kGatherHeads];
#pragma unroll
    for (int i = 0; i < kGatherHeads; ++i)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        x[w][i] = make_uint4(0, 0, 0, 0);
        if (live && h0 + i < h1) x[w][i] = *reinterpret_cast<const uint4*>(src[w] + (h0 + i) * src_sh[w]);
      }
#pragma unroll
    for (int i = 0; i < kGatherHeads; ++i)
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (h0 + i < h1) *reinterpret_cast<uint4*>(out[w] + (h0 + i) * out_sh[w] + t * 16) = x[w][i];
  } else {
    uint32_t c[2][kGatherHeads][G / 2], s[2][kGatherHeads][G / 2];
#pragma unroll
    for (int i = 0; i < kGatherHeads; ++i)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int q = 0; q < G / 2; ++q) c[w][i][q] = s[w][i][q] = 0;
        if (live && h0 + i < h1) {
          const uint8_t* from = src[w] + (h0 + i) * src_sh[w];
          const uint8_t* step = steps[w] + (h0 + i) * steps_sh[w];
          if constexpr (G == 4) {
            const uint2 a = *reinterpret_cast<const uint2*>(from), d = *reinterpret_cast<const uint2*>(step);
            c[w][i][0] = a.x, c[w][i][1] = a.y, s[w][i][0] = d.x, s[w][i][1] = d.y;
          } else {
            c[w][i][0] = *reinterpret_cast<const uint32_t*>(from);
            s[w][i][0] = *reinterpret_cast<const uint32_t*>(step);
          }
        }
      }
#pragma unroll
    for (int i = 0; i < kGatherHeads; ++i)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (h0 + i >= h1) continue;
        uint8_t* to = out[w] + (h0 + i) * out_sh[w] + t * 8;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t h4 = c[w][i][g / 2] >> (16 * (g & 1));
          const float step = (g & 1) ? bf16hi_to_f32(s[w][i][g / 2]) : bf16lo_to_f32(s[w][i][g / 2]);
          float x[4];
          // code times step: 12 significant bits, rounded once; the code becomes a float as the
          // low bits of 2^23 + code
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = step * (__uint_as_float(0x4B000000u | ((h4 >> (4 * e)) & 15)) - 8388616.0f);
          *reinterpret_cast<uint2*>(to + g * 64) =
              live ? make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])) : make_uint2(0, 0);
        }
      }
  }
}

// Heads per thread of the gather: two, unless their threads would be fewer than 1024 per SM.
int gather_heads(int64_t rows, int tpr, int Hkv) {
  return Hkv > 1 && rows * tpr * Hkv >= kGatherHeads * 1024 * static_cast<int64_t>(paged_sm_count()) ? kGatherHeads : 1;
}

// Heads per block of the append: angles (about 2.6 times a row-head's other work, per row) are
// shared by the block's heads, heads behind the last one idle.
int append_heads(int Hkv) {
  int best = 1;
  double cost = 1e30;
  for (int hb = 8; hb >= 1; hb /= 2) {
    const double c = (Hkv + hb - 1) / hb * hb * (1.0 + 2.6 / hb);
    if (c < cost) cost = c, best = hb;
  }
  return best;
}

}  // namespace

cudaError_t launch_paged_append(PagedAppendParams p, int d, int format, bool rope, cudaStream_t stream) {
  const int tpr = format == kPagedQ4 ? 8 : d / 16;
  p.hb = append_heads(p.cache.Hkv);
  const int rb = kThreads / tpr / p.hb;
  p.rb_log2 = 0;
  while (1 << p.rb_log2 < rb) ++p.rb_log2;  // a power of two, as its factors
  void (*kern)(PagedAppendParams) = nullptr;
  if (format == kPagedQ4)
    kern = d == 128 ? (rope ? append_q4_kernel<128, true> : append_q4_kernel<128, false>)
                    : (rope ? append_q4_kernel<64, true> : append_q4_kernel<64, false>);
  else
    kern = d == 128 ? (rope ? append_bf16_kernel<128, true> : append_bf16_kernel<128, false>)
                    : (rope ? append_bf16_kernel<64, true> : append_bf16_kernel<64, false>);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.rows + rb - 1) / rb), (p.cache.Hkv + p.hb - 1) / p.hb);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = rope ? rb * (d / 2) * sizeof(float4) : 0;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_paged_gather(PagedGatherParams p, int d, int format, cudaStream_t stream) {
  const int tpr = format == kPagedQ4 ? 8 : d / 8;
  p.heads_per_thread = gather_heads(p.rows, tpr, p.cache.Hkv);
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
