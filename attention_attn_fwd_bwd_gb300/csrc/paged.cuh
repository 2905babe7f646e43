// The paged key/value cache: how a position finds its row, the 4-bit row format, and the
// rotation whose bf16 result does not depend on how it was computed.
//
// A cache is a pool of pages for K and one for V, each [num_pages, Hkv, page_size, row], and a
// table of page numbers per sequence: position p of sequence b is slot p % page_size of page
// table[b][p / page_size]. A row is d bf16 values (format bf16) or d/2 bytes of codes with d/32
// bf16 scales in a second pool (format q4).
//
// q4 rows. The d elements form groups of 32; element x of a group with scale s is stored as
// code + 8 in a nibble, code = round_half_away(x / s) in [-7, 7], s = bf16(max|x| / 7). The
// codes are interleaved so that one thread of a warp reads what it feeds to one column of
// matrix instructions with a single load: the row is 8 chunks of d/16 bytes; chunk r holds, for
// every group g, the 16-bit word of elements 32g + 4r .. 32g + 4r + 3, lowest nibble first. With
// d = 128 (8-byte chunks, 64-byte rows), slots with bit 1 set hold chunk r at place r ^ 4, so
// that four rows read at once fall in different shared-memory banks.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"

namespace afx {

constexpr int kPagedBf16 = 0, kPagedQ4 = 1;
constexpr int kQ4Group = 32;
// Positions stay exact in fp32 (the angle is pos * frequency with pos an fp32 number).
constexpr int kPagedMaxPos = 1 << 24;
constexpr int kPagedMaxPage = 1 << 16;

struct PagedDev {
  uint8_t *k, *v;                  // pools; all strides in bytes: page, head, slot
  int64_t k_sp, k_sh, k_st, v_sp, v_sh, v_st;
  uint8_t *ks, *vs;                // q4: scales (bf16), page and head strides; slots contiguous
  int64_t ks_sp, ks_sh, vs_sp, vs_sh;
  const int32_t* table;
  int64_t table_stride;
  uint64_t div_mul;                // ceil(2^40 / page_size)
  int num_pages, page_size, max_pages;
  int cap;                         // max_pages * page_size (at most kPagedMaxPos)
  int B, Hkv;
};

// Launch parameters. Strides of the dense sides are in bytes, the innermost is one element.
struct PagedAppendParams {
  PagedDev cache;
  const uint8_t *k, *v;             // bf16 [B, Hkv, N, d]
  int64_t k_sb, k_sh, k_sn, v_sb, v_sh, v_sn;
  const int32_t *first, *count;     // [B]; count may be null: every sequence has N rows
  int N;
  int64_t rows;                     // B * N
  int heads_per_thread;             // set by the launcher
  RopeFreqs freqs;
  int* status;
};
struct PagedGatherParams {
  PagedDev cache;
  uint8_t *k, *v;                   // bf16 [B, Hkv, N, d]
  int64_t k_sb, k_sh, k_sn, v_sb, v_sh, v_sn;
  const int32_t *first, *count;     // [B]; first may be null (0), count too (N)
  int N;
  int64_t rows;
  int heads_per_thread;
  int* status;
};
struct PagedDecodeParams {
  PagedDev cache;
  const __nv_bfloat16* q;           // [B, Hq, d], element strides
  int64_t q_sb, q_sh;
  __nv_bfloat16* out;
  int64_t o_sb, o_sh;
  float* lse;                       // [B, Hq] or null
  const int32_t* lens;              // [B]
  int Hq, g;
  int window;                       // 0: none
  const float* slopes;              // [Hq] or null
  int rope;
  float scale_log2;
  CUtensorMap tmK, tmV;             // bf16: pools [num_pages, Hkv, page_size, d], box (64, frag_rows)
  int frag_rows;                    // rows of a page that one copy takes
  void* workspace;
  // set by the launcher
  float* part_acc;                  // [ctas][2][head_rows][d]: partial rows of a run's ends
  float2* part_ml;                  // (max in log2 units, sum)
  int ctas, head_rows;              // query heads per item
  int chunks, items;                // items per KV head, and per sequence
  RopeFreqs freqs;
  int* status;
};
constexpr int kPagedMaxCtas = 1024;
cudaError_t launch_paged_append(PagedAppendParams p, int d, int format, bool rope, cudaStream_t stream);
cudaError_t launch_paged_gather(PagedGatherParams p, int d, int format, cudaStream_t stream);
size_t paged_decode_workspace(int d, int g, int format);
int paged_frag_rows(int page_size);
cudaError_t launch_paged_decode(const PagedDecodeParams& p, int d, int format, cudaStream_t stream);

// pos / page_size for 0 <= pos < 2^24: pos * (M d - 2^40) < 2^24 * 2^16 keeps the error of
// the rounded-up reciprocal M below 1 / page_size.
__device__ __forceinline__ int page_div(const PagedDev& c, int pos) {
  return static_cast<int>((static_cast<uint64_t>(pos) * c.div_mul) >> 40);
}

// Page number of position pos of sequence b (pos in range), or -1 if the table's entry is none.
__device__ __forceinline__ int page_at(const PagedDev& c, int b, int pos, int* slot) {
  const int i = page_div(c, pos);
  *slot = pos - i * c.page_size;
  const int page = __ldg(c.table + b * c.table_stride + i);
  return static_cast<uint32_t>(page) < static_cast<uint32_t>(c.num_pages) ? page : -1;
}

// The place of chunk r in the row of a slot (see the head of this file).
template <int D>
__device__ __forceinline__ int q4_place(int r, int slot) {
  return D == 128 ? r ^ (((slot >> 1) & 1) << 2) : r;
}

// ---------------------------------------------------------------------------------------------
// Rotation with a reproducible bf16 result
//
// A 4-bit code jumps by a whole step where a value crosses a border between two codes, so the
// rotated key is defined as the exact R_p k rounded to fp32 and then to bf16, whatever
// computes it. The fast path is fp32: (cos, sin) within 2^-22.9 (sincospif and the residual of
// the reduced angle), two roundings on top: |error| < 2^-21.5 (|x_lo| + |x_hi|). Where that
// interval holds a border between two bf16 values (about 3 elements in 10^4) the element is
// computed again in fp64.
// ---------------------------------------------------------------------------------------------

// (cos, sin) of 2 pi * pos * (hi + lo) as rope_cossin, with the rounding of the reduced angle
// put back: the residual rl (turns) turns (c, s) by 2 pi rl to first order.
__device__ __forceinline__ void rope_cossin_fine(float pos, float hi, float lo, float* c, float* s) {
  const float prod = __fmul_rn(pos, hi);
  const float err = __fmaf_rn(pos, hi, -prod);
  const float frac = __fsub_rn(prod, rintf(prod));
  const float low = __fmaf_rn(pos, lo, err);
  const float r = __fadd_rn(frac, low);
  const float bb = __fsub_rn(r, frac);
  const float rl = __fadd_rn(__fsub_rn(frac, __fsub_rn(r, bb)), __fsub_rn(low, bb));
  float c0, s0;
  sincospif(__fmul_rn(2.0f, r), &s0, &c0);
  const float dl = __fmul_rn(6.283185307179586f, rl);
  *c = __fmaf_rn(-s0, dl, c0);
  *s = __fmaf_rn(c0, dl, s0);
}

// One pair in fp64, rounded to fp32.
static __device__ __noinline__ void rot_pair_f64(float xl, float xh, float pos, float hi, float lo, float* yl,
                                          float* yh) {
  const double p = pos;
  double t = p * static_cast<double>(hi);  // 24 x 24 bits: exact
  t -= rint(t);
  t += p * static_cast<double>(lo);
  double s, c;
  sincospi(2.0 * t, &s, &c);
  *yl = static_cast<float>(static_cast<double>(xl) * c - static_cast<double>(xh) * s);
  *yh = static_cast<float>(static_cast<double>(xh) * c + static_cast<double>(xl) * s);
}

// Two consecutive pairs (i, i + 1), each word a bf16x2: rotated and rounded to bf16.
__device__ __forceinline__ void rot_word_exact(uint32_t& lo, uint32_t& hi, const float (&c)[2],
                                               const float (&s)[2], float pos, const RopeFreqs& f, int i) {
  const float xl0 = bf16lo_to_f32(lo), xl1 = bf16hi_to_f32(lo);
  const float xh0 = bf16lo_to_f32(hi), xh1 = bf16hi_to_f32(hi);
  float yl0, yh0, yl1, yh1;
  rot_pair(xl0, xh0, c[0], s[0], yl0, yh0);
  rot_pair(xl1, xh1, c[1], s[1], yl1, yh1);
  const float e0 = 3.4e-7f * (fabsf(xl0) + fabsf(xh0));  // 2^-21.5
  const float e1 = 3.4e-7f * (fabsf(xl1) + fabsf(xh1));
  const uint32_t wl = pack_bf16x2(yl0 + e0, yl1 + e1), wh = pack_bf16x2(yh0 + e0, yh1 + e1);
  if (wl != pack_bf16x2(yl0 - e0, yl1 - e1) || wh != pack_bf16x2(yh0 - e0, yh1 - e1)) {
    rot_pair_f64(xl0, xh0, pos, f.hi[i], f.lo[i], &yl0, &yh0);
    rot_pair_f64(xl1, xh1, pos, f.hi[i + 1], f.lo[i + 1], &yl1, &yh1);
    lo = pack_bf16x2(yl0, yl1);
    hi = pack_bf16x2(yh0, yh1);
  } else {
    lo = wl;
    hi = wh;
  }
}

}  // namespace afx
