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
#include "turn_table.cuh"

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

// theta^(-2i/d) / (2 pi) for i < d/2 as the sum of three floats (about 72 bits), less whole numbers: x + y + z.
// (w: with positions on several axes, the pair's axis, an integer's bits.)
struct PagedFreqs {
  float4 f[64];
};

// Launch parameters. Strides of the dense sides are in bytes, the innermost is one element.
struct PagedAppendParams {
  PagedDev cache;
  const uint8_t *k, *v;             // bf16 [B, Hkv, N, d]
  int64_t k_sb, k_sh, k_sn, v_sb, v_sh, v_sn;
  const int32_t *first, *count;     // [B]; count may be null: every sequence has N rows
  int N;
  int64_t rows;                     // B * N, below 2^31
  uint64_t div_n;                   // ceil(2^64 / N): row / N as a multiplication; 0 for N = 1
  int hb, rb_log2;                  // heads and (log2) rows of a block, set by the launcher
  PagedFreqs freqs;
  int* status;
};
struct PagedGatherParams {
  PagedDev cache;
  uint8_t *k, *v;                   // bf16 [B, Hkv, N, d]
  int64_t k_sb, k_sh, k_sn, v_sb, v_sh, v_sn;
  const int32_t *first, *count;     // [B]; first may be null (0), count too (N)
  int N;
  int64_t rows;
  uint64_t div_n;
  int heads_per_thread;
  int* status;
};
// What the combine kernel needs of them, too.
struct PagedCombineParams {
  PagedDev cache;
  __nv_bfloat16* out;               // [B, Hq, d], element strides
  int64_t o_sb, o_sh;
  float* lse;                       // [B, Hq] or null
  const int32_t* lens;              // [B]
  int Hq, g;
  int window;                       // 0: none
  // set by the launcher
  int ctas, head_rows;              // query heads per item
  int chunks, items;                // items per KV head, and per sequence
  int whole;                        // items are not cut: no partial rows, no combine kernel
  int comb_by_run, comb_heads;      // the combine kernel's blocks
  float* part_acc;                  // [ctas][2][head_rows][d]: partial rows of a run's ends
  float2* part_ml;                  // (max in log2 units, sum)
};
struct PagedDecodeParams : PagedCombineParams {
  const __nv_bfloat16* q;           // [B, Hq, d]
  int64_t q_sb, q_sh;
  const float* slopes;              // [Hq] or null
  int rope;
  float scale_log2;
  CUtensorMap tmK, tmV;             // bf16: pools [num_pages, Hkv, page_size, d], box (64, frag_rows)
  int frag_rows;                    // rows of a page that one copy takes
  void* workspace;
  PagedFreqs freqs;
  int* status;
};
// Attention of a chunk (paged_attend.cu): what the kernel that joins cut work needs, what the one
// that makes its query operands does, and the main kernel's own.
struct PagedAttendPos {  // where a run begins: tile t of unit (b, kvh, r)
  int b, kvh, r, t;
};
struct PagedAttendWork {
  PagedDev cache;
  const int32_t *first, *count;     // [B]; count may be null: every sequence has N rows
  int Hq, g, N;
  int window;                       // 0: none
  __nv_bfloat16* out;               // [B, Hq, N, d], element strides
  int64_t o_sb, o_sh, o_sn;
  float* lse;                       // [B, Hq, N] or null
  int ctas, unit, unit_log2;        // CTAs, and rows of a unit (128 or 256)
  int half_cost;                    // of a unit of one row tile among those of two, in quarters
  uint64_t div_g;                   // ceil(2^63 / g)
  PagedAttendPos* bounds;           // [ctas], written by the main kernel
  float* part_acc;                  // [ctas][2][unit][d]: partial rows of a run's ends
  float2* part_ml;                  // (max in log2 units, sum)
};
struct PagedQueryParams {
  const uint8_t* q;                 // bf16 [B, Hq, N, d], byte strides
  int64_t q_sb, q_sh, q_sn;
  const int32_t *first, *count;
  int cap, Hq, N;
  int64_t rows;                     // B * N
  uint64_t div_n;
  uint16_t *hi, *lo;                // 16-bit parts [B, Hq, N, d]; lo null: one part
  float* factor;                    // [B, Hq, N], 4-bit caches: what the parts of a row are to be multiplied by
  int rb_log2;
  PagedFreqs freqs;
};
struct PagedAttendParams : PagedAttendWork {
  const __nv_bfloat16* q;           // bf16 rows as they are, or the first parts; element strides
  int64_t q_sb, q_sh, q_sn;
  int64_t q_lo;                     // elements from a first part to its second
  const float* factor;
  const float* slopes;              // [Hq] or null
  float scale_log2;
  CUtensorMap tmK, tmV;             // bf16: pools [num_pages, Hkv, page_size, d], box (64, frag_rows)
  CUtensorMap tmV16, tmV1;          // and of 16 rows, of one
  int frag_rows;                    // rows of a page that one copy takes
  int* status;
};
// What the C entry point hands over.
struct PagedAttendCall {
  PagedAttendParams p;
  PagedFreqs freqs;
  int rope;
  void* workspace;
};
constexpr int kAttendTile = 128;    // keys
size_t paged_attend_workspace(int B, int Hq, int Hkv, int N, int d, int format, bool rope);
cudaError_t launch_paged_attend(const PagedAttendCall& c, int d, int format, cudaStream_t stream);
// Rotation by given positions (rope_axes.cu): q and k [B, H, N, d] bf16, byte strides (b, h, n).
struct RopeAxesParams {
  const uint8_t *x[2];              // q, k
  uint8_t *y[2];
  int64_t x_sb[2], x_sh[2], x_sn[2], y_sb[2], y_sh[2], y_sn[2];
  int Hq, H;                        // heads of q, of both
  int N;
  int64_t rows;                     // B * N, below 2^31
  uint64_t div_n;                   // as PagedAppendParams
  const int32_t* pos;               // [axes, B, N], element strides
  int64_t pos_sa, pos_sb, pos_sn;
  int inverse;
  int rb_log2, passes;              // (log2) rows of a block, heads in turn per thread: set by the launcher
  PagedFreqs freqs;
};
cudaError_t launch_rope_axes(RopeAxesParams p, int d, cudaStream_t stream);
constexpr int kPagedMaxCtas = 1024;
int paged_sm_count();  // SMs of the current device
cudaError_t launch_paged_append(PagedAppendParams p, int d, int format, bool rope, cudaStream_t stream);
cudaError_t launch_paged_gather(PagedGatherParams p, int d, int format, cudaStream_t stream);
size_t paged_decode_workspace(int d, int g, int format);
// Rows of a page that one copy takes: the largest that pages and tiles are both whole multiples of.
int paged_frag_rows(int page_size, int d, int g, int format);
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
// rotated key is R_p k, off by at most 2^-34 (|x| + |y|) for a pair (x, y), rounded to fp32 and then
// to bf16: one element in some 10^8 differs from the exact one's rounding. fp32 alone would move
// about one in 10^6, and the GPU's fp64 units are few (a first version recomputed doubtful elements
// in fp64: 126 us for 18.5k rows of 8 heads, d = 128, of which 20 are traffic; now 28). So angles and
// products are carried as the sum of two floats, to 2^-35: some 60 instructions per angle, shared by
// the heads of a block, and 11 packed ones per pair and head.
// ---------------------------------------------------------------------------------------------

// Entry i of the frequencies, which are a kernel parameter: through a generic address, since an
// indexed read of constant memory takes one pass per different index of the warp.
__device__ __forceinline__ float4 freq_at(const PagedFreqs& f, int i) {
  float4 v;
  asm("ld.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(f.f + i));
  return v;
}

// pos (f.x + f.y + f.z) less whole numbers, as r + lo: |pos| <= 2^24 a whole number.
struct Turns {
  float r, lo;
};
__device__ __forceinline__ Turns turns_of(float pos, float f1, float f2, float f3) {
  const float p1 = __fmul_rn(pos, f1), e1 = __fmaf_rn(pos, f1, -p1);
  const float frac = __fsub_rn(p1, rintf(p1));
  const float p2 = __fmul_rn(pos, f2), e2 = __fmaf_rn(pos, f2, -p2);
  const float a = __fadd_rn(e1, p2), ab = __fsub_rn(a, e1);
  const float ea = __fadd_rn(__fsub_rn(e1, __fsub_rn(a, ab)), __fsub_rn(p2, ab));
  const float r = __fadd_rn(frac, a), rb = __fsub_rn(r, frac);
  const float er = __fadd_rn(__fsub_rn(frac, __fsub_rn(r, rb)), __fsub_rn(a, rb));
  return {r, __fadd_rn(__fadd_rn(er, ea), __fmaf_rn(pos, f3, e2))};
}

// (cos, sin) of 2 pi (t.r + t.lo), each as hi + lo, hi a multiple of 2^-16 (so that its
// product with a bf16 is exact in fp32). The angle's
// nearest multiple of 1/256 of a turn is looked up (table-driven reduction as in Tang, "Table-driven
// implementation of the exponential function", 1989) and the rest, |d| <= 2 pi / 512, added by
// the angle-sum formulas with Taylor series to d^5. d is dh + dl, |dl| < 2^-23; of its powers in dl,
// dl (sine) and dh dl (cosine, up to 2^-29) count. Against 113-bit arithmetic the largest error in
// 10^6 angles of positions below 2^24 was 2^-35.3.
__device__ __forceinline__ float4 cossin_of(const Turns& t) {
  const float r = t.r, lo = t.lo;
  const float kf = rintf(__fmul_rn(r, 256.0f));
  const float rs = __fmaf_rn(kf, -1.0f / 256.0f, r);  // exact
  const int k = static_cast<int>(kf);
  const float4 T = __ldg(kTurn256 + (k & 63));
  constexpr float kTwoPiHi = 0x1.921fb6p+2f, kTwoPiLo = -0x1.777a5cp-23f;
  const float dh = __fmul_rn(rs, kTwoPiHi);
  const float dl = __fmaf_rn(rs, kTwoPiLo, __fmaf_rn(lo, kTwoPiHi, __fmaf_rn(rs, kTwoPiHi, -dh)));
  const float d2 = __fmul_rn(dh, dh);
  const float u = __fmaf_rn(-dh, dl, __fmul_rn(d2, __fmaf_rn(d2, 1.0f / 24.0f, -0.5f)));          // cos d - 1
  const float v = __fmaf_rn(__fmul_rn(dh, d2), __fmaf_rn(d2, 1.0f / 120.0f, -1.0f / 6.0f), dl);  // sin d - dh
  const float pc = __fmul_rn(T.z, dh), pce = __fmaf_rn(T.z, dh, -pc);
  float tc = __fmaf_rn(T.x, u, T.y);
  tc = __fmaf_rn(-T.z, v, tc);
  tc = __fmaf_rn(-T.w, dh, tc);
  const float c = __fsub_rn(T.x, pc);
  const float ce = __fadd_rn(__fsub_rn(__fsub_rn(T.x, c), pc), __fsub_rn(tc, pce));
  const float ps = __fmul_rn(T.x, dh), pse = __fmaf_rn(T.x, dh, -ps);
  float ts = __fmaf_rn(T.z, u, T.w);
  ts = __fmaf_rn(T.x, v, ts);
  ts = __fmaf_rn(T.y, dh, ts);
  const float s = __fadd_rn(T.z, ps);
  const float se = __fadd_rn(__fsub_rn(ps, __fsub_rn(s, T.z)), __fadd_rn(ts, pse));
  // 192 + x rounds x to a multiple of 2^-16
  const float ch = __fsub_rn(__fadd_rn(c, 192.0f), 192.0f), cl = __fadd_rn(__fsub_rn(c, ch), ce);
  const float sh = __fsub_rn(__fadd_rn(s, 192.0f), 192.0f), sl = __fadd_rn(__fsub_rn(s, sh), se);
  // quarter turns: (c, s) -> (-s, c) -> (-c, -s) -> (s, -c)
  const int q = (k >> 6) & 3;
  const float4 w = (q & 1) ? make_float4(-sh, -sl, ch, cl) : make_float4(ch, cl, sh, sl);
  return (q & 2) ? make_float4(-w.x, -w.y, -w.z, -w.w) : w;
}

__device__ __forceinline__ float4 turn_cossin(float pos, const float4& f) {
  return cossin_of(turns_of(pos, f.x, f.y, f.z));
}

// The same for any 32-bit position: from 2^24 on as 2^12 (pos >> 12) + the rest, whose turns are
// added (2^12 times a frequency's parts are exact, less whole numbers in the first).
__device__ __forceinline__ float4 turn_cossin_far(int pos, const float4& f) {
  if (pos <= kPagedMaxPos && pos >= -kPagedMaxPos) return turn_cossin(static_cast<float>(pos), f);
  const float x = __fmul_rn(4096.0f, f.x);
  const Turns a = turns_of(static_cast<float>(pos >> 12), __fsub_rn(x, rintf(x)), __fmul_rn(4096.0f, f.y), __fmul_rn(4096.0f, f.z));
  const Turns b = turns_of(static_cast<float>(pos & 4095), f.x, f.y, f.z);
  const float ra = __fsub_rn(a.r, rintf(a.r)), rb = __fsub_rn(b.r, rintf(b.r));  // exact
  const float s = __fadd_rn(ra, rb), bb = __fsub_rn(s, ra);
  const float es = __fadd_rn(__fsub_rn(ra, __fsub_rn(s, bb)), __fsub_rn(rb, bb));
  const float sr = __fsub_rn(s, rintf(s)), lo = __fadd_rn(es, __fadd_rn(a.lo, b.lo));
  const float r = __fadd_rn(sr, lo);
  return cossin_of({r, __fsub_rn(lo, __fsub_rn(r, sr))});
}

// x c + y s of two lanes, c and s as hi + lo: h + t, h the rounded sum of the (exact) products
// with the hi parts, t what that rounding lost and the products with the lo parts.
__device__ __forceinline__ void dot2_exact(uint64_t x, uint64_t y, uint64_t ch, uint64_t cl, uint64_t sh, uint64_t sl,
                                           uint64_t& h, uint64_t& t) {
  const uint64_t m1 = f2_pack(-1.0f, -1.0f);
  const uint64_t p1 = mul2(x, ch), p2 = mul2(y, sh);
  h = add2(p1, p2);
  const uint64_t bb = fma2(p1, m1, h);
  const uint64_t er = add2(fma2(fma2(bb, m1, h), m1, p1), fma2(bb, m1, p2));
  t = fma2(x, cl, fma2(y, sl, er));
}

// Two consecutive pairs, each word a bf16x2, rotated by the two angles packed in ch .. sl.
__device__ __forceinline__ void rot_word_exact(uint32_t& lo, uint32_t& hi, uint64_t ch, uint64_t cl, uint64_t sh,
                                               uint64_t sl) {
  constexpr uint64_t kSigns = 0x8000000080000000ull;
  const uint64_t xl = bf16x2_to_f2(lo), xh = bf16x2_to_f2(hi);
  uint64_t h0, t0, h1, t1;
  dot2_exact(xl, xh ^ kSigns, ch, cl, sh, sl, h0, t0);  // xl c - xh s
  dot2_exact(xh, xl, ch, cl, sh, sl, h1, t1);  // xh c + xl s
  const uint64_t y0 = add2(h0, t0), y1 = add2(h1, t1);
  lo = pack_bf16x2(f2_lo(y0), f2_hi(y0));
  hi = pack_bf16x2(f2_lo(y1), f2_hi(y1));
  const uint32_t big = __vmaxu2(lo & 0x7FFF7FFFu, hi & 0x7FFF7FFFu);
  if (big >= 0x7F800000u || (big & 0xFFFFu) >= 0x7F80u) {
    // an infinity makes the error terms NaN: the rounded sum itself is the value
    auto pick = [](float y, float h) { return y == y ? y : h; };
    lo = pack_bf16x2(pick(f2_lo(y0), f2_lo(h0)), pick(f2_hi(y0), f2_hi(h0)));
    hi = pack_bf16x2(pick(f2_lo(y1), f2_lo(h1)), pick(f2_hi(y1), f2_hi(h1)));
  }
}

}  // namespace afx
