// Decode over a paged cache for sm_103a: one query per sequence against that sequence's own length.
//
//   O_h = sum_n p_n v_n,  p = softmax over n in [max(0, L - W), L) of
//   s_n = scale <R_{L-1} q_h, k_n> + slope_h (n - (L - 1)),  L = lens[b].
//
// The cache is read once, from HBM, and that bounds the bf16 kernel (8 sequences of 32768 keys,
// Hq = 64, Hkv = 8, d = 128: 162 us, 97% of a copy's rate). The matrix instructions are warp-level
// ones with the KEYS as rows (S^T = K Q^T, O^T = V^T P^T): their operands come straight from
// registers, which is where 4-bit codes have to be expanded (writing them back to shared memory as
// 16-bit values for tcgen05 would move 94 of the 128 bytes per cycle that shared memory has, and as
// much again to read them), and a group of 8 query heads fills the instruction's 8 columns, where
// a 128-row query tile would be padding.
//
// The 4-bit kernel (the same sequences: 87 us, 51% of a copy's rate) is bound by no single unit: the
// tensor pipe is busy 36% of the time, integer logic 48%, issue slots 55%, and three consumer warps
// per scheduler, at 128 registers with a few of them spilled (48 bytes a thread; 372 bytes at 168
// registers for more than 8 heads on a KV head), leave latencies in the open. Its loads alone,
// without any arithmetic, take 52 to 63 us. Of what can be cut, products weigh most: measured on
// GB300, a warp-level product takes a sub-partition 8 cycles and no FMA-pipe instruction runs beside
// it (packed fp16 takes that pipe 2 cycles), while integer logic (2 cycles each) does. So codes are
// expanded by logic alone, and what that leaves out, the offset of the codes, is taken out by
// products of a constant.
//
// Work. Sequences are cut into tiles of 64 or 128 keys; the tiles of the whole batch, ordered by
// (sequence, KV head, chunk of query heads), are dealt to the CTAs in equal runs, from lengths read
// on the device; an item counts for its tiles and for what its two ends cost (without that, 64
// sequences of 1 to 8192 keys took 121 us from the 4-bit cache where they took 98 with it). A CTA
// walks the segments of its run. A segment that is a whole item (all tiles of one (sequence, head chunk)) is
// finished in place; otherwise its (max, sum, acc) goes to the workspace, at most two per CTA, and
// the combine kernel joins them in a fixed order. In caches of short sequences every segment is a
// whole item, and there is no second kernel.
//
// CTA: 4 consumer warps, each with its own keys of every tile and its own running (max, sum, acc)
// (joined once per segment), and a producer warp that looks pages up and fills a ring of tiles: TMA
// boxes of one page's rows (bf16, 128-byte swizzle) or bulk copies (q4: codes and steps of a
// page's rows are contiguous). Warps that filled rings of their own, without a producer, took 8%
// (bf16) and 14% (q4) longer.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "launch.h"
#include "paged.cuh"

namespace afx {

namespace {

constexpr int kWarps = 4;              // consumers
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;
constexpr float kLazy = 8.0f;          // the running maximum may lag by 2^8

// Weights from a 4-bit cache enter the second product as ONE fp16 of p * step * mul, mul a power of
// two for each head and group (a second fp16 would cost 16 more products per 16 keys, of 32). mul
// takes the largest p * step that the warp has seen in its segment, not the largest step, to
// 2^kWeightBits or more: a key of large values that a head gives no weight leaves the other keys
// their bits. It is renewed where a step * mul passes 2^kStepBits or the maximum is renewed, which
// may lag by 2^kLazyQ4, so weights stay below 2^15. They have their 11 bits down to 2^-14 and are
// off by at most 2^-25 below that: n keys together by n 2^-(25 + kWeightBits) of the largest.
// (8 x 32k keys, 64 heads, normal values: 86.5 us, with one mul for all heads, from the largest
// step alone, 85; values of sizes e^(2z), z normal: 90 and 85; a first key 2^10 above the others
// with values 1/64 of theirs, after which every tile of its segment renews mul: 104 and 85.
// kLazyQ4, kWeightBits, kStepBits 3, 5, 11: 87, 94, 107; 5, 3, 10: 86.5, 89, 105; 3, 4, 12: 87, 89, 88.)
constexpr float kLazyQ4 = 4.0f;
constexpr uint32_t kWeightBits = 4, kStepBits = 11;
constexpr uint32_t kFirstMul = 253;    // biased exponent before any key: every step renews it

template <int D, int NT, bool Q4, bool PK>
struct Cfg {
  // PK (q4, at most 4 heads): columns 0-3 of the column tile take the heads' first parts of q,
  // columns 4-7 the second ones, and the scores of both are added. One product then does for two
  // (64 sequences of 1 to 8192 keys, 4 heads on each KV head: 88 us, without 96).
  static constexpr int ROWS = PK ? 4 : 8 * NT;                          // query heads per item
  // 16-key blocks of a tile per warp: two hide each other's latencies and share the per-tile
  // work (q4, 8 x 32k keys, 64 heads: 87 us, with one 102); rows of 256 bytes (bf16, d = 128) keep
  // the HBM busy with one.
  static constexpr int BPW = Q4 || D == 64 ? 2 : 1;
  static constexpr int TILE = kWarps * 16 * BPW;                        // keys
  // What the two ends of a segment cost, in tiles: items count as so many more when work is dealt.
  static constexpr int ENDS = Q4 ? 2 : 1;
  static constexpr uint32_t KB = TILE * (Q4 ? D / 2 : 2 * D);           // K (and V) bytes of a tile
  static constexpr uint32_t SB = Q4 ? TILE * (D / 16) : 0;              // and their steps
  static constexpr uint32_t STAGE = 2 * KB + 2 * SB;
  // bf16 with one column tile keeps its query operands in registers, the others read them again
  // for every tile (of 16 heads, d = 128: one CTA per SM with, two CTAs without, 193 and 172 us for
  // 8 x 32k keys)
  static constexpr bool QREG = !Q4 && NT == 1;
  // (q4, one column tile: four CTAs, of 96 registers a thread, 117 us; 8 consumer warps in each of
  // two CTAs 103)
  static constexpr int CTAS = Q4 ? (NT == 1 ? 3 : 2) : 2;
  static constexpr int STAGES = Q4 || (NT == 2 && D == 128) ? 2 : 3;
  static constexpr uint32_t QROW = 2 * D + 16;                          // padded query row
  static constexpr uint32_t QFRAG = 512 * (D / 32);                     // q4: a column tile's fragments
  static constexpr uint32_t OFF_Q = STAGES * STAGE;
  static constexpr uint32_t OFF_O = OFF_Q + (Q4 ? 2 * NT * QFRAG : 3 * ROWS * QROW);  // two warps' accumulators
  static constexpr uint32_t OBUF = (D / 16) * NT * 512;
  static constexpr uint32_t OFF_CTL = OFF_O + 2 * OBUF;
};

struct Ctl {
  uint64_t full[8], empty[8];
  uint32_t frags[8];                   // fragments of the tile that were loaded
  int abort_flag;
  int b0;                              // first sequence of this CTA's run, and the units of it
  int rem0;                            // before the run
  int64_t wsum[kThreads / 32];
  float m[kWarps][16], l[kWarps][16];
  float slope[16];                     // ALiBi slopes over c2
  float2 qsum[2][4][4];                // q4: minus 8 times a column's sum, per column tile, group, column pair
  float qmax[16][2];                   // q4: largest |q| of a head, by half rows
};

template <int D, int NT, bool Q4, bool PK>
constexpr size_t smem_bytes() {
  return 1024 + Cfg<D, NT, Q4, PK>::OFF_CTL + sizeof(Ctl);
}

// ---------------------------------------------------------------------------------------------
// Warp-level matrix instructions and shared-memory fragments
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Transpose of an 8x8 b16 matrix held one row pair per lane.
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// D (16 x 8, fp32) = A (16 x 16) B (16 x 8) + C
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma_bf16_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from c0, c1 in both row halves.
__device__ __forceinline__ void mma_f16_c(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                          float c1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %10, %11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t w;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(x), "r"(y));
  return w;
}
// (saturating: scores past 2^25, whose neighbours lie 4 apart in fp32, may pass a lagging maximum by more)
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
// Bulk copy of `bytes` (a multiple of 16; both addresses 16-byte aligned) that completes on bar.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// ---------------------------------------------------------------------------------------------
// Work: lengths -> tiles -> this CTA's run
// ---------------------------------------------------------------------------------------------
struct Span {
  int L, first, t0, nt;  // visible keys [first, L), first tile, tiles
};

template <int TILE>
__device__ __forceinline__ Span span_of(const PagedCombineParams& p, int b) {
  Span s;
  s.L = min(max(__ldg(p.lens + b), 0), p.cache.cap);
  s.first = p.window > 0 && s.L > p.window ? s.L - p.window : 0;
  s.t0 = s.first / TILE;
  s.nt = s.L > 0 ? (s.L - 1) / TILE - s.t0 + 1 : 0;
  return s;
}

// Exclusive prefix over the block's threads of v, and the total (all threads call).
template <int NTHREADS>
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t* wsum, int64_t* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NTHREADS / 32; ++w) {
    if (w < warp) before += wsum[w];
    all += wsum[w];
  }
  *total = all;
  return before + x - v;
}

__device__ __forceinline__ int64_t div_units(int64_t a, int64_t b) {  // a / b, a >= 0, b > 0
  return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// T units in equal runs over min(ctas, T) CTAs, so that no run is empty; the first `more` runs are
// one unit longer.
struct Deal {
  int64_t each, more;
  int runs;
  __device__ Deal(int64_t T, int ctas) {
    runs = T < ctas ? static_cast<int>(T) : ctas;
    each = runs ? div_units(T, runs) : 0;
    more = T - each * runs;
  }
  __device__ int64_t start(int i) const { return i * each + min(static_cast<int64_t>(i), more); }
  __device__ int run_of(int64_t unit) const {
    const int64_t longer = more * (each + 1);
    return static_cast<int>(unit < longer ? div_units(unit, each + 1) : more + div_units(unit - longer, each));
  }
};

// An item is `ends` units without tiles, then one per tile; or one unit where items are not cut.
template <class C>
__device__ __forceinline__ int units_of(const PagedCombineParams& p, const Span& s) {
  return s.nt ? (p.whole ? 1 : s.nt + C::ENDS) : 0;
}

// Walks the segments of a run that have tiles: all roles step through the same ones.
template <class C>
struct Walk {
  const PagedDecodeParams& p;
  Span s;
  int b, hh, u, left;     // item (b, hh), and in units: where in it the run goes on, what the run has left
  int t, n;               // first tile of the segment (within the item), its tiles
  bool head;              // the segment is the run's first
  __device__ Walk(const PagedDecodeParams& p_, int b0, int rem0, int left_) : p(p_), b(b0), left(left_), n(0), head(true) {
    if (left <= 0) return;
    s = span_of<C::TILE>(p, b);
    hh = rem0 / units_of<C>(p, s);
    u = rem0 - hh * units_of<C>(p, s);
    find();
  }
  __device__ bool live() const { return n > 0; }
  __device__ bool whole() const { return n == s.nt; }
  __device__ void next() {
    head = false;
    find();
  }

 private:
  __device__ void find() {
    for (n = 0; n == 0 && left > 0;) {
      if (u == units_of<C>(p, s)) {
        u = 0;
        if (++hh == p.items) {
          hh = 0;
          do s = span_of<C::TILE>(p, ++b);
          while (s.nt == 0);
        }
      }
      const int take = min(left, units_of<C>(p, s) - u);
      t = p.whole ? 0 : max(0, u - C::ENDS);
      n = p.whole ? s.nt : max(0, u + take - C::ENDS) - t;
      u += take;
      left -= take;
    }
  }
};

// ---------------------------------------------------------------------------------------------
// Producer
// ---------------------------------------------------------------------------------------------
template <int D, int NT, bool Q4, bool PK>
__device__ __forceinline__ void produce(const PagedDecodeParams& p, uint8_t* smem, Ctl* ctl,
                                        Walk<Cfg<D, NT, Q4, PK>> w) {
  using C = Cfg<D, NT, Q4, PK>;
  constexpr int kTile = C::TILE;
  const int lane = threadIdx.x % 32;
  const PagedDev& c = p.cache;
  const int F = p.frag_rows, nf = kTile / F;
  int it = 0, st = 0;
  uint32_t phase = 1;  // of `empty`: the first round finds every stage free
  bool ok = true;
  for (; w.live() && ok; w.next()) {
    const int kvh = w.hh / p.chunks;
    // fragments of F rows, one per lane and 32 at a time, looked up one window ahead
    int base = (w.s.t0 + w.t) * nf;
    const int end = base + w.n * nf;
    auto look = [&](int f, int* slot, bool* bad) {
      const int pos = f * F;
      const bool need = f < end && pos < w.s.L && pos + F > w.s.first;
      *slot = 0;
      const int page = need ? page_at(c, w.b, pos, slot) : -1;
      *bad = need && page < 0;
      return page;
    };
    int slot, slot_n;
    bool bad, bad_n;
    int page = look(base + lane, &slot, &bad);
    int page_n = look(base + 32 + lane, &slot_n, &bad_n);
    for (int i = 0; i < w.n; ++i, ++it, st = st + 1 == C::STAGES ? 0 : st + 1, phase ^= st == 0) {
      const int f0 = (w.s.t0 + w.t + i) * nf;
      if (f0 == base + 32) {
        base += 32;
        page = page_n, slot = slot_n, bad = bad_n;
        page_n = look(base + 32 + lane, &slot_n, &bad_n);
      }
      if (it >= C::STAGES) ok = mbar_wait(&ctl->empty[st], phase, p.status, &ctl->abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int src = (f0 - base + lane) & 31;
      const int pg = __shfl_sync(0xffffffffu, page, src), sl = __shfl_sync(0xffffffffu, slot, src);
      const bool bd = __shfl_sync(0xffffffffu, bad, src);
      const bool mine = lane < nf && pg >= 0;
      const uint32_t got = __ballot_sync(0xffffffffu, mine);
      if (lane < nf && bd) atomicOr(p.status, kDevPageRange);
      uint8_t* stage = smem + st * C::STAGE;
      if (lane == 0) {
        ctl->frags[st] = got;
        mbar_arrive_expect_tx(&ctl->full[st], __popc(got) * F * (C::STAGE / kTile));
      }
      __syncwarp();
      if (mine) {
        if constexpr (Q4) {
          const uint32_t dst = smem_u32(stage);
          const uint32_t cb = F * (D / 2), sb = F * (D / 16);
          bulk_load(dst + lane * cb, c.k + pg * c.k_sp + kvh * c.k_sh + sl * (D / 2), cb, &ctl->full[st]);
          bulk_load(dst + C::KB + lane * cb, c.v + pg * c.v_sp + kvh * c.v_sh + sl * (D / 2), cb, &ctl->full[st]);
          bulk_load(dst + 2 * C::KB + lane * sb, c.ks + pg * c.ks_sp + kvh * c.ks_sh + sl * (D / 16), sb,
                    &ctl->full[st]);
          bulk_load(dst + 2 * C::KB + C::SB + lane * sb, c.vs + pg * c.vs_sp + kvh * c.vs_sh + sl * (D / 16), sb,
                    &ctl->full[st]);
        } else {
#pragma unroll
          for (int pn = 0; pn < D / 64; ++pn) {
            uint8_t* kd = stage + pn * (kTile * 128) + lane * F * 128;
            tma_load_4d(kd, &p.tmK, &ctl->full[st], pn * 64, sl, kvh, pg);
            tma_load_4d(kd + C::KB, &p.tmV, &ctl->full[st], pn * 64, sl, kvh, pg);
          }
        }
      }
    }
  }
  // no copy may still be landing in shared memory when the CTA exits
  if (lane == 0)
    for (int k = max(0, it - C::STAGES); k < it; ++k)
      mbar_wait(&ctl->full[k % C::STAGES], (k / C::STAGES) & 1, p.status, nullptr);
}

// ---------------------------------------------------------------------------------------------
// Consumers. lane = 4 r + t. Matrix rows r, r + 8 are keys (S) or elements (O), columns 2t, 2t + 1
// query heads; accumulator i: (row r + 8 (i / 2), column 2t + i % 2).
// ---------------------------------------------------------------------------------------------

// The key of a 16-key block that S row i stands for. q4: lane t of the V fragments reads rows
// 2t, 2t + 1, 2t + 8, 2t + 9; this order makes the four keys of each such read differ modulo 4
// (different banks, with the row format's exchange of halves), and the two keys of a quarter
// warp's K read odd and even.
template <bool Q4>
__device__ __forceinline__ int key_of(int i) {
  if (!Q4) return i;
  const int j = i & 7;
  return (i & 8) + ((j & 1) ? 4 + ((j >> 1) ^ 1) : j >> 1);
}

// A word of 4 nibbles n (bits 4i, in both halves) as fp16 pairs, by bits alone: a nibble moved to
// bits 2-5 is the subnormal n 2^-22, one at bits 6-9 is n 2^-18 (whose q carry 1/16). What enters
// a product so is n = code + 8; the 8 is taken out by another product, of the constant 8. (At
// bits 0-3 and 4-7 one shift would do for two, but products of numbers that far below the type's
// normal range lose bits in the tensor core: scores were off by 1.5e-6 instead of 4e-7.)
__device__ __forceinline__ void raw_nibbles(uint32_t x, uint32_t& a0, uint32_t& a1, uint32_t& a2, uint32_t& a3) {
  const uint32_t y = x << 2, z = x >> 6;
  a0 = y & 0x003C003Cu;
  a1 = y & 0x03C003C0u;
  a2 = z & 0x003C003Cu;
  a3 = z & 0x03C003C0u;
}

// q4: the power of two that takes the largest |q| of head j to [2^14, 2^15) (or 2^22 over it, what
// turns a product with raw nibbles back into q).
template <int D>
__device__ __forceinline__ float q_scale(const Ctl* ctl, int j, bool up) {
  const float m = D == 128 ? fmaxf(ctl->qmax[j][0], ctl->qmax[j][1]) : ctl->qmax[j][0];
  const uint32_t ex = __float_as_uint(m) >> 23;  // biased; 0: zero or subnormal, 255: not finite
  const uint32_t e = ex == 0 || ex == 255 ? 127u : min(max(ex, 16u), 240u);  // m in [2^(e - 127), 2^(e - 126))
  return __uint_as_float((up ? 127u + 14u + 127u - e : 127u + 22u - 14u + e - 127u) << 23);
}

template <int D, int NT, bool Q4, bool PK>
__device__ __forceinline__ void consume(const PagedDecodeParams& p, uint8_t* smem, Ctl* ctl,
                                        Walk<Cfg<D, NT, Q4, PK>> w) {
  using C = Cfg<D, NT, Q4, PK>;
  constexpr int BPW = C::BPW;
  constexpr int KS = D / 16;       // 16-element steps of a row
  constexpr int G = D / kQ4Group;
  constexpr int MT = D / 16;       // 16-element tiles of O
  constexpr int JS = kConsumers / (D / 2), JN = C::ROWS / JS;  // query heads a thread prepares
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, r = lane / 4, t = lane % 4;
  const uint32_t base = smem_u32(smem);
  // this lane's places in a stage, block 0 of its warp; block u and keys + 8 are constants away
  constexpr int RB = Q4 ? D / 2 : 128;  // bytes of a row (bf16: of a 64-element panel)
  const int ka = key_of<Q4>(r), kb = ka + 8;  // the keys of its S rows r and r + 8
  uint32_t koff, soff = 0, voff, voff1 = 0;
  {
    const uint32_t wrow = warp * (16 * BPW);
    if constexpr (Q4) {
      const int k0 = key_of<true>(2 * t), k1 = key_of<true>(2 * t + 1);  // its V rows 2t, 2t + 1
      koff = (wrow + ka) * RB + (D == 128 ? (t ^ (ka & 2)) * 16 : t * 8);
      soff = 2 * C::KB + (wrow + ka) * (D / 16);
      voff = C::KB + (wrow + k0) * RB + (D == 128 ? (r ^ ((k0 & 2) << 1)) * 8 : r * 4);
      voff1 = C::KB + (wrow + k1) * RB + (D == 128 ? (r ^ ((k1 & 2) << 1)) * 8 : r * 4);
    } else {
      // chunk index c ^ (row & 7): c = 2 (k & 3) + 0 or 1 enters as an exclusive or of 32 (k & 3)
      koff = (wrow + (lane & 15)) * RB + (((lane >> 4) ^ (lane & 7)) * 16);
      voff = C::KB + (wrow + (lane & 7) + ((lane >> 4) << 3)) * RB + ((((lane >> 3) & 1) ^ (lane & 7)) * 16);
    }
  }
  int st = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (; w.live(); w.next()) {
    const int kvh = w.hh / p.chunks, h0 = kvh * p.g + (w.hh % p.chunks) * C::ROWS;
    const int rows = min(C::ROWS, kvh * p.g + p.g - h0);
    // ---- the item's queries, rotated in fp32 and kept as the sum of 16-bit parts: three of bf16,
    // or for q4 two of fp16 after a power of two per head has taken the largest to [2^14, 2^15) ----
    {
      const int i = tid % (D / 2), j0 = tid / (D / 2);
      float x[JN], y[JN];
#pragma unroll
      for (int k = 0; k < JN; ++k) {
        x[k] = y[k] = 0.f;
        if (j0 + k * JS < rows) {
          const __nv_bfloat16* q = p.q + w.b * p.q_sb + (h0 + j0 + k * JS) * p.q_sh + i;
          x[k] = __bfloat162float(q[0]);
          y[k] = __bfloat162float(q[D / 2]);
        }
      }
      if (p.rope) {
        const float4 a = turn_cossin(static_cast<float>(w.s.L - 1), freq_at(p.freqs, i));
        const float cs = a.x + a.y, sn = a.z + a.w;
#pragma unroll
        for (int k = 0; k < JN; ++k) {
          float u, v;
          rot_pair(x[k], y[k], cs, sn, u, v);
          x[k] = u, y[k] = v;
        }
      }
      if constexpr (Q4) {
#pragma unroll
        for (int k = 0; k < JN; ++k) {
          uint32_t m = max(__float_as_uint(fabsf(x[k])), __float_as_uint(fabsf(y[k])));
          m = __reduce_max_sync(0xffffffffu, m);
          if (lane == 0) ctl->qmax[j0 + k * JS][D == 128 ? warp & 1 : 0] = __uint_as_float(m);
        }
        named_bar_sync(1, kConsumers);
      }
#pragma unroll
      for (int k = 0; k < JN; ++k) {
        const int j = j0 + k * JS;
        if constexpr (Q4) {
          // element c of head j goes where the lane that feeds it to the product reads 16 bytes per
          // group: lane 4 (j % 8) + (c % 32) / 8, pairs (e, e + 4) of its 8 elements
          const float f = q_scale<D>(ctl, j, true);
          const float f16 = (i & 1) ? f * 0.0625f : f;  // elements 1 and 3 of 4 meet 16 times their nibble
          const float u = x[k] * f16, v = y[k] * f16;
          const __half a = __float2half_rn(u), b = __float2half_rn(v);
          uint8_t* at = smem + C::OFF_Q + (j / 8) * C::QFRAG + (i / 32) * 512 + ((j & 7) * 4 + (i & 31) / 8) * 16 +
                        (i & 3) * 4 + ((i >> 2) & 1) * 2;
          *reinterpret_cast<__half*>(at) = a;
          *reinterpret_cast<__half*>(at + D / 64 * 512) = b;
          uint8_t* rest = at + (PK ? 4 * 4 * 16 : NT * C::QFRAG);
          *reinterpret_cast<__half*>(rest) = __float2half_rn(u - __half2float(a));
          *reinterpret_cast<__half*>(rest + D / 64 * 512) = __float2half_rn(v - __half2float(b));
        } else {
          uint16_t* hi = reinterpret_cast<uint16_t*>(smem + C::OFF_Q + j * C::QROW);
          uint16_t* lo = reinterpret_cast<uint16_t*>(smem + C::OFF_Q + (C::ROWS + j) * C::QROW);
          const __nv_bfloat16 a = __float2bfloat16_rn(x[k]), b = __float2bfloat16_rn(y[k]);
          hi[i] = __bfloat16_as_ushort(a);
          hi[i + D / 2] = __bfloat16_as_ushort(b);
          const float u = x[k] - __bfloat162float(a), v = y[k] - __bfloat162float(b);
          const __nv_bfloat16 c = __float2bfloat16_rn(u), d = __float2bfloat16_rn(v);
          lo[i] = __bfloat16_as_ushort(c);
          lo[i + D / 2] = __bfloat16_as_ushort(d);
          uint16_t* rest = reinterpret_cast<uint16_t*>(smem + C::OFF_Q + (2 * C::ROWS + j) * C::QROW);
          rest[i] = __bfloat16_as_ushort(__float2bfloat16_rn(u - __bfloat162float(c)));
          rest[i + D / 2] = __bfloat16_as_ushort(__float2bfloat16_rn(v - __bfloat162float(d)));
        }
      }
    }
    named_bar_sync(1, kConsumers);
    // bf16 keeps the fragments in registers; q4, short of those, reads them again for every tile
    uint32_t qf[2][NT][C::QREG ? KS : 1][2];  // [hi, lo]
    if constexpr (C::QREG) {
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t row = base + C::OFF_Q + (part * C::ROWS + nt * 8 + r) * C::QROW;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            qf[part][nt][k][0] = lds32(row + k * 32 + t * 4);
            qf[part][nt][k][1] = lds32(row + k * 32 + t * 4 + 16);
          }
        }
    }
    // q4: raw nibbles are code + 8, so each group's sum starts at minus that of 8 everywhere
    if constexpr (Q4) {
      const uint32_t eight[4] = {0x00200020u, 0x00200020u, 0x02000200u, 0x02000200u};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float x[4];
          const uint4 h = lds128(base + C::OFF_Q + nt * C::QFRAG + g * 512 + lane * 16);
          mma_f16_0(x, eight, h.x, h.y);
          mma_f16(x, eight, h.z, h.w);
          if constexpr (!PK) {
            const uint4 v = lds128(base + C::OFF_Q + (NT + nt) * C::QFRAG + g * 512 + lane * 16);
            mma_f16(x, eight, v.x, v.y);
            mma_f16(x, eight, v.z, v.w);
          }
          if (r == 0) ctl->qsum[nt][g][t] = make_float2(-x[0], -x[1]);
        }
    }
    const uint32_t qrest = base + C::OFF_Q + (2 * C::ROWS + r) * C::QROW + t * 4;
    // Scores stay as the matrix product gives them, S; x = S c2 (log2 units). A bias is added as
    // bias / c2, and a score renews the maximum where S > th.
    float c2[NT][2], th[NT][2], nm[NT][2], l[NT][2] = {};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = nt * 8 + 2 * t + e, head = PK ? j & 3 : j;
        c2[nt][e] = Q4 ? fmaxf(p.scale_log2 * q_scale<D>(ctl, head, false), 1e-44f) : p.scale_log2;
        // (every warp writes the same values, and reads its own)
        if (p.slopes && r == 0) ctl->slope[j] = head < rows ? __fdiv_rn(__ldg(p.slopes + h0 + head) * kLog2e, c2[nt][e]) : 0.f;
        th[nt][e] = kNegInf;
        nm[nt][e] = 0.f;  // minus the maximum (log2 units); 0 while there is none (th is -inf then)
      }
    __syncwarp();
    float o[NT][MT][4] = {};
    // q4: O rows r come out 2^-22 and rows r + 8 2^-18 times what they should be. After the products
    // with 16 keys' n, the same with -8: the sums never carry more than one block's 8 w, whose
    // rounding an element keeps (about 2^-20 of the largest p * |value| in its group).
    const uint32_t minus8[4] = {0x80208020u, 0x82008200u, 0x80208020u, 0x82008200u};
    uint32_t mul[NT][2][Q4 ? G / 2 : 1];  // of this lane's columns, for two groups each as bf16
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int q = 0; q < (Q4 ? G / 2 : 1); ++q) mul[nt][e][q] = kFirstMul * 0x00800080u;

    for (int i = 0; i < w.n; ++i, st = st + 1 == C::STAGES ? 0 : st + 1, phase ^= st == 0) {
      if (ok) ok = mbar_wait(&ctl->full[st], phase, p.status, &ctl->abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) continue;  // unwind through the same barriers as the other warps
      const uint32_t stage = base + st * C::STAGE;
      const int n0 = (w.s.t0 + w.t + i) * C::TILE + warp * (16 * BPW);
      const uint32_t got = ctl->frags[st] >> (warp * (16 * BPW) / p.frag_rows);
      bool loaded[BPW], any = false, edge = n0 < w.s.first || n0 + 16 * BPW > w.s.L;
#pragma unroll
      for (int u = 0; u < BPW; ++u) {
        loaded[u] = (got >> (u && p.frag_rows == 16 ? 1 : 0)) & 1;
        any |= loaded[u] && n0 + 16 * u < w.s.L && n0 + 16 * u + 16 > w.s.first;
        edge |= !loaded[u];
      }
      if (any) {
        // ---- scores: s[u][nt][i], key rows r and r + 8 of block u ----
        float s[BPW][NT][4];
        uint32_t vs[BPW][2][Q4 ? G / 2 : 1];  // q4: steps of V's rows r, r + 8 (two bf16 per word)
        if constexpr (Q4) {
          uint32_t kw[BPW][2][G], ks[BPW][2][G / 2];
#pragma unroll
          for (int u = 0; u < BPW; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t kat = stage + koff + (16 * u + 8 * e) * RB, sat = stage + soff + (16 * u + 8 * e) * (D / 16);
              if constexpr (D == 128) {
                const uint4 x = lds128(kat);
                kw[u][e][0] = __byte_perm(x.x, x.z, 0x5410);
                kw[u][e][1] = __byte_perm(x.x, x.z, 0x7632);
                kw[u][e][2] = __byte_perm(x.y, x.w, 0x5410);
                kw[u][e][3] = __byte_perm(x.y, x.w, 0x7632);
                const uint2 y = lds64(sat);
                ks[u][e][0] = y.x, ks[u][e][1] = y.y;
                const uint2 z = lds64(sat + C::SB);
                vs[u][e][0] = z.x, vs[u][e][1] = z.y;
              } else {
                const uint2 x = lds64(kat);
                kw[u][e][0] = __byte_perm(x.x, x.y, 0x5410);
                kw[u][e][1] = __byte_perm(x.x, x.y, 0x7632);
                ks[u][e][0] = lds32(sat);
                vs[u][e][0] = lds32(sat + C::SB);
              }
            }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            uint4 qh[NT], ql[NT];
            uint2 qs[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              qh[nt] = lds128(base + C::OFF_Q + nt * C::QFRAG + g * 512 + lane * 16);
              if constexpr (!PK) ql[nt] = lds128(base + C::OFF_Q + (NT + nt) * C::QFRAG + g * 512 + lane * 16);
              qs[nt] = lds64(smem_u32(&ctl->qsum[nt][g][t]));
            }
#pragma unroll
            for (int u = 0; u < BPW; ++u) {
              uint32_t a[2][4];
#pragma unroll
              for (int e = 0; e < 2; ++e) raw_nibbles(kw[u][e][g], a[0][e], a[0][2 + e], a[1][e], a[1][2 + e]);
              const float sa = (g & 1) ? bf16hi_to_f32(ks[u][0][g / 2]) : bf16lo_to_f32(ks[u][0][g / 2]);
              const float sb = (g & 1) ? bf16hi_to_f32(ks[u][1][g / 2]) : bf16lo_to_f32(ks[u][1][g / 2]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float x[4];
                mma_f16_c(x, a[0], qh[nt].x, qh[nt].y, __uint_as_float(qs[nt].x), __uint_as_float(qs[nt].y));
                mma_f16(x, a[1], qh[nt].z, qh[nt].w);
                if constexpr (!PK) {
                  mma_f16(x, a[0], ql[nt].x, ql[nt].y);
                  mma_f16(x, a[1], ql[nt].z, ql[nt].w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float f = e < 2 ? sa : sb;
                  s[u][nt][e] = g == 0 ? f * x[e] : fmaf(f, x[e], s[u][nt][e]);
                }
              }
            }
          }
          if constexpr (PK) {  // both parts of q; columns j and j + 4 are the same head from here on
#pragma unroll
            for (int u = 0; u < BPW; ++u)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[u][0][e] += __shfl_xor_sync(0xffffffffu, s[u][0][e], 2);
          }
        } else {
#pragma unroll
          for (int u = 0; u < BPW; ++u) {
            float x[2][NT][4];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint32_t a[4];
              ldsm4(a, stage + (koff ^ ((k & 3) * 32)) + (k / 4) * (C::TILE * 128) + u * 2048);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                  uint32_t b0, b1;
                  if constexpr (C::QREG) {
                    b0 = qf[part][nt][k][0], b1 = qf[part][nt][k][1];
                  } else {
                    const uint32_t row = qrest - (2 - part) * C::ROWS * C::QROW + nt * 8 * C::QROW + k * 32;
                    b0 = lds32(row), b1 = lds32(row + 16);
                  }
                  if (k == 0) mma_bf16_0(x[part][nt], a, b0, b1);
                  else mma_bf16(x[part][nt], a, b0, b1);
                }
              if (p.rope) {  // the last part, zero where q was not rotated
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const uint32_t row = qrest + nt * 8 * C::QROW + k * 32;
                  mma_bf16(x[1][nt], a, lds32(row), lds32(row + 16));
                }
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[u][nt][e] = x[0][nt][e] + x[1][nt][e];
          }
        }
        // ---- bias, mask ----
        if (p.slopes) {
          float slope[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) slope[nt][e] = ctl->slope[nt * 8 + 2 * t + e];
#pragma unroll
          for (int u = 0; u < BPW; ++u) {
            const int n = n0 + 16 * u - (w.s.L - 1);
            const float da = static_cast<float>(n + ka), db = static_cast<float>(n + kb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[u][nt][e] = fmaf(slope[nt][e & 1], e < 2 ? da : db, s[u][nt][e]);
          }
        }
        if (edge) {
#pragma unroll
          for (int u = 0; u < BPW; ++u) {
            const int na = n0 + 16 * u + ka, nb = n0 + 16 * u + kb;
            const bool va = loaded[u] && na >= w.s.first && na < w.s.L, vb = loaded[u] && nb >= w.s.first && nb < w.s.L;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (!(e < 2 ? va : vb)) s[u][nt][e] = kNegInf;
            if constexpr (Q4) {
#pragma unroll
              for (int q = 0; q < G / 2; ++q) {
                if (!va) vs[u][0][q] = 0;
                if (!vb) vs[u][1][q] = 0;
              }
            }
          }
        }
        // ---- running maximum, renewed only where a score passes it by 2^8 ----
        bool up = false;
        float mx[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[nt][e] = fmaxf(s[0][nt][e], s[0][nt][e + 2]);
            if constexpr (BPW == 2) mx[nt][e] = fmaxf(fmaxf(mx[nt][e], s[BPW - 1][nt][e]), s[BPW - 1][nt][e + 2]);
            up |= mx[nt][e] > th[nt][e];
          }
        if constexpr (Q4) {
          constexpr uint32_t kMost = (127 + kStepBits) * 0x00800080u;
          uint32_t most = kMost;
#pragma unroll
          for (int q = 0; q < G / 2; ++q) {
            const uint32_t x = __vmaxu2(__vmaxu2(vs[0][0][q], vs[0][1][q]), __vmaxu2(vs[BPW - 1][0][q], vs[BPW - 1][1][q]));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) most = __vmaxu2(most, mul_bf16x2(x, mul[nt][e][q]));
          }
          up |= most != kMost;
        }
        if (__any_sync(0xffffffffu, up)) {
          float f[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = mx[nt][e];
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
              f[nt][e] = 1.f;
              const float lazy = __fdividef(Q4 ? kLazyQ4 : kLazy, c2[nt][e]);
              if (x > th[nt][e] - lazy) {  // above the present maximum
                const float m = x * c2[nt][e];
                f[nt][e] = th[nt][e] == kNegInf ? 0.f : ex2_approx(-nm[nt][e] - m);
                nm[nt][e] = -m;
                th[nt][e] = x + lazy;
                l[nt][e] *= f[nt][e];
              }
            }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if constexpr (Q4) {
                float p4[2 * BPW];  // the weights of this lane's keys
#pragma unroll
                for (int i = 0; i < 2 * BPW; ++i) p4[i] = ex2_approx(fmaf(s[i / 2][nt][e + 2 * (i & 1)], c2[nt][e], nm[nt][e]));
#pragma unroll
                for (int q = 0; q < G / 2; ++q) {
                  float big[2] = {0.f, 0.f};  // the tile's largest p * step of both groups
#pragma unroll
                  for (int i = 0; i < 2 * BPW; ++i) {
                    big[0] = fmaxf(big[0], p4[i] * bf16lo_to_f32(vs[i / 2][i & 1][q]));
                    big[1] = fmaxf(big[1], p4[i] * bf16hi_to_f32(vs[i / 2][i & 1][q]));
                  }
                  uint32_t two = __byte_perm(__float_as_uint(big[0]), __float_as_uint(big[1]), 0x7632);
#pragma unroll
                  for (int off = 4; off < 32; off <<= 1) two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, off));
                  const uint32_t old = mul[nt][e][q];
                  mul[nt][e][q] = 0;
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    // biased exponents: of mul, and of the largest p * step by the new maximum
                    const uint32_t was = (old >> (16 * h + 7)) & 0xFFu;
                    const float seen = f[nt][e] * __uint_as_float((254u + kWeightBits - was) << 23);
                    const float x = fmaxf(seen, h ? bf16hi_to_f32(two) : bf16lo_to_f32(two));
                    const uint32_t now = 254u + kWeightBits - min(max(__float_as_uint(x) >> 23, 1u + kWeightBits), 254u);
                    mul[nt][e][q] |= now << (16 * h + 7);
                    const int d = min(max(static_cast<int>(now) - static_cast<int>(was), -126), 126);
                    const float by = f[nt][e] * __uint_as_float((127u + d) << 23);
                    const int k = 2 * (2 * q + h);
                    o[nt][k][e] *= by;
                    o[nt][k][e + 2] *= by;
                    o[nt][k + 1][e] *= by;
                    o[nt][k + 1][e + 2] *= by;
                  }
                }
              } else {
#pragma unroll
                for (int k = 0; k < MT; ++k) {
                  o[nt][k][e] *= f[nt][e];
                  o[nt][k][e + 2] *= f[nt][e];
                }
              }
            }
        }
        // ---- weights (ex2.approx: within 2 units of fp32's last place, and 16 or 11 bits are kept) ----
#pragma unroll
        for (int u = 0; u < BPW; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[u][nt][e] = ex2_approx(fmaf(s[u][nt][e], c2[nt][e & 1], nm[nt][e & 1]));
              l[nt][e & 1] += s[u][nt][e];
            }
        // ---- O^T += V^T P^T ----
#pragma unroll
        for (int u = 0; u < BPW; ++u) {
          if constexpr (Q4) {
            uint32_t vw[2][G];  // keys (2t, 2t + 1), (2t + 8, 2t + 9): 4 nibbles of each per group
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t a0 = stage + voff + (16 * u + 8 * e) * RB, a1 = stage + voff1 + (16 * u + 8 * e) * RB;
              if constexpr (D == 128) {
                const uint2 x = lds64(a0), y = lds64(a1);
                vw[e][0] = __byte_perm(x.x, y.x, 0x5410);
                vw[e][1] = __byte_perm(x.x, y.x, 0x7632);
                vw[e][2] = __byte_perm(x.y, y.y, 0x5410);
                vw[e][3] = __byte_perm(x.y, y.y, 0x7632);
              } else {
                const uint32_t x = lds32(a0), y = lds32(a1);
                vw[e][0] = __byte_perm(x, y, 0x5410);
                vw[e][1] = __byte_perm(x, y, 0x7632);
              }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
              uint32_t a[2][4];
#pragma unroll
              for (int e = 0; e < 2; ++e) raw_nibbles(vw[e][g], a[0][2 * e], a[0][2 * e + 1], a[1][2 * e], a[1][2 * e + 1]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float x[4];  // p * step * mul
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t two = mul_bf16x2(vs[u][e / 2][g / 2], mul[nt][e & 1][g / 2]);
                  x[e] = s[u][nt][e] * ((g & 1) ? bf16hi_to_f32(two) : bf16lo_to_f32(two));
                }
                const uint32_t b0 = movm(pack_f16x2(x[0], x[1]));
                const uint32_t b1 = movm(pack_f16x2(x[2], x[3]));
                mma_f16(o[nt][2 * g], a[0], b0, b1);
                mma_f16(o[nt][2 * g + 1], a[1], b0, b1);
                mma_f16(o[nt][2 * g], minus8, b0, b1);
                mma_f16(o[nt][2 * g + 1], minus8, b0, b1);
              }
            }
          } else {
            // p as the sum of two bf16: rounded once, its error would be as large as that of the
            // bf16 output itself
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float a = s[u][nt][2 * e], b = s[u][nt][2 * e + 1];
                const uint32_t x = pack_bf16x2(a, b);
                ph[nt][e] = movm(x);
                pl[nt][e] = movm(pack_bf16x2(a - bf16lo_to_f32(x), b - bf16hi_to_f32(x)));
              }
            uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};  // rows behind the length may hold anything, NaN too
            if (edge) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int n = n0 + 16 * u + 8 * e + 2 * t;
                keep[e] = !loaded[u] ? 0u : (n >= w.s.first && n < w.s.L ? 0xFFFFu : 0u) |
                                            (n + 1 >= w.s.first && n + 1 < w.s.L ? 0xFFFF0000u : 0u);
              }
            }
#pragma unroll
            for (int k = 0; k < MT; ++k) {
              uint32_t a[4];
              ldsm4t(a, stage + (voff ^ ((k & 3) * 32)) + (k / 4) * (C::TILE * 128) + u * 2048);
              if (edge) {
                a[0] &= keep[0], a[1] &= keep[0];
                a[2] &= keep[1], a[3] &= keep[1];
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_bf16(o[nt][k], a, ph[nt][0], ph[nt][1]);
                mma_bf16(o[nt][k], a, pl[nt][0], pl[nt][1]);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->empty[st]);
    }

    // ---- join the warps: weights 2^(m_w - M), then pairwise sums in a fixed order ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
        if (r == 0) {
          ctl->m[warp][nt * 8 + 2 * t + e] = th[nt][e] == kNegInf ? kNegInf : -nm[nt][e];
          ctl->l[warp][nt * 8 + 2 * t + e] = l[nt][e];
        }
      }
    named_bar_sync(1, kConsumers);
    float M[NT][2], total[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = nt * 8 + 2 * t + e;
        float x = ctl->m[0][j];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) x = fmaxf(x, ctl->m[k][j]);
        const float bs = x == kNegInf ? 0.f : x;
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) y += ctl->l[k][j] * ex2_approx(ctl->m[k][j] - bs);
        M[nt][e] = x;
        total[nt][e] = y;
        const float f = th[nt][e] == kNegInf ? 0.f : ex2_approx(-nm[nt][e] - bs);
#pragma unroll
        for (int k = 0; k < MT; ++k) {
          // (mul is a power of two of exponent 1 to 253)
          const float fk = Q4 ? f * __uint_as_float((254u << 23) - (((mul[nt][e][Q4 ? k / 4 : 0] >> (16 * (k / 2 & 1))) & 0xFFFFu) << 16)) : f;
          o[nt][k][e] *= Q4 ? 0x1p22f : 1.f;
          o[nt][k][e + 2] *= Q4 ? 0x1p18f : 1.f;
          o[nt][k][e] *= fk;
          o[nt][k][e + 2] *= fk;
        }
      }
    const uint32_t obuf = base + C::OFF_O + lane * 16;
    auto put = [&](uint32_t at) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < MT; ++k)
          sts128(at + (nt * MT + k) * 512, o[nt][k][0], o[nt][k][1], o[nt][k][2], o[nt][k][3]);
    };
    auto add = [&](uint32_t at) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < MT; ++k) {
          const uint4 x = lds128(at + (nt * MT + k) * 512);
          o[nt][k][0] += __uint_as_float(x.x);
          o[nt][k][1] += __uint_as_float(x.y);
          o[nt][k][2] += __uint_as_float(x.z);
          o[nt][k][3] += __uint_as_float(x.w);
        }
    };
    if (warp >= 2) put(obuf + (warp - 2) * C::OBUF);
    named_bar_sync(1, kConsumers);
    if (warp < 2) add(obuf + warp * C::OBUF);
    if (warp == 1) put(obuf + C::OBUF);
    named_bar_sync(1, kConsumers);
    if (warp == 0) {
      add(obuf + C::OBUF);
      const bool whole = w.whole();
      const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + (w.head ? 0 : 1)) * C::ROWS;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = nt * 8 + 2 * t + e;
          if (j >= rows) continue;
          const float tot = total[nt][e];
          const bool any = !(tot == 0.f);  // a NaN goes to the output
          if (whole) {
            __nv_bfloat16* out = p.out + w.b * p.o_sb + (h0 + j) * p.o_sh;
            const float inv = any ? __fdiv_rn(1.f, tot) : 0.f;
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int d = Q4 ? (k / 2) * 32 + 4 * r + 2 * (k & 1) + u : k * 16 + r + 8 * u;
                out[d] = __float2bfloat16_rn(any ? o[nt][k][e + 2 * u] * inv : 0.f);
              }
            if (p.lse && r == 0)
              p.lse[static_cast<int64_t>(w.b) * p.Hq + h0 + j] = any ? (M[nt][e] + log2f(tot)) * kLn2 : kNegInf;
          } else {
            float* acc = p.part_acc + (part + j) * D;
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int d = Q4 ? (k / 2) * 32 + 4 * r + 2 * (k & 1) + u : k * 16 + r + 8 * u;
                acc[d] = o[nt][k][e + 2 * u];
              }
            if (r == 0) p.part_ml[part + j] = make_float2(M[nt][e], tot);
          }
        }
    }
  }
}

// The rows of this block's share of the sequences that are empty.
template <class C, int D>
__device__ __forceinline__ void empty_rows(const PagedCombineParams& p) {
  for (int e = blockIdx.x; e < p.cache.B; e += gridDim.x) {
    if (span_of<C::TILE>(p, e).nt) continue;
    for (int i = threadIdx.x; i < p.Hq * D; i += blockDim.x)
      p.out[e * p.o_sb + (i / D) * p.o_sh + i % D] = __float2bfloat16_rn(0.f);
    if (p.lse)
      for (int h = threadIdx.x; h < p.Hq; h += blockDim.x) p.lse[static_cast<int64_t>(e) * p.Hq + h] = kNegInf;
  }
}

template <int D, int NT, bool Q4, bool PK>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT, Q4, PK>::CTAS)
    paged_decode_kernel(const __grid_constant__ PagedDecodeParams p) {
  using C = Cfg<D, NT, Q4, PK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::OFF_CTL);
  const int tid = threadIdx.x;
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], kWarps);
    }
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  // Launched as a programmatic dependent: global memory is touched only from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // this CTA's run: thread j sums the units of its share of the sequences
  const int B = p.cache.B, share = (B + kThreads - 1) / kThreads;
  int64_t mine = 0;
  for (int b = tid * share; b < min(B, (tid + 1) * share); ++b) {
    const int L = __ldg(p.lens + b);
    if (blockIdx.x == 0 && (L < 0 || L > p.cache.cap)) atomicOr(p.status, kDevPageRange);
    mine += units_of<C>(p, span_of<C::TILE>(p, b));
  }
  int64_t units;
  int64_t before = block_prefix<kThreads>(mine, ctl->wsum, &units);
  const Deal deal(units * p.items, gridDim.x);
  const int cta = blockIdx.x;
  const int64_t lo = deal.start(cta);
  const int len = cta < deal.runs ? static_cast<int>(deal.start(cta + 1) - lo) : 0;
  if (len > 0 && before * p.items <= lo && lo < (before + mine) * p.items) {
    int b = tid * share;
    for (;; ++b) {
      const int units = units_of<C>(p, span_of<C::TILE>(p, b));
      if (lo < (before + units) * p.items) break;
      before += units;
    }
    ctl->b0 = b;
    ctl->rem0 = static_cast<int>(lo - before * p.items);
  }
  // every CTA is resident by now: the combine kernel may come in and find its own place in the
  // work while this grid runs (what both read was complete before this grid's wait returned)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  if (p.whole) empty_rows<C, D>(p);
  if (len > 0) {
    const Walk<C> w(p, ctl->b0, ctl->rem0, len);
    if (tid >= kConsumers) produce<D, NT, Q4, PK>(p, smem, ctl, w);
    else consume<D, NT, Q4, PK>(p, smem, ctl, w);
  }
}

// Joins the segments of items that more than one CTA walked, and writes the rows of empty
// sequences. There are at most as many such items as items, or as places where runs meet,
// whichever are fewer: block x takes item x, or (by_run) the item that run x + 1 begins within if
// run x has its first tiles. Block y: its query heads p.comb_heads y and on. Little shared memory,
// so that blocks fit beside the decode kernel's.
template <class C, int D>
__global__ void __launch_bounds__(256) paged_combine_kernel(const __grid_constant__ PagedCombineParams p) {
  constexpr int N = 256, KG = N / D;  // threads; groups that share an element's partials
  __shared__ int64_t wsum[N / 32];
  __shared__ int64_t item_before;
  __shared__ int item_b;
  __shared__ float part[KG][D];
  // the stream's next kernel may come in and wait
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid % 32;
  const int B = p.cache.B, share = (B + N - 1) / N;
  const bool by_run = p.comb_by_run;
  const int want_b = by_run ? -1 : static_cast<int>(blockIdx.x) / p.items;
  int64_t mine = 0;
  for (int b = tid * share; b < min(B, (tid + 1) * share); ++b) mine += units_of<C>(p, span_of<C::TILE>(p, b));
  int64_t units;
  int64_t before = block_prefix<N>(mine, wsum, &units);
  const Deal deal(units * p.items, p.ctas);
  const int run = blockIdx.x + 1;
  const int64_t lo = by_run && run < deal.runs ? deal.start(run) : -1;
  if (by_run ? lo >= 0 && before * p.items <= lo && lo < (before + mine) * p.items : tid == want_b / share) {
    int b = tid * share;
    for (;; ++b) {
      const int n = units_of<C>(p, span_of<C::TILE>(p, b));
      if (by_run ? lo < (before + n) * p.items : b == want_b) break;
      before += n;
    }
    item_b = b;
    item_before = before;
  }
  __syncthreads();
  int b = 0, n = 0, i0 = 0, first_slot = 0, h0 = 0, j1 = 0;
  if (!by_run || lo >= 0) {
    b = item_b;
    const int len = units_of<C>(p, span_of<C::TILE>(p, b));
    if (len) {
      const int hh = by_run ? static_cast<int>(div_units(lo - item_before * p.items, len)) : static_cast<int>(blockIdx.x) % p.items;
      const int64_t s = item_before * p.items + static_cast<int64_t>(hh) * len;  // the item's first unit
      i0 = deal.run_of(s + C::ENDS);                                             // runs with tiles of it
      const int i1 = deal.run_of(s + len - 1);
      if (i1 > i0 && (!by_run || i0 == run - 1)) n = i1 - i0 + 1;
      first_slot = deal.start(i0) < s ? 1 : 0;
      const int kvh = hh / p.chunks;
      h0 = kvh * p.g + (hh % p.chunks) * p.head_rows;
      j1 = min(min(static_cast<int>(blockIdx.y + 1) * p.comb_heads, p.head_rows), kvh * p.g + p.g - h0);
    }
  }
  // partial rows, and the order of writes to out and lse against earlier kernels, from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.y == 0) empty_rows<C, D>(p);
  if (n == 0) return;
  auto row_of = [&](int k, int j) { return (static_cast<int64_t>(i0 + k) * 2 + (k == 0 ? first_slot : 0)) * p.head_rows + j; };
  // A warp finds the runs' weights 32 at a time, a run per lane. The groups share the runs of one
  // head, or each take heads of their own.
  const int c = tid % D, group = tid / D;
  const bool share_runs = p.comb_heads == 1;
  const int step = share_runs ? KG : 1, j_step = share_runs ? 1 : KG;
  for (int j = blockIdx.y * p.comb_heads + (share_runs ? 0 : group); j < j1; j += j_step) {
    float mx = kNegInf;
    for (int k = lane; k < n; k += 32) mx = fmaxf(mx, p.part_ml[row_of(k, j)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float base = mx == kNegInf ? 0.f : mx;
    float acc = 0.f, sum = 0.f;
    for (int k0 = 0; k0 < n; k0 += 32) {
      float w = 0.f;
      if (k0 + lane < n) {
        const float2 ml = p.part_ml[row_of(k0 + lane, j)];
        w = ex2_approx(ml.x - base);
        sum += w * ml.y;
      }
      const int kn = min(32, n - k0);
#pragma unroll 8
      for (int k = share_runs ? group : 0; k < kn; k += step)
        acc += __shfl_sync(0xffffffffu, w, k) * p.part_acc[row_of(k0 + k, j) * D + c];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (share_runs) {
      part[group][c] = acc;
      __syncthreads();
      if (group > 0) break;  // one head per block
#pragma unroll
      for (int k = 1; k < KG; ++k) acc += part[k][c];
    }
    const bool any = !(sum == 0.f);  // a NaN goes to the output
    p.out[b * p.o_sb + (h0 + j) * p.o_sh + c] = __float2bfloat16_rn(any ? acc / sum : 0.f);
    if (p.lse && c == 0) p.lse[static_cast<int64_t>(b) * p.Hq + h0 + j] = any ? (mx + log2f(sum)) * kLn2 : kNegInf;
  }
}

// In caches whose sequences cannot be long, which the host knows by the table's width alone (the
// lengths are on the device, and a captured call has to serve all of them), items are not cut, and a call is one launch instead of
// two (eagerly 22 us instead of 25): up to kFewCap keys, or kManyCap where items alone fill a
// quarter of the CTAs. On the GPU, 32 heads on 8, d = 128, bf16, lengths up to the capacity, uncut
// against cut: 16 sequences at 512 10.3 and 11.8 us, at 1024 16.5 and 13.8; 64 at 512 19.1 and
// 22.6, at 1024 37.3 and 31.7; one at 256 7.0 and 7.5, at 512 9.9 and 8.2; 4-bit caches alike.
constexpr int kFewCap = 320, kManyCap = 640;

template <int D, int NT, bool Q4, bool PK>
int cta_count() {
  return std::min(paged_sm_count() * Cfg<D, NT, Q4, PK>::CTAS, kPagedMaxCtas);
}

template <int D, int NT, bool Q4, bool PK>
cudaError_t launch(PagedDecodeParams p, cudaStream_t stream) {
  using C = Cfg<D, NT, Q4, PK>;
  static_assert(smem_bytes<D, NT, Q4, PK>() <= 232448 && (smem_bytes<D, NT, Q4, PK>() + 1024) * C::CTAS <= 233472,
                "shared memory of the resident CTAs");
  static_assert(C::STAGES <= 8, "barriers");
  auto kern = paged_decode_kernel<D, NT, Q4, PK>;
  static std::atomic<uint64_t> ready;  // devices that the kernel's shared memory was allowed on
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit) || dev > 63) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<D, NT, Q4, PK>());
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  p.head_rows = C::ROWS;
  p.chunks = (p.g + C::ROWS - 1) / C::ROWS;
  p.items = p.cache.Hkv * p.chunks;
  const int64_t all_items = (int64_t)p.cache.B * p.items;
  p.ctas = cta_count<D, NT, Q4, PK>();
  p.whole = p.cache.cap <= (4 * all_items >= p.ctas ? kManyCap : kFewCap);
  p.part_acc = static_cast<float*>(p.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_acc + (int64_t)p.ctas * 2 * C::ROWS * D);
  if (p.whole) p.ctas = (int)std::min<int64_t>(p.ctas, all_items);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D, NT, Q4, PK>();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess || p.whole) return e;
  // about two blocks per SM where that many have work
  p.comb_by_run = all_items > p.ctas;
  const int heads = std::min(p.g, C::ROWS);
  p.comb_heads = p.comb_by_run ? std::min(heads, 4) : (int)std::max<int64_t>(1, std::min<int64_t>(heads, all_items * heads / (2 * paged_sm_count())));
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(all_items, p.ctas),
                     (heads + p.comb_heads - 1) / p.comb_heads);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<C, D>, static_cast<const PagedCombineParams&>(p));
}

template <int D, int NT, bool Q4, bool PK>
size_t workspace() {
  return (size_t)cta_count<D, NT, Q4, PK>() * 2 * Cfg<D, NT, Q4, PK>::ROWS * (D * sizeof(float) + sizeof(float2));
}

}  // namespace

int paged_sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Up to 8 query heads per KV head fill one column tile; more take two (16 heads a pass), and
// groups above 16 read the cache once per 16 heads (through L2). (4-bit, 8 x 32k keys, 16 heads on
// each KV head, d = 128: 140 us, as two passes of 8 162.) A last pass of fewer heads costs what a
// full one does (8 x 16k keys, 4 KV heads, 16, 17, 24 and 32 heads on each: 46, 79, 80, 80 us).
// Up to 4 heads, with a 4-bit cache, put
// the two parts of q side by side.
#define AFX_PAGED_DISPATCH(fn, ...)                                                                                    \
  (format == kPagedQ4                                                                                                  \
       ? (d == 128 ? (g <= 4 ? fn<128, 1, true, true>(__VA_ARGS__)                                                     \
                             : g <= 8 ? fn<128, 1, true, false>(__VA_ARGS__) : fn<128, 2, true, false>(__VA_ARGS__))   \
                   : (g <= 4 ? fn<64, 1, true, true>(__VA_ARGS__)                                                      \
                             : g <= 8 ? fn<64, 1, true, false>(__VA_ARGS__) : fn<64, 2, true, false>(__VA_ARGS__)))    \
       : (d == 128 ? (g <= 8 ? fn<128, 1, false, false>(__VA_ARGS__) : fn<128, 2, false, false>(__VA_ARGS__))          \
                   : (g <= 8 ? fn<64, 1, false, false>(__VA_ARGS__) : fn<64, 2, false, false>(__VA_ARGS__))))

size_t paged_decode_workspace(int d, int g, int format) { return AFX_PAGED_DISPATCH(workspace); }

cudaError_t launch_paged_decode(const PagedDecodeParams& p, int d, int format, cudaStream_t stream) {
  const int g = p.g;
  return AFX_PAGED_DISPATCH(launch, p, stream);
}

template <int D, int NT, bool Q4, bool PK>
int tile() {
  return Cfg<D, NT, Q4, PK>::TILE;
}

int paged_frag_rows(int page_size, int d, int g, int format) {
  int a = page_size, b = AFX_PAGED_DISPATCH(tile);
  while (b) {
    const int r = a % b;
    a = b;
    b = r;
  }
  return a;
}

}  // namespace afx
