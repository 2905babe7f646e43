// Attention of a chunk of new tokens over a paged cache for sm_103a.
//
//   O = sum_m p_m v_m,  p = softmax over m in (P - W, P] of  s_m = scale <R_P q, k_m> + slope_h (m - P)
//
// for query row n of sequence b at position P = first[b] + n.
//
// Work. The query heads of a KV head read the same keys, so a row of the products is a (query,
// head of the group) pair, row n g + j: groups of any size fill 128-row tiles. A unit is up to 256
// rows, two tiles, of one (sequence, KV head), and walks the tiles of 128 keys that its rows see.
// The units of the whole batch, ordered by (sequence, KV head, rows), are dealt to the CTAs, one on each SM, in
// equal runs of keys, from lengths read on the device. A unit that a run's end cuts leaves (max,
// sum, acc) of its parts in the workspace, at most two per CTA, and a second kernel joins them in a
// fixed order.
//
// CTA. tcgen05 products: S_s = Q_s K^T of row tile s = 0, 1 in tensor memory, a softmax warpgroup
// for each, one row per thread, which writes its weights as bf16 over S_s, and O_s += P_s V with P_s
// read from tensor memory. The issuing thread goes PV_0(i), S_0(i + 1), PV_1(i), S_1(i + 1): while one
// tile's softmax runs, the other's products do. K and V tiles come through one ring of shared
// memory, TMA boxes of a page's rows (bf16) or codes expanded by two warpgroups (4 bits).
// TMEM (512 columns): S_0 [0, 128), S_1 [128, 256), O_0 [256, 384), O_1 [384, 512); P_s over S_s.
//
// What bounds it. bf16: the chain of scores, softmax and values of a row tile beside the other's
// (4096 tokens over 28672 keys, Hq 32 / Hkv 8, d 128: 1.54 ms, 1339 TFLOP/s, 70% of a library product's rate; with a
// rotated q, whose scores take twice the products, 1024 tokens over 15360 keys take 0.285 instead of
// 0.228 ms). 4 bits: the expansion and, with queries and weights in two parts, twice the products (the
// same tokens: 0.396 ms, tensor pipe 61%, integer pipe 43%).
//
// Keys of a 4-bit cache are s_g c (8 and 3 bits): exact in fp16 under a power of two of the tile's
// largest step, for steps down to 2^-28 of it (and off by at most 2^-36 of it below); q enters as fp16
// under a power of two of its row. A rotated q is two 16-bit parts. Weights are one bf16, beside a
// 4-bit cache, whose values are rounded to bf16, two (an output's error 2.2e-3 instead of 2.8e-3, of
// which its own rounding is 1.7e-3).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "launch.h"
#include "paged.cuh"

namespace afx {

namespace {

constexpr int kTile = kAttendTile;       // keys of a tile
// Keys that a unit's two ends cost: Q's load, O's way out. A compromise: with 128, 256 and 384, 4 x 2048 tokens
// over up to 6144 keys take 536, 524, 519 us; windows of 1024 keys with ALiBi, d = 64, 74, 78, 80; a batch of
// chunks and single tokens 357, 327, 327; over 4-bit caches 4 x 1024 tokens 382, 365, 369, 16 x 8 tokens 155, 136, 136.
constexpr int kEnds = 256;
constexpr float kLazy = 8.0f;            // the running maximum may lag by 2^8

template <int D, bool Q4, bool TWO, int ROWS_>
struct Cfg {
  static constexpr int WARPS = Q4 ? 20 : 12;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int PANELS = D / 64;                            // of 64 elements, 128 bytes a row
  static constexpr int ROWS = ROWS_;                               // of a unit: one row tile or two
  static constexpr uint32_t TILE = kTile * 128 * PANELS;           // bytes of a K, V or Q tile
  static constexpr uint32_t QSLOT = TILE * (TWO ? 2 : 1);
  static constexpr int STAGES = D == 64 ? 6 : Q4 ? (ROWS == 256 && TWO ? 2 : 4) : TWO ? 3 : 5;
  // (K and V are expanded independently: each has stages of its own)
  static_assert(!Q4 || STAGES % 2 == 0, "stages of K and of V");
  // Key tiles whose notes (factors, bad pages) may be in use at once, with tile t the first that a
  // softmax still reads. bf16: the ring's producer is at most STAGES ahead of V(t), which is held until
  // then. 4 bits: K(u) is written once the scores of tile u - STAGES / 2 are complete, and those of
  // tile t + 2 (t + 1, where slots do not alternate) follow t's weights.
  static constexpr int NOTES = Q4 ? STAGES / 2 + 2 : STAGES <= 3 ? 2 : STAGES <= 5 ? 3 : 4;
  // 4 bits: K or V of a tile as the cache has it, codes and then steps
  static constexpr uint32_t CODES = kTile * (D / 2), RAW = CODES + kTile * (D / 16);
  static constexpr int RAWS = !Q4 ? 0 : D == 128 && (TWO || ROWS == 256) ? 3 : 6;
  static constexpr uint32_t OFF_KV = (ROWS / 128) * QSLOT;
  static constexpr uint32_t OFF_RAW = OFF_KV + STAGES * TILE;
  static constexpr uint32_t OFF_CTL = OFF_RAW + RAWS * RAW;
  // registers of the warpgroups: producer, issuer and query loaders; softmax; expanders
  static constexpr uint32_t LOW = Q4 ? 80 : 104, SM = Q4 ? 120 : 200, EXP = 80;
  static_assert(LOW + 2 * SM + (Q4 ? 2 * EXP : 0) <= (WARPS / 4) * (65536 / THREADS / 8 * 8), "registers of the launch");
};

using Pos = PagedAttendPos;

// ---------------------------------------------------------------------------------------------
// Work: starts and counts -> units -> this CTA's run
// ---------------------------------------------------------------------------------------------
struct Chunk {
  int first, count;
  bool bad;
};
__device__ __forceinline__ Chunk chunk_of(const int32_t* firsts, const int32_t* counts, int b, int N, int cap) {
  Chunk c;
  c.first = __ldg(firsts + b);
  c.count = counts ? __ldg(counts + b) : N;
  c.bad = c.count < 0 || c.count > N;
  c.count = min(max(c.count, 0), N);
  if (c.count > 0 && (c.first < 0 || c.first > cap - c.count)) {
    c.bad = true;
    c.count = c.first < 0 ? 0 : max(0, cap - c.first);
  }
  if (c.count == 0) c.first = 0;
  return c;
}
__device__ __forceinline__ Chunk chunk_of(const PagedAttendWork& p, int b) {
  return chunk_of(p.first, p.count, b, p.N, p.cache.cap);
}

__device__ __forceinline__ int units_of(const PagedAttendWork& p, const Chunk& c) {
  return static_cast<int>((static_cast<int64_t>(c.count) * p.g + p.unit - 1) >> p.unit_log2);
}

// What units before unit r of a (sequence, KV head) cost, in 1/g of a key: unit i reads the keys up
// to the position of row (i + 1) unit, of which a window leaves W and what its rows spread over.
__device__ __forceinline__ int64_t cost_before(const PagedAttendWork& p, const Chunk& c, int64_t r) {
  const int64_t base = static_cast<int64_t>(c.first) * p.g + p.unit;
  int64_t k = r, cap = 0;
  if (p.window > 0) {
    cap = (static_cast<int64_t>(p.window) + 1) * p.g + p.unit;
    k = cap > base ? min(r, (cap - base + p.unit - 1) >> p.unit_log2) : 0;
  }
  return base * k + p.unit / 2 * k * (k - 1) + (r - k) * cap + r * kEnds * p.g;
}
// What unit r of n costs: a last one of half the rows less for each key (p.half_cost quarters).
__device__ __forceinline__ int64_t cost_of(const PagedAttendWork& p, const Chunk& c, int r, int n) {
  const int64_t all = cost_before(p, c, r + 1) - cost_before(p, c, r), ends = static_cast<int64_t>(kEnds) * p.g;
  return r == n - 1 && p.unit > 128 && c.count * p.g - (r << p.unit_log2) <= 128 ? ends + (all - ends) / 4 * p.half_cost : all;
}
// All units of a (sequence, KV head).
__device__ __forceinline__ int64_t cost_all(const PagedAttendWork& p, const Chunk& c) {
  const int n = units_of(p, c);
  return n ? cost_before(p, c, n - 1) + cost_of(p, c, n - 1, n) : 0;
}

// row / g for row < 2^30: row (M g - 2^63) < 2^30 g keeps the error of the rounded-up reciprocal M
// below 1 / g.
__device__ __forceinline__ int row_div(const PagedAttendWork& p, int row) {
  return static_cast<int>(__umul64hi(2ull * static_cast<uint32_t>(row), p.div_g));
}

// Keys [lo, hi) that a unit's rows see, their first tile and number of tiles.
struct Span {
  int lo, hi, t0, nt;
};
__device__ __forceinline__ Span span_of(const PagedAttendWork& p, const Chunk& c, int r) {
  const int row0 = r << p.unit_log2, rows = c.count * p.g;
  Span s;
  const int p0 = c.first + row_div(p, row0);
  s.hi = c.first + row_div(p, min(row0 + p.unit, rows) - 1) + 1;
  s.lo = p.window > 0 ? max(0, p0 - p.window + 1) : 0;
  s.t0 = s.lo / kTile;
  s.nt = (s.hi - 1) / kTile - s.t0 + 1;
  return s;
}

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

// Run i of `ctas` starts at start(i) of T.
struct Deal {
  int64_t each, more;
  __device__ Deal(int64_t T, int ctas) : each(T / ctas), more(T - T / ctas * ctas) {}
  __device__ int64_t start(int i) const { return i * each + min(static_cast<int64_t>(i), more); }
};

// The tile at which offset x >= 0 of a unit's cost falls.
__device__ __forceinline__ int tile_at(const PagedAttendWork& p, int64_t x, int64_t cost, int nt) {
  const int64_t ends = static_cast<int64_t>(kEnds) * p.g;
  if (x <= ends) return 0;
  return static_cast<int>((x - ends) * nt / (cost - ends));
}

// Offset x of the work that (sequence b, all KV heads) has -> the unit and tile there.
__device__ __forceinline__ Pos find_in(const PagedAttendWork& p, int b, const Chunk& c, int64_t x) {
  const int n = units_of(p, c);
  const int64_t head = cost_all(p, c);
  Pos f;
  f.b = b;
  f.kvh = static_cast<int>(x / head);
  x -= f.kvh * head;
  int a = 0, z = n - 1;
  while (a < z) {  // the last unit that begins at x or before
    const int m = (a + z + 1) / 2;
    if (cost_before(p, c, m) <= x) a = m;
    else z = m - 1;
  }
  f.r = a;
  const int64_t u = cost_before(p, c, a);
  f.t = tile_at(p, x - u, cost_of(p, c, a, n), span_of(p, c, a).nt);
  return f;
}

// How a segment's tiles go to the two row tiles' accumulators ("slots"): units of up to 128 rows have
// one row tile, whose key tiles alternate between both, joined at the segment's end, so that one's
// softmax runs beside the other's products.
constexpr int kOne = 0, kTwo = 1, kSplit = 2;

// The part of a unit that a run has.
struct Seg {
  int b, kvh, row0, rows;    // first row of the unit, rows of the sequence and KV head
  int first, lo, hi;         // position of query 0; the unit's keys
  int t, n;                  // first tile of the segment, its tiles
  int8_t part;               // -1: the whole unit, else which of the CTA's two partial results it is
  int8_t kind;
};

// Steps through a run's segments; a converged warp calls it. The state and the segment lie in shared
// memory, a copy for each warp, for the softmax has no registers to spare.
struct WalkState {
  Pos at;
  Seg seg;
};
struct Walk {
  const PagedAttendWork& p;
  const Pos& end;
  WalkState* st;
  __device__ Walk(const PagedAttendWork& p_, const Pos& begin, const Pos& end_, WalkState* st_) : p(p_), end(end_), st(st_) {
    if (threadIdx.x % 32 == 0) st->at = begin;
    __syncwarp();
  }
  // The next segment, or null. It stays until the next call.
  __device__ __forceinline__ const Seg* next() {
    __syncwarp();
    if (threadIdx.x % 32 == 0) step();
    __syncwarp();
    return st->seg.n > 0 ? &st->seg : nullptr;
  }

 private:
  __device__ __forceinline__ void step() {
    Seg& s = st->seg;
    Pos at = st->at;
    s.n = 0;
#pragma unroll 1
    while (at.b < p.cache.B) {
      const Chunk c = chunk_of(p, at.b);
      if (c.count == 0) {
        ++at.b;
        continue;
      }
      const Span w = span_of(p, c, at.r);
      const bool stop = at.b == end.b && at.kvh == end.kvh && at.r == end.r;
      const int t1 = stop ? end.t : w.nt;
      s.b = at.b, s.kvh = at.kvh, s.row0 = at.r << p.unit_log2, s.rows = c.count * p.g;
      s.first = c.first, s.lo = w.lo, s.hi = w.hi;
      s.t = w.t0 + at.t, s.n = max(0, t1 - at.t);
      s.part = at.t > 0 ? 0 : t1 < w.nt ? 1 : -1;
      s.kind = min(s.rows - s.row0, p.unit) > 128 ? kTwo : s.n > 1 ? kSplit : kOne;
      at.t = 0;
      if (stop) {
        at.b = p.cache.B;
      } else if (++at.r == units_of(p, c)) {
        at.r = 0;
        if (++at.kvh == p.cache.Hkv) {
          at.kvh = 0;
          ++at.b;
        }
      }
      if (s.n > 0) break;
    }
    st->at = at;
  }
};

template <int NOTES, bool Q4>
struct Ctl {
  uint64_t q_full[2], q_empty[2], kv_full[6], kv_empty[6], s_full[2], p_full[2], o_full[2], last;
  uint64_t joint_full, joint_empty;      // split segments: slot 1's result is complete, is taken
  uint64_t raw_full[Q4 ? 6 : 0], raw_empty[Q4 ? 6 : 0], raw_bad[Q4 ? 6 : 0], most_full[Q4 ? 2 : 0];
  uint64_t bad[NOTES];                   // a byte for each 16 keys: on a page that is none
  float factor[Q4 ? NOTES : 0];          // what the tile's scores are to be multiplied by
  uint32_t most[Q4 ? 2 : 0][4];          // its largest step, by expanding warp
  uint32_t tmem_base;
  int abort_flag;
  Pos end;
  WalkState walk[Q4 ? 20 : 12];
  union {
    struct {
      Pos begin;
      int64_t wsum[20];
    };
    float2 joint[128];                   // slot 1's (max, sum)
  };
};

template <int D, bool Q4, bool TWO, int ROWS_>
constexpr size_t smem_bytes() {
  using C = Cfg<D, Q4, TWO, ROWS_>;
  return 1024 + C::OFF_CTL + sizeof(Ctl<C::NOTES, Q4>);
}

// ---------------------------------------------------------------------------------------------
// Producer of bf16 tiles (one warp)
// ---------------------------------------------------------------------------------------------
template <class C, class T>
__device__ __forceinline__ void produce(const PagedAttendParams& p, uint8_t* smem, T* ctl, Walk w) {
  const int lane = threadIdx.x % 32;
  volatile int* abort_flag = &ctl->abort_flag;
  const PagedDev& cache = p.cache;
  const int frag = p.frag_rows, frags = kTile / frag, panel = lane % C::PANELS;
  const uint32_t ops = frags * C::PANELS;
  int it = 0, tiles = 0;
  bool ok = true;
  // page and slot of a key's fragment; -1: none
  auto lookup = [&](int b, int key, int* slot) {
    return page_at(cache, b, key, slot);
  };
  const Seg* seg;
  while (ok && (seg = w.next())) {
    const Seg& s = *seg;
    for (int i = 0; ok && i < s.n; ++i, ++tiles) {
      const int k0 = (s.t + i) * kTile;
      const int key = k0 + lane / C::PANELS * frag;
      const bool op = lane < ops;
      const bool seen = op && key < s.hi && key + frag > s.lo;
      int slot = 0, page = -1;
      if (seen) page = lookup(s.b, key, &slot);
      const uint32_t none = __ballot_sync(0xffffffffu, seen && page < 0);
      if (none && lane == 0) atomicOr(p.status, kDevPageRange);
      // K: fragments that no row sees stay as they are, their scores are masked
      int st = it % C::STAGES;
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl->kv_empty[st], ((it / C::STAGES) & 1) ^ 1, p.status, abort_flag));
      if (!ok) break;
      const uint32_t loads = __ballot_sync(0xffffffffu, page >= 0);
      if (lane == 0) {
        uint64_t bad = 0;
#pragma unroll 1
        for (uint32_t m = none; m; m &= m - 1) {
          const int f = (__ffs(m) - 1) / C::PANELS;
#pragma unroll 1
          for (int x = 0; x < frag / 16; ++x) bad |= 0xFFull << (8 * (f * (frag / 16) + x));
        }
        ctl->bad[tiles % C::NOTES] = bad;
        mbar_arrive_expect_tx(&ctl->kv_full[st], __popc(loads) * frag * 128);
      }
      __syncwarp();
      uint8_t* dst = smem + C::OFF_KV + st * C::TILE;
      if (page >= 0)
        tma_load_4d(dst + panel * (kTile * 128) + (lane / C::PANELS) * frag * 128, &p.tmK, &ctl->kv_full[st], panel * 64, slot,
                    s.kvh, page);
      ++it;
      // V: what no row sees or has no page is filled with zeros (a box outside the pool)
      st = it % C::STAGES;
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl->kv_empty[st], ((it / C::STAGES) & 1) ^ 1, p.status, abort_flag));
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&ctl->kv_full[st], C::TILE);
      __syncwarp();
      dst = smem + C::OFF_KV + st * C::TILE;
      if (k0 >= s.lo && k0 + kTile <= s.hi) {
        if (op)
          tma_load_4d(dst + panel * (kTile * 128) + (lane / C::PANELS) * frag * 128, &p.tmV, &ctl->kv_full[st], panel * 64, slot,
                      s.kvh, page >= 0 ? page : cache.num_pages);
      } else {
        // 16 keys at a time, one at a time where only some of them are seen
        const int grp = lane / C::PANELS, a = k0 + grp * 16;
        const bool mine = lane < 8 * C::PANELS;
        const int from = max(a, s.lo), to = min(a + 16, s.hi);
        page = -1, slot = 0;
        if (mine && from < to) page = lookup(s.b, a, &slot);
        const bool some = mine && page >= 0 && to - from < 16;
        if (mine && !some)
          tma_load_4d(dst + panel * (kTile * 128) + grp * 2048, &p.tmV16, &ctl->kv_full[st], panel * 64, slot, s.kvh,
                      page >= 0 ? page : cache.num_pages);
#pragma unroll 1
        for (uint32_t m = __ballot_sync(0xffffffffu, some); m; m &= m - 1) {
          const int src = __ffs(m) - 1;
          const int a2 = __shfl_sync(0xffffffffu, a, src), pg = __shfl_sync(0xffffffffu, page, src);
          const int sl = __shfl_sync(0xffffffffu, slot, src);
          if (lane < 16) {
            const int k = a2 + lane;
            tma_load_4d(dst + (src % C::PANELS) * (kTile * 128) + (a2 - k0 + lane) * 128, &p.tmV1, &ctl->kv_full[st],
                        (src % C::PANELS) * 64, sl + lane, s.kvh, k >= s.lo && k < s.hi ? pg : cache.num_pages);
          }
        }
      }
      ++it;
    }
  }
  // no copy may be in flight when the CTA ends
#pragma unroll 1
  for (int i = max(0, it - C::STAGES); i < it; ++i)
    mbar_wait(&ctl->kv_full[i % C::STAGES], (i / C::STAGES) & 1, p.status, nullptr);
}

// ---------------------------------------------------------------------------------------------
// 4-bit tiles: a producer (one warp) copies codes and steps to shared memory, expanders (four warps
// for K, four for V, a thread takes a key) write them to the ring as 16-bit values
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void bulk_load(uint8_t* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <int D, class C, class T>
__device__ __forceinline__ void produce4(const PagedAttendParams& p, uint8_t* smem, T* ctl, Walk w) {
  const int lane = threadIdx.x % 32;
  volatile int* abort_flag = &ctl->abort_flag;
  const PagedDev& cache = p.cache;
  const int frag = p.frag_rows, frags = kTile / frag;
  int it = 0;
  bool ok = true;
  const Seg* seg;
  while (ok && (seg = w.next())) {
    const Seg& s = *seg;
    for (int i = 0; ok && i < s.n; ++i) {
      const int key = (s.t + i) * kTile + lane * frag;
      const bool seen = lane < frags && key < s.hi && key + frag > s.lo;
      int slot = 0, page = -1;
      if (seen) page = page_at(cache, s.b, key, &slot);
      const uint32_t none = __ballot_sync(0xffffffffu, seen && page < 0), loads = __ballot_sync(0xffffffffu, page >= 0);
      if (none && lane == 0) atomicOr(p.status, kDevPageRange);
#pragma unroll 1
      for (int v = 0; v < 2; ++v, ++it) {
        const int st = it % C::RAWS;
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&ctl->raw_empty[st], ((it / C::RAWS) & 1) ^ 1, p.status, abort_flag));
        if (!ok) break;
        if (lane == 0) {
          uint64_t bad = 0;
#pragma unroll 1
          for (uint32_t m = none; m; m &= m - 1)
#pragma unroll 1
            for (int x = 0; x < frag / 16; ++x) bad |= 0xFFull << (8 * ((__ffs(m) - 1) * (frag / 16) + x));
          ctl->raw_bad[st] = bad;
          mbar_arrive_expect_tx(&ctl->raw_full[st], __popc(loads) * frag * (D / 2 + D / 16));
        }
        __syncwarp();
        if (page >= 0) {
          uint8_t* dst = smem + C::OFF_RAW + st * C::RAW;
          const uint8_t* codes = v ? cache.v + page * cache.v_sp + s.kvh * cache.v_sh : cache.k + page * cache.k_sp + s.kvh * cache.k_sh;
          const uint8_t* steps = v ? cache.vs + page * cache.vs_sp + s.kvh * cache.vs_sh : cache.ks + page * cache.ks_sp + s.kvh * cache.ks_sh;
          bulk_load(dst + lane * frag * (D / 2), codes + static_cast<int64_t>(slot) * (D / 2), frag * (D / 2), &ctl->raw_full[st]);
          bulk_load(dst + C::CODES + lane * frag * (D / 16), steps + static_cast<int64_t>(slot) * (D / 16), frag * (D / 16),
                    &ctl->raw_full[st]);
        }
      }
    }
  }
  // no copy may be in flight when the CTA ends
#pragma unroll 1
  for (int i = max(0, it - C::RAWS); i < it; ++i) mbar_wait(&ctl->raw_full[i % C::RAWS], (i / C::RAWS) & 1, p.status, nullptr);
}

// Order of a head's elements in these tiles: of every 64, elements e and 32 + e (e < 32), of two groups,
// lie side by side, as a register of codes has them; sorting them took a fifth of the instructions. The
// query pass writes the same order, and the way out undoes it for the values.

// Four elements of each of two groups, from a word of their codes (the first group's in the low half):
// fp16 (F16) or bf16 pairs, times the groups' steps (a pair).
template <bool F16>
__device__ __forceinline__ uint4 expand8(uint32_t w, uint32_t step2) {
  uint32_t y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t c;
    if constexpr (F16) {
      // 1024 + n, or 1024 + 16 n times 1/16, less what makes it n - 8: all exact
      const uint32_t u = e < 2 ? w : w >> 8;
      if (e & 1) {
        const uint32_t x = (u & 0x00F000F0u) | 0x64006400u;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(c) : "r"(x), "r"(0x2C002C00u), "r"(0xD480D480u));
      } else {
        const uint32_t x = (u & 0x000F000Fu) | 0x64006400u;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(x), "r"(0x64086408u));
      }
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y[e]) : "r"(c), "r"(step2));
    } else {
      const uint32_t x = ((w >> (4 * e)) & 0x000F000Fu) | 0x43004300u;  // 128 + n
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(x), "r"(0x43084308u));
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y[e]) : "r"(c), "r"(step2));
    }
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

// Expands row `row` of a copied tile into a tile of the ring (128-byte swizzle, panels of 64
// elements). With d = 128 rows take their 16-byte pieces in different orders, so that neither the
// loads nor the stores of eight rows meet in a bank (d = 64: the two loads do, in pairs).
template <int D, bool F16>
__device__ __forceinline__ void expand_row(const uint8_t* raw, const uint32_t (&step2)[D / 64], uint8_t* tile, int row) {
  const int turn = D == 128 ? (row & 2) | ((row >> 2) & 1) : 0;
#pragma unroll 1
  for (int j = 0; j < D / 32; ++j) {
    const int at = j ^ turn;
    const uint4 c = *reinterpret_cast<const uint4*>(raw + row * (D / 2) + at * 16);
    auto put = [&](int panel, int chunk, uint32_t w) {
      *reinterpret_cast<uint4*>(tile + panel * (kTile * 128) + sw128_offset(row, chunk)) = expand8<F16>(w, step2[panel]);
    };
    if constexpr (D == 128) {
      // two chunks of four groups; slots (as rows: pages are multiples of 16) with bit 1 have their halves swapped
      const int m = at ^ (row & 2);
      put(0, 2 * m, c.x), put(0, 2 * m + 1, c.z);
      put(1, 2 * m, c.y), put(1, 2 * m + 1, c.w);
    } else {
      // four chunks of two groups
      put(0, 4 * at, c.x), put(0, 4 * at + 1, c.y), put(0, 4 * at + 2, c.z), put(0, 4 * at + 3, c.w);
    }
  }
}

template <int D, bool VALUES, class C, class T>
__device__ __forceinline__ void expand(const PagedAttendParams& p, uint8_t* smem, T* ctl, Walk w) {
  const int row = threadIdx.x % 128, lane = threadIdx.x % 32;
  volatile int* abort_flag = &ctl->abort_flag;
  int tiles = 0;
  bool ok = true;
  const Seg* seg;
  while (ok && (seg = w.next())) {
    const Seg& s = *seg;
    for (int i = 0; i < s.n; ++i, ++tiles) {
      const int key = (s.t + i) * kTile + row, it = 2 * tiles + VALUES;
      const int rs = it % C::RAWS, st = it % C::STAGES;
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl->raw_full[rs], (it / C::RAWS) & 1, p.status, abort_flag) &&
                                       mbar_wait(&ctl->kv_empty[st], ((it / C::STAGES) & 1) ^ 1, p.status, abort_flag));
      if (!ok) break;
      const uint8_t* raw = smem + C::OFF_RAW + rs * C::RAW;
      const uint64_t bad = *reinterpret_cast<volatile uint64_t*>(&ctl->raw_bad[rs]);
      // keys that no row sees, or without a page, are zeros (steps of 0, whatever lies there)
      const bool seen = key >= s.lo && key < s.hi && !((bad >> (8 * (row / 16))) & 1);
      uint32_t step2[D / 64];
#pragma unroll
      for (int g = 0; g < D / 64; ++g)
        step2[g] = seen ? *reinterpret_cast<const uint32_t*>(raw + C::CODES + row * (D / 16) + g * 4) : 0u;
      if constexpr (!VALUES) {
        // steps under a power of two that takes the tile's largest (finite) one to [2^11, 2^12):
        // products of 11 bits at most, exact in fp16's normal range
        uint32_t most = 0;
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
          const uint32_t a = step2[g] & 0x7FFFu, b = (step2[g] >> 16) & 0x7FFFu;
          most = max(most, max(a < 0x7F80u ? a : 0u, b < 0x7F80u ? b : 0u));
        }
        most = __reduce_max_sync(0xffffffffu, most);
        uint32_t(&all)[4] = ctl->most[tiles & 1];
        if (lane == 0) {
          all[row / 32] = most;
          mbar_arrive(&ctl->most_full[tiles & 1]);
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl->most_full[tiles & 1], (tiles >> 1) & 1, p.status, abort_flag));
        if (!ok) break;
        const uint32_t e = max(max(max(all[0], all[1]), max(all[2], all[3])) >> 7, 12u);
        const float up = __uint_as_float((254u + 11u - e) << 23);
        if (row == 0) {
          ctl->factor[tiles % C::NOTES] = __uint_as_float((e - 11u) << 23);
          ctl->bad[tiles % C::NOTES] = bad;
        }
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
          const __half2 h = __floats2half2_rn(bf16lo_to_f32(step2[g]) * up, bf16hi_to_f32(step2[g]) * up);
          step2[g] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      expand_row<D, !VALUES>(raw, step2, smem + C::OFF_KV + st * C::TILE, row);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->kv_full[st]);
        mbar_arrive(&ctl->raw_empty[rs]);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Query loaders (two warps)
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int D, bool TWO, class C, class T>
__device__ __forceinline__ void load_queries(const PagedAttendParams& p, uint8_t* smem, T* ctl, Walk w) {
  constexpr int CH = D / 8;  // 16-byte pieces of a row
  const int tid = threadIdx.x - 64, lane = threadIdx.x % 32;
  const int chunk = tid % CH;
  volatile int* abort_flag = &ctl->abort_flag;
  uint32_t used = 0;  // bit s: phase of q_empty[s]
  bool ok = true;
  const Seg* seg;
  while (ok && (seg = w.next())) {
    const Seg& s = *seg;
#pragma unroll 1
    for (int slot = 0; slot < 2; ++slot) {
      const int r0 = s.row0 + 128 * slot;
      if (slot > 0 && s.kind != kTwo) continue;
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&ctl->q_empty[slot], ((used >> slot) & 1) ^ 1, p.status, abort_flag));
      if (!ok) break;
      used ^= 1u << slot;
      const uint32_t to = smem_u32(smem + slot * C::QSLOT) + (chunk >> 3) * (kTile * 128);
      const __nv_bfloat16* from = p.q + s.b * p.q_sb + static_cast<int64_t>(s.kvh) * p.g * p.q_sh + chunk * 8;
      constexpr int STEP = 64 / CH;
      const int g = p.g, dn = row_div(p, STEP), dj = STEP - dn * g, last = s.rows - r0;  // rows behind the last are not used
      int n = row_div(p, r0 + tid / CH), j = r0 + tid / CH - n * g;
#pragma unroll 2
      for (int r = tid / CH; r < min(128, last); r += STEP) {
        const uint32_t dst = to + sw128_offset(r, chunk & 7);
        const __nv_bfloat16* x = from + n * p.q_sn + j * p.q_sh;
        cp_async16(dst, x);
        if (TWO) cp_async16(dst + C::TILE, x + p.q_lo);
        n += dn, j += dj;
        if (j >= g) j -= g, ++n;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full[slot]);
    }
  }
  // then, while the last products run, padding: rows [count, N) of every head, 64 rows of a head at a time
  constexpr int kPad = 64, LINES = 32 / CH;  // rows that a warp's 16-byte pieces cover
  const int pads = (p.N + kPad - 1) / kPad;
  const int64_t all = static_cast<int64_t>(p.cache.B) * p.Hq * pads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 2 + tid / 32; i < all; i += 2 * p.ctas) {
    const int64_t bh = i / pads;
    const int b = static_cast<int>(bh / p.Hq), h = static_cast<int>(bh - static_cast<int64_t>(b) * p.Hq);
    const int n0 = static_cast<int>(i - bh * pads) * kPad, n1 = min(p.N, n0 + kPad), from = max(n0, chunk_of(p, b).count);
    if (from >= n1) continue;
    int n = from + lane / CH;
    __nv_bfloat16* out = p.out + b * p.o_sb + h * p.o_sh + n * p.o_sn + chunk * 8;
#pragma unroll 1
    for (; n < n1; n += LINES, out += LINES * p.o_sn) __stcs(reinterpret_cast<uint4*>(out), make_uint4(0, 0, 0, 0));
    if (p.lse)
#pragma unroll 1
      for (n = from + lane; n < n1; n += 32) p.lse[bh * p.N + n] = kNegInf;
  }
}

// ---------------------------------------------------------------------------------------------
// Issuer of the products: a converged warp, of which one thread is elected for a tile's products.
// Their bases are made the warp's own by a shuffle: values of one thread alone, or an election for
// each product, take the compiler ten times the instructions to bring to the uniform registers that
// the products want (one thread took 100 cycles for a product of 64; and instruction fetches bound
// the 4-bit kernel: 8 tokens over each of 16 contexts 0.176 ms with elections for each, 0.147 so; later
// steps brought that to 0.137).
// ---------------------------------------------------------------------------------------------
template <int D, bool Q4, bool TWO, class C, class T>
__device__ __forceinline__ void issue(const PagedAttendParams& p, uint8_t* smem, T* ctl, Walk w, uint32_t tmem) {
  constexpr uint32_t idesc_s = idesc_f32acc(128, 128, 0, 0, Q4), idesc_o = idesc_f32acc(128, D, 0, 1);
  volatile int* abort_flag = &ctl->abort_flag;
  int* status = p.status;
  // descriptors as a low word, to which a product's place in the tile adds a constant, and one high word
  static_assert(sizeof(T) + C::OFF_CTL + 1024 < (1u << 18), "descriptor address field");
  constexpr uint32_t dhi = desc_sw128_hi(1024);
  const uint32_t dQ = desc_sw128_lo(smem_u32(smem), 16), dK = desc_sw128_lo(smem_u32(smem + C::OFF_KV), 16);
  const uint32_t dV = desc_sw128_lo(smem_u32(smem + C::OFF_KV), kTile * 128);
  uint32_t phases = 0;  // bit s: of q_full[s], bit 2 + s: of p_full[s]
  bool ok = true;
  auto wait = [&](uint64_t* bar, int parity) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, status, abort_flag));
  };
  auto wait_tile = [&](int it) { wait(&ctl->kv_full[it % C::STAGES], (it / C::STAGES) & 1); };
  auto ready = [&](int it) {
    return __all_sync(0xffffffffu, mbar_test(&ctl->kv_full[it % C::STAGES], (it / C::STAGES) & 1)) != 0;
  };
  auto base = [&](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
  // S of slot s from row tile `qs`
  auto scores = [&](int s, int qs, int it, bool first, bool last) {
    if (first) {
      wait(&ctl->q_full[qs], (phases >> qs) & 1);
      phases ^= 1u << qs;
    }
    if (!ok) return;
    tc_fence_after();
    const uint32_t q = base(dQ + qs * (C::QSLOT >> 4)), k = base(dK + (it % C::STAGES) * (C::TILE >> 4)), d = base(tmem + 128 * s);
    if (elect_one()) {
      mma_ss_w<0>(d, q, k, dhi, idesc_s);
#pragma unroll
      for (int kk = 1; kk < (TWO ? 2 : 1) * (D / 16); ++kk) {
        const uint32_t off = ((kk % (D / 16)) >> 2) * (kTile * 128) + (kk & 3) * 32;
        mma_ss_w<1>(d, q + (((kk / (D / 16)) * C::TILE + off) >> 4), k + (off >> 4), dhi, idesc_s);
      }
    }
    __syncwarp();
    mma_commit_warp(&ctl->s_full[s]);
    if (last) mma_commit_warp(&ctl->q_empty[qs]);
  };
  auto values = [&](int s, int it, bool first, bool last) {
    wait(&ctl->p_full[s], (phases >> (2 + s)) & 1);
    phases ^= 4u << s;
    if (!ok) return;
    tc_fence_after();
    const uint32_t v = base(dV + (it % C::STAGES) * (C::TILE >> 4)), w = base(tmem + 128 * s), o = w + 256;
    if (elect_one()) {
      if (first) mma_ts_w<0>(o, w, v, dhi, idesc_o);
      else mma_ts_w<1>(o, w, v, dhi, idesc_o);
      // 4 bits: of every 32 columns, 16 of weights and 16 of what their rounding left
      if constexpr (Q4) mma_ts_w<1>(o, w + 16, v, dhi, idesc_o);
#pragma unroll
      for (int kk = 1; kk < 8; ++kk) {
        const uint32_t at = w + (Q4 ? kk / 2 * 32 + kk % 2 * 8 : kk * 8);
        mma_ts_w<1>(o, at, v + kk * (2048 >> 4), dhi, idesc_o);
        if constexpr (Q4) mma_ts_w<1>(o, at + 16, v + kk * (2048 >> 4), dhi, idesc_o);
      }
    }
    __syncwarp();
    if (last) mma_commit_warp(&ctl->o_full[s]);
  };
  // the next segment's tiles and kind (as votes, so that branches on them are known to be the warp's)
  int nn = 0;
  bool have = false, two = false, split = false;
  auto next = [&]() {
    const Seg* s = w.next();
    nn = __shfl_sync(0xffffffffu, s ? s->n : 0, 0);
    have = __any_sync(0xffffffffu, s != nullptr);
    two = __any_sync(0xffffffffu, s && s->kind == kTwo);
    split = __any_sync(0xffffffffu, s && s->kind == kSplit);
  };
  next();
  int vt = -1;  // ring index of the V before the next K
  while (ok && have) {
    if (split) {
      // the next tile's scores, in the other slot, go before a tile's values, unless its K is late
      int kt = vt + 1;
      wait_tile(kt);
      scores(0, 0, kt, true, false);
      if (ok) mma_commit_warp(&ctl->kv_empty[kt % C::STAGES]);
#pragma unroll 1
      for (int i = 0; i < nn && ok; ++i, kt += 2) {
        const bool more = i + 1 < nn;
        const bool late = more && !ready(kt + 2) && ready(kt + 1) &&
                          __all_sync(0xffffffffu, mbar_test(&ctl->p_full[i & 1], (phases >> (2 + (i & 1))) & 1));
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          if ((x == 0) == late || !more) {
            if (!more && x == 0) continue;
            wait_tile(kt + 1);
            values(i & 1, kt + 1, i < 2, i >= nn - 2);
            if (ok) mma_commit_warp(&ctl->kv_empty[(kt + 1) % C::STAGES]);
          } else {
            wait_tile(kt + 2);
            scores(~i & 1, 0, kt + 2, false, i + 2 == nn);
            if (ok) mma_commit_warp(&ctl->kv_empty[(kt + 2) % C::STAGES]);
          }
        }
      }
      vt += 2 * nn;
      next();
      continue;
    }
    // a step: the values' products of a tile and the scores' of the next one, row tile by row tile
    int cn = 0, ci = 0, ni = 0;  // tiles of the segment, the tiles' numbers
    bool act1 = false, cur = false;
    while (ok && (cur || (have && !split))) {
      const bool more = have && !split, first = ci == 0, last = ci == cn - 1, nfirst = ni == 0, nlast = ni == nn - 1;
      const int kt = vt + 1;
      if (cur) wait_tile(vt);
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {
        if (cur && (s == 0 || act1)) values(s, vt, first, last);
        if (cur && s == act1 && ok) mma_commit_warp(&ctl->kv_empty[vt % C::STAGES]);
        if (more && s == 0) wait_tile(kt);
        if (more && (s == 0 || two)) scores(s, s, kt, nfirst, nlast);
      }
      if (more && ok) mma_commit_warp(&ctl->kv_empty[kt % C::STAGES]);
      cur = more, cn = nn, ci = ni, act1 = two;
      if (more) {
        vt += 2;
        if (++ni == nn) {
          next();
          ni = 0;
        }
      }
    }
  }
  // all products have ended before tensor memory is given back
  mma_commit_warp(&ctl->last);
  mbar_wait(&ctl->last, 0, status, nullptr);
}

// ---------------------------------------------------------------------------------------------
// Softmax of row tile s (four warps, one row per thread)
// ---------------------------------------------------------------------------------------------
template <int D, bool Q4, class C, class T>
__device__ __forceinline__ void softmax(const PagedAttendParams& p, T* ctl, Walk w, uint32_t tmem, int slot) {
  constexpr int CW = 32;  // columns of the scores that a thread takes at once
  const int lane = threadIdx.x % 32, quarter = (threadIdx.x / 32) % 4, r = quarter * 32 + lane;
  volatile int* abort_flag = &ctl->abort_flag;
  int* status = p.status;
  const uint32_t tS = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 128 * slot, tO = tS + 256;
  int sc = 0, oc = 0, jc = 0, tiles = 0;
  bool ok = true;
  const Seg* seg;
  while (ok && (seg = w.next())) {
    const Seg& s = *seg;
    const bool split = s.kind == kSplit;
    if (slot == 1 && s.kind == kOne) {
      tiles += s.n;
      continue;
    }
    const int row = s.row0 + (split ? 0 : 128 * slot) + r;
    const bool live = row < s.rows;
    const int n = row_div(p, min(row, s.rows - 1));
    const int h = s.kvh * p.g + (min(row, s.rows - 1) - n * p.g);
    const int pos = live ? s.first + n : INT_MAX;  // a row behind the last needs no mask
    const bool some = __any_sync(0xffffffffu, live);
    const int lo = p.window > 0 && live ? max(0, pos - p.window + 1) : 0;
    float mul = p.scale_log2;
    if (Q4) mul *= __ldg(p.factor + (static_cast<int64_t>(s.b) * p.Hq + h) * p.N + n);
    const float slope = p.slopes ? __ldg(p.slopes + h) * kLog2e : 0.f;
    float m_run = kNegInf, l_run = 0.f;
    for (int i = split ? slot : 0; i < s.n; i += split ? 2 : 1) {
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl->s_full[slot], sc & 1, status, abort_flag));
      if (!ok) break;
      ++sc;
      if (!some) {  // none of the warp's rows is one: the weights stay as they are
        if (lane == 0) mbar_arrive(&ctl->p_full[slot]);
        continue;
      }
      tc_fence_after();
      const uint64_t bad = *reinterpret_cast<volatile uint64_t*>(&ctl->bad[(tiles + i) % C::NOTES]);
      float part = 1.f;  // of the scores: a power of two
      if constexpr (Q4) part = *reinterpret_cast<volatile float*>(&ctl->factor[(tiles + i) % C::NOTES]);
      const int k0 = (s.t + i) * kTile;
      // 4 bits: not 0, which times a masked column's -inf would be NaN (a row of zeros has a factor of
      // 2^-100, a tile of zeros one of 2^-126). Scores as they come are below 2^15 * 2^15 * 128 = 2^37, so
      // that at 2^-126 they move no weight. (bf16: the scale alone, which may be below 2^-126 in earnest.)
      const float unit = p.slopes ? 1.f : Q4 ? fmaxf(mul * part, 0x1p-126f) : mul;
      const bool masked = __any_sync(0xffffffffu, k0 + kTile - 1 > pos || k0 < lo || bad != 0);
      // Passes over the tile read its scores from tensor memory, CW columns at a time, in loops: all 128
      // at once, unrolled, take registers and instruction cache that the warps of five roles do not have.
      auto scores = [&](int ch, float (&x)[CW]) {
        uint32_t xr[CW];
        tmem_ld32(tS + CW * ch, xr);
        tmem_wait_ld_dep(xr);
#pragma unroll
        for (int c = 0; c < CW; ++c) x[c] = __uint_as_float(xr[c]);
      };
      if (p.slopes || masked) {
        // a pass of its own writes them back with the bias and the mask
#pragma unroll 1
        for (int ch = 0; ch < kTile / CW; ++ch) {
          float x[CW];
          scores(ch, x);
          if (p.slopes) {
            const float from = slope * static_cast<float>(k0 + CW * ch - pos), f = mul * part;
#pragma unroll
            for (int c = 0; c < CW; c += 2) {
              const uint64_t y = fma2(f2_pack(slope, slope), f2_pack(c, c + 1),
                                      fma2(f2_pack(x[c], x[c + 1]), f2_pack(f, f), f2_pack(from, from)));
              x[c] = f2_lo(y), x[c + 1] = f2_hi(y);
            }
          }
          if (masked) {
            // a bit for each column that the row sees
            const uint32_t gone = static_cast<uint32_t>(bad >> (CW / 2 * ch));
            const int at = k0 + CW * ch, c0 = min(max(lo - at, 0), 32), c1 = min(max(pos - at, -1), 31) + 1;
            uint32_t see = static_cast<uint32_t>(((1ull << c1) - 1) & ~((1ull << c0) - 1));
            if (gone & 1) see &= 0xFFFF0000u;
            if (gone & 0x100) see &= 0x0000FFFFu;
#pragma unroll
            for (int c = 0; c < CW; ++c) x[c] = (see >> c) & 1 ? x[c] : kNegInf;
          }
          uint32_t y[CW];
#pragma unroll
          for (int c = 0; c < CW; ++c) y[c] = __float_as_uint(x[c]);
          tmem_st32(tS + CW * ch, y);
        }
        tmem_wait_st();
      }
      float mx = kNegInf;
#pragma unroll 1
      for (int ch = 0; ch < kTile / CW; ++ch) {
        float x[CW], m[CW / 8];
        scores(ch, x);
#pragma unroll
        for (int k = 0; k < CW / 8; ++k) m[k] = fmaxf(x[2 * k], x[2 * k + 1]);
#pragma unroll
        for (int j = 1; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < CW / 8; ++k) m[k] = max3f(m[k], x[CW / 4 * j + 2 * k], x[CW / 4 * j + 2 * k + 1]);
#pragma unroll
        for (int k = 0; k < CW / 8; k += 2) mx = max3f(mx, m[k], m[k + 1]);
      }
      mx *= unit;
      // O keeps its scale unless this tile exceeds it by more than 2^kLazy
      const float m_new = mx > m_run + kLazy ? mx : m_run;
      const bool grow = m_new > m_run && m_run != kNegInf && live;
      if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
        // (the products of the tile before are complete: S of this one was issued behind them)
        const float alpha = grow ? ex2_approx(m_run - m_new) : 1.f;
        l_run *= alpha;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          tmem_ld32(tO + ch * 32, o);
          tmem_wait_ld_dep(o);
#pragma unroll
          for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
          tmem_st32(tO + ch * 32, o);
        }
      }
      m_run = m_new;
      const float nb = m_new == kNegInf ? 0.f : -m_new;
      const uint64_t u2 = f2_pack(unit, unit), nb2 = f2_pack(nb, nb);
      uint64_t acc[2] = {0, 0};
#pragma unroll 1
      for (int ch = 0; ch < kTile / CW; ++ch) {
        float x[CW];
        scores(ch, x);
        uint32_t pk[CW / 2], rest[Q4 ? CW / 2 : 1] = {};
#pragma unroll
        for (int c = 0; c < CW / 2; ++c) {
          const uint64_t a = fma2(f2_pack(x[2 * c], x[2 * c + 1]), u2, nb2);
          const uint64_t w = f2_pack(ex2_approx(f2_lo(a)), ex2_approx(f2_hi(a)));
          acc[c & 1] = add2(acc[c & 1], w);
          pk[c] = pack_bf16x2(f2_lo(w), f2_hi(w));
          if constexpr (Q4) {
            const uint64_t r = add2(w, bf16x2_to_f2(pk[c] ^ 0x80008000u));
            rest[c] = pack_bf16x2(f2_lo(r), f2_hi(r));
          }
        }
        // over scores that are weighed already
        if constexpr (Q4) {
          tmem_st16(tS + CW * ch, pk);
          tmem_st16(tS + CW * ch + CW / 2, rest);
        } else {
          tmem_st16(tS + CW / 2 * ch, pk);
        }
      }
      const uint64_t both = add2(acc[0], acc[1]);
      l_run += f2_lo(both) + f2_hi(both);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_full[slot]);
    }
    tiles += s.n;
    if (!ok) break;
    ok = __all_sync(0xffffffffu, mbar_wait(&ctl->o_full[slot], oc & 1, status, abort_flag));
    if (!ok) break;
    ++oc;
    tc_fence_after();
    float w0 = 1.f, w1 = 0.f;  // the slots' weights
    if (split) {
      if (slot == 1) {
        // O_1 stays as it is until slot 0 has taken it
        ctl->joint[r] = make_float2(m_run, l_run);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->joint_full);
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl->joint_empty, jc & 1, status, abort_flag));
        ++jc;
        continue;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl->joint_full, jc & 1, status, abort_flag));
      if (!ok) break;
      ++jc;
      tc_fence_after();
      const float2 ml = ctl->joint[r];
      const float m = fmaxf(m_run, ml.x), base = m == kNegInf ? 0.f : m;
      w0 = ex2_approx(m_run - base), w1 = ex2_approx(ml.x - base);
      l_run = w0 * l_run + w1 * ml.y;
      m_run = m;
    }
    // Columns 32 ch .. of the row's accumulator: two runs of 16 elements, the k-th from place_of(ch, k) on.
    auto result = [&](int ch, uint32_t (&y)[32]) {
      uint32_t o[32];
      tmem_ld32(tO + ch * 32, o);
      tmem_wait_ld_dep(o);
      if (split) {
        uint32_t o1[32];
        tmem_ld32(tO + 128 + ch * 32, o1);
        tmem_wait_ld_dep(o1);
#pragma unroll
        for (int q = 0; q < 32; ++q)
          o[q] = __float_as_uint(__fmaf_rn(__uint_as_float(o1[q]), w1, __uint_as_float(o[q]) * w0));
      }
#pragma unroll
      for (int q = 0; q < 32; ++q) y[q] = o[Q4 ? 2 * (q % 16) + q / 16 : q];
    };
    auto place_of = [](int ch, int k) { return Q4 ? 64 * (ch >> 1) + 32 * k + 16 * (ch & 1) : 32 * ch + 16 * k; };
    const bool any = !(l_run == 0.f);  // a NaN goes to the output
    if (s.part < 0) {
      const float inv = any ? 1.f / l_run : 0.f;
      __nv_bfloat16* out = p.out + s.b * p.o_sb + h * p.o_sh + n * p.o_sn;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t o[32];
        result(ch, o);
        if (live) {
#pragma unroll
          for (int v4 = 0; v4 < 4; ++v4) {
            uint4* dst = reinterpret_cast<uint4*>(out + place_of(ch, v4 / 2) + v4 % 2 * 8);
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int q = v4 * 8 + 2 * e;
              y[e] = any ? pack_bf16x2(__uint_as_float(o[q]) * inv, __uint_as_float(o[q + 1]) * inv) : 0u;
            }
            __stcs(dst, make_uint4(y[0], y[1], y[2], y[3]));
          }
        }
      }
      if (p.lse && live)
        p.lse[(static_cast<int64_t>(s.b) * p.Hq + h) * p.N + n] = any ? (m_run + log2f(l_run)) * kLn2 : kNegInf;
    } else {
      const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + s.part) * p.unit + 128 * slot + r;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t o[32];
        result(ch, o);
        if (live) {
#pragma unroll
          for (int v4 = 0; v4 < 8; ++v4)
            *reinterpret_cast<uint4*>(p.part_acc + at * D + place_of(ch, v4 / 4) + v4 % 4 * 4) =
                make_uint4(o[4 * v4], o[4 * v4 + 1], o[4 * v4 + 2], o[4 * v4 + 3]);
        }
      }
      if (live) p.part_ml[at] = make_float2(m_run, l_run);
    }
    if (split) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->joint_empty);
    }
  }
}

template <int D, bool Q4, bool TWO, int ROWS_>
__global__ void __launch_bounds__(Cfg<D, Q4, TWO, ROWS_>::THREADS, 1) attend_kernel(const __grid_constant__ PagedAttendParams p) {
  using C = Cfg<D, Q4, TWO, ROWS_>;
  using T = Ctl<C::NOTES, Q4>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  T* ctl = reinterpret_cast<T*>(smem + C::OFF_CTL);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 2);
      mbar_init(&ctl->q_empty[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], 4);
      mbar_init(&ctl->o_full[i], 1);
    }
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&ctl->kv_full[i], Q4 ? 4 : 1);
      mbar_init(&ctl->kv_empty[i], 1);
    }
    for (int i = 0; i < C::RAWS; ++i) {
      mbar_init(&ctl->raw_full[i], 1);
      mbar_init(&ctl->raw_empty[i], 4);
    }
    if constexpr (Q4) {
      mbar_init(&ctl->most_full[0], 4);
      mbar_init(&ctl->most_full[1], 4);
    }
    mbar_init(&ctl->joint_full, 4);
    mbar_init(&ctl->joint_empty, 4);
    mbar_init(&ctl->last, 1);
    ctl->abort_flag = 0;
    ctl->begin = ctl->end = Pos{p.cache.B, 0, 0, 0};
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  // Launched as a programmatic dependent: global memory is touched only from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // thread j sums the work of its share of the sequences
  const int B = p.cache.B, share = (B + C::THREADS - 1) / C::THREADS;
  int64_t mine = 0;
#pragma unroll 1
  for (int b = tid * share; b < min(B, (tid + 1) * share); ++b) {
    const Chunk c = chunk_of(p, b);
    if (blockIdx.x == 0 && c.bad) atomicOr(p.status, kDevPageRange);
    mine += cost_all(p, c) * p.cache.Hkv;
  }
  int64_t total;
  const int64_t before = block_prefix<C::THREADS>(mine, ctl->wsum, &total);
  const Deal deal(total, p.ctas);
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const int64_t x = deal.start(blockIdx.x + e);
    if (mine > 0 && x >= before && x < before + mine) {
      int64_t y = x - before;
#pragma unroll 1
      for (int b = tid * share;; ++b) {
        const Chunk c = chunk_of(p, b);
        const int64_t all = cost_all(p, c) * p.cache.Hkv;
        if (y < all) {
          (e ? ctl->end : ctl->begin) = find_in(p, b, c, y);
          break;
        }
        y -= all;
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  if (tid == 0) p.bounds[blockIdx.x] = ctl->begin;
  Walk w(p, ctl->begin, ctl->end, &ctl->walk[warp]);
  __syncthreads();  // (the begin's place is used for other things from here on)
  if (warp < 4) {
    setmaxnreg_dec<C::LOW>();
    if (warp == 0) {
      if constexpr (Q4) produce4<D, C>(p, smem, ctl, w);
      else produce<C>(p, smem, ctl, w);
    } else if (warp == 1) {
      issue<D, Q4, TWO, C>(p, smem, ctl, w, tmem);
    } else {
      load_queries<D, TWO, C>(p, smem, ctl, w);
    }
  } else if (warp < 12) {
    setmaxnreg_inc<C::SM>();
    softmax<D, Q4, C>(p, ctl, w, tmem, (warp - 4) / 4);
  } else if constexpr (Q4) {
    setmaxnreg_dec<C::EXP>();
    if (warp < 16) expand<D, false, C>(p, smem, ctl, w);
    else expand<D, true, C>(p, smem, ctl, w);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------------------------
// Joining cut units
// ---------------------------------------------------------------------------------------------
// Block (x, y): if run x + 1 begins within a unit whose first tiles run x has, rows 32 y .. of that unit.
constexpr int kJoinRows = 32;

template <int D>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ PagedAttendWork p) {
  __shared__ int16_t order[kPagedMaxCtas];
  __shared__ int order_n;
  const int tid = threadIdx.x, run = blockIdx.x + 1;
  // the stream's next kernel may come in and wait
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // partial rows, the runs' bounds, and the order of writes to out and lse against earlier kernels
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Pos f = run < p.ctas ? p.bounds[run] : Pos{p.cache.B, 0, 0, 0};
  auto within = [&](const Pos& q) { return q.b == f.b && q.kvh == f.kvh && q.r == f.r && q.t > 0; };
  if (f.b >= p.cache.B || f.t == 0 || within(p.bounds[run - 1])) return;
  // Partial results of the unit, in the order of its tiles: run - 1's last segment, then the first ones
  // of the runs that begin within it. (A run of less than a tile has none.)
  for (int k = run + tid; k < p.ctas; k += 256) {
    const Pos q = p.bounds[k];
    const Pos z = k + 1 < p.ctas ? p.bounds[k + 1] : Pos{p.cache.B, 0, 0, 0};
    order[k - run] = !within(q) ? -1 : !within(z) || z.t > q.t ? 1 : 0;
  }
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    for (int k = 0; k < p.ctas - run && order[k] >= 0; ++k)
      if (order[k]) order[n++] = static_cast<int16_t>(k + 1);
    order_n = n;
  }
  __syncthreads();
  const int parts = order_n + 1;
  const Chunk c = chunk_of(p, f.b);
  constexpr int L = D / 4;  // threads of a row
  const int col = tid % L * 4;
  for (int i = tid / L; i < kJoinRows; i += 256 / L) {
    const int r = blockIdx.y * kJoinRows + i, row = (f.r << p.unit_log2) + r;
    if (r >= p.unit || row >= c.count * p.g) break;
    auto at = [&](int i) {
      const int k = i == 0 ? 0 : order[i - 1];
      return (static_cast<int64_t>(run - 1 + k) * 2 + (k == 0 ? 1 : 0)) * p.unit + r;
    };
    float mx = kNegInf;
    for (int k = 0; k < parts; ++k) mx = fmaxf(mx, p.part_ml[at(k)].x);
    const float base = mx == kNegInf ? 0.f : mx;
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < parts; ++k) {
      const float2 ml = p.part_ml[at(k)];
      const float4 o = *reinterpret_cast<const float4*>(p.part_acc + at(k) * D + col);
      const float wgt = ex2_approx(ml.x - base);
      sum += wgt * ml.y;
      acc.x += wgt * o.x, acc.y += wgt * o.y, acc.z += wgt * o.z, acc.w += wgt * o.w;
    }
    const bool any = !(sum == 0.f);
    const float inv = any ? 1.f / sum : 0.f;
    const int n = row_div(p, row), h = f.kvh * p.g + (row - n * p.g);
    *reinterpret_cast<uint2*>(p.out + f.b * p.o_sb + h * p.o_sh + n * p.o_sn + col) =
        any ? make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv)) : make_uint2(0, 0);
    if (p.lse && col == 0) p.lse[(static_cast<int64_t>(f.b) * p.Hq + h) * p.N + n] = any ? (mx + log2f(sum)) * kLn2 : kNegInf;
  }
}

// ---------------------------------------------------------------------------------------------
// Query operands: rotated rows in two parts; for 4-bit caches in fp16 under a power of two
// ---------------------------------------------------------------------------------------------
constexpr int kQueryThreads = 128;

template <int D, bool Q4, bool ROPE>
__global__ void __launch_bounds__(kQueryThreads) attend_query_kernel(const __grid_constant__ PagedQueryParams p) {
  constexpr int CP = D / 16, H2 = D / 2;
  extern __shared__ float4 ang[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) << p.rb_log2;
  const int t = threadIdx.x % CP, k = threadIdx.x / CP, rr = k & ((1 << p.rb_log2) - 1);
  const int step = (kQueryThreads / CP) >> p.rb_log2;
  auto where = [&](int64_t row, int* n) {
    const int b = static_cast<int>(p.div_n ? __umul64hi(static_cast<uint64_t>(row), p.div_n) : row);
    *n = static_cast<int>(row - static_cast<int64_t>(b) * p.N);
    return b;
  };
  const int64_t row = row0 + rr;
  int n = 0, b = 0;
  bool live = row < p.rows;
  if (live) {
    b = where(row, &n);
    live = n < chunk_of(p.first, p.count, b, p.N, p.cap).count;
  }
  if (ROPE) {
    for (int i = threadIdx.x; i < H2 << p.rb_log2; i += kQueryThreads) {
      const int64_t r = row0 + i / H2;
      if (r >= p.rows) break;
      int rn;
      const int rb = where(r, &rn);
      const Chunk c = chunk_of(p.first, p.count, rb, p.N, p.cap);
      if (rn >= c.count) continue;
      const int j = i % H2, q = j / CP, u = j % CP;
      const float4 a = turn_cossin(static_cast<float>(c.first + rn), freq_at(p.freqs, 8 * u + q));
      ang[(i / H2) * H2 + q * CP + u] = a;
    }
    __syncthreads();
  }
  for (int h0 = 0; h0 < p.Hq; h0 += step) {  // (all threads alike: the warp exchanges maxima)
    const int h = h0 + (k >> p.rb_log2);
    const bool on = live && h < p.Hq;
    float x[16];
    if (on) {
      const uint8_t* from = p.q + b * p.q_sb + n * p.q_sn + h * p.q_sh + t * 16;
      const uint4 lo = __ldg(reinterpret_cast<const uint4*>(from)), hi = __ldg(reinterpret_cast<const uint4*>(from + D));
      const uint32_t L[4] = {lo.x, lo.y, lo.z, lo.w}, G[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float xl = (q & 1) ? bf16hi_to_f32(L[q / 2]) : bf16lo_to_f32(L[q / 2]);
        const float xh = (q & 1) ? bf16hi_to_f32(G[q / 2]) : bf16lo_to_f32(G[q / 2]);
        x[q] = xl, x[8 + q] = xh;
        if (ROPE) {
          const float4 a = ang[rr * H2 + q * CP + t];
          const float c = a.x + a.y, s = a.z + a.w;
          x[q] = __fmaf_rn(xl, c, -xh * s);
          x[8 + q] = __fmaf_rn(xh, c, xl * s);
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q) x[q] = 0.f;
    }
    float f = 1.f;
    if (Q4) {
      float most = 0.f;
#pragma unroll
      for (int q = 0; q < 16; ++q) most = fmaxf(most, fabsf(x[q]));
#pragma unroll
      for (int o = CP / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      // to [2^14, 2^15), by 2^100 at most
      const uint32_t e = max(__float_as_uint(most) >> 23, 41u);
      const float up = __uint_as_float((254u + 14u - e) << 23);
      f = __uint_as_float((e - 14u) << 23);
#pragma unroll
      for (int q = 0; q < 16; ++q) x[q] *= up;
    }
    // 4 bits: of every 64 elements, e and 32 + e side by side. With d = 128 the thread four further on
    // has the partners: the first keeps the first four of each eight.
    int at = t * 8, next = D / 2;  // where the first eight values go, and how far on the others
    if constexpr (Q4) {
      float y[16];
      if constexpr (D == 128) {
        const bool up = t & 4;
#pragma unroll
        for (int q = 0; q < 16; q += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float other = __shfl_xor_sync(0xffffffffu, up ? x[q + e] : x[q + 4 + e], 4);
            y[q + 2 * e] = up ? other : x[q + e];
            y[q + 2 * e + 1] = up ? x[q + 4 + e] : other;
          }
        at = 16 * (t & 3) + (up ? 8 : 0);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[2 * e] = x[e], y[2 * e + 1] = x[8 + e];
        at = 16 * t, next = 8;
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) x[q] = y[q];
    }
    if (!on) continue;
    const int64_t to = (static_cast<int64_t>(b) * p.Hq + h) * p.N + n;
    if (Q4 && t == 0) p.factor[to] = f;
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float a = x[2 * w], c = x[2 * w + 1];
      if (Q4) {
        const __half2 y = __floats2half2_rn(a, c);
        hi[w] = *reinterpret_cast<const uint32_t*>(&y);
        const float2 back = __half22float2(y);
        const __half2 z = __floats2half2_rn(a - back.x, c - back.y);
        lo[w] = *reinterpret_cast<const uint32_t*>(&z);
      } else {
        hi[w] = pack_bf16x2(a, c);
        lo[w] = pack_bf16x2(a - bf16lo_to_f32(hi[w]), c - bf16hi_to_f32(hi[w]));
      }
    }
    uint16_t* dst = p.hi + to * D + at;
    *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(dst + next) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
    if (ROPE) {
      dst = p.lo + to * D + at;
      *reinterpret_cast<uint4*>(dst) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      *reinterpret_cast<uint4*>(dst + next) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class... P>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const P&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, bool Q4, bool TWO, int ROWS_>
cudaError_t launch(const PagedAttendParams& p, cudaStream_t stream) {
  using C = Cfg<D, Q4, TWO, ROWS_>;
  constexpr size_t bytes = smem_bytes<D, Q4, TWO, ROWS_>();
  static_assert(bytes <= 232448, "shared memory");
  auto kern = attend_kernel<D, Q4, TWO, ROWS_>;
  static std::atomic<uint64_t> ready;  // devices that the kernel's shared memory was allowed on
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit) || dev > 63) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  e = launch_pdl<PagedAttendParams>(kern, dim3(p.ctas), C::THREADS, bytes, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl<PagedAttendWork>(attend_join_kernel<D>, dim3(p.ctas, C::ROWS / kJoinRows), 256, 0, stream, p);
}

// Rows of a unit. Two row tiles share the keys that are read (and, 4 bits, expanded); where a 4-bit
// cache's calls have one row tile anyway, shared memory has more of the keys instead.
int unit_rows(int format, int N, int g) { return format == kPagedQ4 && static_cast<int64_t>(N) * g <= 128 ? 128 : 256; }

size_t part_bytes(int d, int unit) {
  return (size_t)std::min(paged_sm_count(), kPagedMaxCtas) * 2 * unit * (d * sizeof(float) + sizeof(float2)) +
         kPagedMaxCtas * sizeof(Pos);
}

}  // namespace

// Partial rows of each CTA; where q is rotated or the cache has 4 bits, its parts and their factors.
size_t paged_attend_workspace(int B, int Hq, int Hkv, int N, int d, int format, bool rope) {
  const size_t rows = (size_t)B * Hq * N;
  size_t n = part_bytes(d, unit_rows(format, N, Hq / Hkv));
  if (rope || format == kPagedQ4) n += rows * d * 2 * (rope ? 2 : 1);
  if (format == kPagedQ4) n += rows * sizeof(float);
  return n;
}

cudaError_t launch_paged_attend(const PagedAttendCall& c, int d, int format, cudaStream_t stream) {
  PagedAttendParams p = c.p;
  const bool q4 = format == kPagedQ4, two = c.rope;
  p.ctas = std::min(paged_sm_count(), kPagedMaxCtas);
  p.unit = unit_rows(format, p.N, p.g);
  p.unit_log2 = p.unit == 128 ? 7 : 8;
  // Half of a unit's rows have half of its products and weights, but all of its keys: more than half of the
  // time where few tiles of them fit into shared memory, q in two parts and d = 128 (bf16: 3; 4 bits: one of K,
  // one of V). With 4 bits and d = 64 or windows either way is better in some cases. Measured with 2, 3 and 4
  // quarters, us, Hq 32, Hkv 8: 24 chunks of up to 300 tokens over up to 6001 keys, and 32 of one or up to 512
  // tokens over up to 4096.
  //   d 128, two parts: bf16 295, 267, 260 and 413, 328, 333; windows of 1024 keys 136, 131, 128 and 245, 218, 220;
  //     4 bits 339, 326, 342 and 451, 409, 422; with windows 158, 161, 159 and 275, 277, 279
  //   d 128, one part: bf16 195, 200, 212 and 256, 263, 275; with windows 101, 103, 101 and 167, 169, 171;
  //     4 bits 297, 294, 304 and 377, 377, 391; with windows 148, 149, 146 and 256, 256, 255
  //   d 64, one part: bf16 152, 157, 168 and 193, 198, 209; with windows 75, 77, 78 and 129, 131, 134;
  //     4 bits 271, 256, 268 and 325, 313, 339; with windows 122, 127, 123 and 219, 214, 220
  //   d 64, two parts: bf16 171, 175, 186 and 220, 225, 237; with windows 89, 91, 91 and 155, 156, 158;
  //     4 bits 266, 260, 270 and 328, 323, 336; with windows 124, 127, 125 and 222, 220, 221
  // (Groups of one, Hkv 16: the same, but that 4 bits with d = 64 take 190, 193, 221.)
  p.half_cost = two && d == 128 ? 3 : 2;
  p.div_g = ((1ull << 63) + p.g - 1) / p.g;
  p.bounds = static_cast<Pos*>(c.workspace);
  p.part_acc = reinterpret_cast<float*>(p.bounds + kPagedMaxCtas);
  p.part_ml = reinterpret_cast<float2*>(p.part_acc + (int64_t)p.ctas * 2 * p.unit * d);
  if (two || q4) {
    PagedQueryParams q;
    q.q = reinterpret_cast<const uint8_t*>(p.q);
    q.q_sb = p.q_sb * 2, q.q_sh = p.q_sh * 2, q.q_sn = p.q_sn * 2;
    q.first = p.first;
    q.count = p.count;
    q.cap = p.cache.cap;
    q.Hq = p.Hq;
    q.N = p.N;
    q.rows = (int64_t)p.cache.B * p.N;
    q.div_n = p.N > 1 ? ~0ull / p.N + 1 : 0;
    const int64_t plane = q.rows * p.Hq * d;
    q.hi = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(c.workspace) + part_bytes(d, p.unit));
    q.lo = two ? q.hi + plane : nullptr;
    q.factor = reinterpret_cast<float*>(q.hi + plane * (two ? 2 : 1));
    q.freqs = c.freqs;
    const int places = kQueryThreads / (d / 16);
    q.rb_log2 = 0;
    while ((places >> q.rb_log2) > p.Hq) ++q.rb_log2;
    void (*kern)(PagedQueryParams);
    if (q4)
      kern = d == 128 ? (two ? attend_query_kernel<128, true, true> : attend_query_kernel<128, true, false>)
                      : (two ? attend_query_kernel<64, true, true> : attend_query_kernel<64, true, false>);
    else
      kern = d == 128 ? attend_query_kernel<128, false, true> : attend_query_kernel<64, false, true>;
    const cudaError_t e = launch_pdl<PagedQueryParams>(
        kern, dim3(static_cast<unsigned>((q.rows + (1 << q.rb_log2) - 1) >> q.rb_log2)), kQueryThreads,
        two ? (d / 2 * sizeof(float4)) << q.rb_log2 : 0, stream, q);
    if (e != cudaSuccess) return e;
    p.q = reinterpret_cast<const __nv_bfloat16*>(q.hi);
    p.q_sn = d, p.q_sh = (int64_t)p.N * d, p.q_sb = (int64_t)p.Hq * p.N * d;
    p.q_lo = plane;
    p.factor = q.factor;
  }
  if (q4 && p.unit == 128) {
    if (d == 128) return two ? launch<128, true, true, 128>(p, stream) : launch<128, true, false, 128>(p, stream);
    return two ? launch<64, true, true, 128>(p, stream) : launch<64, true, false, 128>(p, stream);
  }
  if (q4) {
    if (d == 128) return two ? launch<128, true, true, 256>(p, stream) : launch<128, true, false, 256>(p, stream);
    return two ? launch<64, true, true, 256>(p, stream) : launch<64, true, false, 256>(p, stream);
  }
  if (d == 128) return two ? launch<128, false, true, 256>(p, stream) : launch<128, false, false, 256>(p, stream);
  return two ? launch<64, false, true, 256>(p, stream) : launch<64, false, false, 256>(p, stream);
}

}  // namespace afx
