// Rotation of q and k by positions that the caller gives for each token on up to four axes (time,
// height and width of an image or a video, say), and its inverse, which is its gradient.
//
//   y_i = x_i cos a - x_{i + d/2} sin a,  y_{i + d/2} = x_{i + d/2} cos a + x_i sin a,
//   a = pos[axis(i)][b][n] f_i  (negative for the inverse)
//
// Each element is read once and written once, and HBM bounds it (2 x 8000 tokens of 40 heads, d = 128:
// 61 us, 79% of a copy's rate; 24 x 1025 of 32 heads, d = 64: 39 us, 76%; blocks of 64 or 256 threads, 8 rows,
// or two heads in flight: within 5%). A block takes a few rows (tokens)
// and a run of their heads, of q and k alike: the angles of its rows are computed once, finer than
// fp32 as in the paged append (some 60 instructions each), into shared memory, and serve all of
// the block's heads.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "paged.cuh"

namespace afx {

namespace {

constexpr int kThreads = 128;
// Angles of a row in shared memory, in 16-byte words: with d = 64 padded, so that the four rows that a
// warp reads at once fall in different banks (200 MB of images' rows: 44.8 us without).
template <int D>
constexpr int kAngleRow = D == 64 ? D / 2 + D / 16 : D / 2;

template <int D>
__global__ void __launch_bounds__(kThreads) rope_axes_kernel(const __grid_constant__ RopeAxesParams p) {
  constexpr int CP = D / 16;  // threads of a row: 8 pairs (x_i, x_{i + D/2}) each, two 16-byte pieces
  constexpr int H2 = D / 2, AR = kAngleRow<D>;
  extern __shared__ float4 ang[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) << p.rb_log2;
  const int t = threadIdx.x % CP, k = threadIdx.x / CP, rr = k & ((1 << p.rb_log2) - 1);
  const int64_t row = row0 + rr;
  const int step = (kThreads / CP) >> p.rb_log2;  // heads of a pass
  const int h0 = blockIdx.y * step * p.passes + (k >> p.rb_log2);
  const int h1 = min(p.H, static_cast<int>(blockIdx.y + 1) * step * p.passes);
  const bool in = row < p.rows;
  const int b = in ? static_cast<int>(p.div_n ? __umul64hi(static_cast<uint64_t>(row), p.div_n) : row) : 0;
  const int n = in ? static_cast<int>(row - static_cast<int64_t>(b) * p.N) : 0;
  auto at = [&](const uint8_t* const (&base)[2], const int64_t (&sb)[2], const int64_t (&sh)[2], const int64_t (&sn)[2], int h) {
    const int w = h >= p.Hq;
    return base[w] + b * sb[w] + n * sn[w] + (h - (w ? p.Hq : 0)) * sh[w] + t * 16;
  };
  uint4 lo, hi;
  auto load = [&](int h) {
    if (!in || h >= h1) return;
    const uint8_t* x = at(p.x, p.x_sb, p.x_sh, p.x_sn, h);
    lo = *reinterpret_cast<const uint4*>(x);  // (not the read-only path: y may be x)
    hi = *reinterpret_cast<const uint4*>(x + D);
  };
  load(h0);
  for (int i = threadIdx.x; i < H2 << p.rb_log2; i += kThreads) {
    const int64_t r = row0 + i / H2;
    if (r >= p.rows) break;
    const int j = i % H2;
    const int rb = static_cast<int>(p.div_n ? __umul64hi(static_cast<uint64_t>(r), p.div_n) : r);
    const int rn = static_cast<int>(r - static_cast<int64_t>(rb) * p.N);
    const int q = j / CP, u = j % CP;  // angle slot (q, u) is that of thread u's q-th pair
    const float4 f = freq_at(p.freqs, 8 * u + q);
    const int pos = __ldg(p.pos + __float_as_int(f.w) * p.pos_sa + rb * p.pos_sb + rn * p.pos_sn);
    const float4 a = turn_cossin_far(pos, f);
    const float s = p.inverse ? -1.0f : 1.0f;
    // angles 2m and 2m + 1 of a thread packed: (cos hi, cos hi, cos lo, cos lo), then the sines
    float* to = reinterpret_cast<float*>(ang + (i / H2) * AR + (q / 2) * 2 * CP + u) + (q & 1);
    to[0] = a.x;
    to[2] = a.y;
    to[4 * CP] = s * a.z;
    to[4 * CP + 2] = s * a.w;
  }
  __syncthreads();
  const ulonglong2* mine = reinterpret_cast<const ulonglong2*>(ang + rr * AR + t);
  for (int h = h0; h < h1; h += step) {
    uint4 l = lo, g = hi;
    load(h + step);
    if (!in) continue;
    uint32_t* L = reinterpret_cast<uint32_t*>(&l);
    uint32_t* G = reinterpret_cast<uint32_t*>(&g);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const ulonglong2 c = mine[q * 2 * CP], s = mine[(q * 2 + 1) * CP];
      rot_word_exact(L[q], G[q], c.x, c.y, s.x, s.y);
    }
    uint8_t* y = const_cast<uint8_t*>(at({p.y[0], p.y[1]}, p.y_sb, p.y_sh, p.y_sn, h));
    *reinterpret_cast<uint4*>(y) = l;
    *reinterpret_cast<uint4*>(y + D) = g;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace

cudaError_t launch_rope_axes(RopeAxesParams p, int d, cudaStream_t stream) {
  const int places = kThreads / (d / 16);  // (row, head) places of a pass
  // rows of a block: 4 are contiguous in memory for each head; with few rows one, so that all of
  // its heads go out at once. Heads in turn: as many as leave 8 blocks per SM.
  const int64_t sms = paged_sm_count();
  p.rb_log2 = p.rows * p.H >= 8 * sms * places ? 2 : 0;
  const int step = places >> p.rb_log2;
  const int64_t blocks = (p.rows + (1 << p.rb_log2) - 1) >> p.rb_log2;
  const int most = (p.H + step - 1) / step;
  p.passes = (int)std::max<int64_t>(1, std::min<int64_t>(most, blocks * most / (8 * sms)));
  p.passes = (most + (most + p.passes - 1) / p.passes - 1) / ((most + p.passes - 1) / p.passes);  // even runs
  auto kern = d == 128 ? rope_axes_kernel<128> : rope_axes_kernel<64>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), (most + p.passes - 1) / p.passes);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = ((d == 128 ? kAngleRow<128> : kAngleRow<64>) * sizeof(float4)) << p.rb_log2;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace afx
