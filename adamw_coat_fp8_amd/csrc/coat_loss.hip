// coat_loss.hip -- gfx950 softmax cross entropy from hidden states and the
// output projection's weights, with its gradients, and its C ABI.

#include <hip/hip_runtime.h>

#include <float.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "coat_tile.h"

using namespace coat;

namespace {

// With l = c x W^T (never stored) a row's loss is
//   lse - l[t] + z lse^2,  lse = log sum over v of exp(l[v]),
// and the gradient of l is
//   g[v] = d ((1 + 2 z lse) exp(l[v] - lse) - [v = t]),  dx = c g W,  dW = c g^T x.
//
// Forward: one product whose tiles end in a maximum and a sum of exponentials
// for each row and strip of columns (in powers of two), joined by a second
// kernel.  Backward, for one piece of the vocabulary after the other: the
// piece's logits again, whose tiles end in g as BF16; then g W and g^T x.
//
// Rows without a target take no part: the rows that have one are listed first
// (prep_kernel), the products run over those alone, and the number of them
// stays on the device, where blocks without work end at once.
//
// g is stored divided by the largest |d| of the call, which multiplies the
// products' FP32 results: with one d for all rows, a mean's, the target's
// value 1 - p of an unlikely target then lies near 1, where BF16 is exact, and
// is not rounded alike in every row.  In BF16, as the matrix cores take it at
// their rate: with one part the gradients of 8192 x 32000 x 4096 are 1.9e-3 of
// their norm off, 1.65e-3 if only the results are rounded, and a second part
// takes a product more for each of dx and dW (1.5 to 1.7 ms of 4.8).
//
// Large calls are bound by the matrix cores and, within those, by the card's
// power (coat_tile.h); the logits never leave the chip, so that the forward
// pass reads x and W and writes 8 bytes a row and strip.  8192 x 32000 x 4096 in
// BF16: loss 1508 to 1550 us (1.40 PFLOP/s; the library's product of these
// sizes, which writes logits, 1440 to 1540), gradients 4730 to 4825 (three
// products, 1.34; the library's three 4900 to 5140); of codes 808 to 855 (2.6).
// Of a tile's 99 us some 12 are its beginning, where nothing is loaded yet, and
// its end: exponentials, 16 cycles each, and g's way out.  One row is bound by reading W: 57 us for 262 MB (4.6 TB/s).

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

constexpr int mf_of(bool fp8) { return fp8 ? 32 : 16; }
template <bool kFP8>
using LargeOf = MmaTile<mf_of(kFP8), 4, 2, 2, 4>;                        // 256 x 256, eight waves of 64 x 128
template <bool kFP8>
using HalfOf = MmaTile<mf_of(kFP8), 2, 4, 2, 2, LargeOf<kFP8>::kA>;      // 128 x 256, eight waves of 64 x 64
template <bool kFP8>
using SmallOf = MmaTile<mf_of(kFP8), 2, 2, 2, 2>;                        // 128 x 128, four waves of 64 x 64
using Large = LargeOf<false>;
using Half = HalfOf<false>;
using Small = SmallOf<false>;
template <int kI>
using Thin = MmaTile<32, 1, 2, kI, 1, 0, 5>;    // 32 kI x 64, two waves, five stages
constexpr int kThinCols = 64, kThinStrip = 32;
using ThinDx = MmaTile<16, 1, 4, 4, 1>;         // 128 x 128, four waves of 128 x 32
constexpr int64_t kThinRows = 64, kFewRows = 128, kSmallSteps = 2, kSmallCols = 2048;

constexpr int kStrip = 128;       // columns of a partial softmax, but for thin tiles
constexpr int kGroupM = 4;        // tile rows that are walked together
constexpr int kUnits = 256;       // compute units of the device the plans are made for

// What the backward pass needs of a row: log2(e) lse, the factor of
// exp(l - lse), what the target's value is lowered by (of codes that value),
// the target.
struct RowInfo {
  float lse2, coef, hot;
  int32_t target;
};

struct Header {
  int32_t live;   // rows that have a target
  float d_max;    // what g was divided by
  int32_t pad[14];
};

// Over the kL lanes that share a row of a tile.
template <class Op>
__device__ __forceinline__ float halves_join(float x, Op op) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

template <int kL, class Op>
__device__ __forceinline__ float row_join(float x, Op op) {
  if constexpr (kL == 4) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return halves_join(x, op);
}

template <int kL>
__device__ __forceinline__ float row_max(float x) {
  return row_join<kL>(x, [](float a, float b) { return fmaxf(a, b); });
}

template <int kL>
__device__ __forceinline__ float row_sum(float x) {
  return row_join<kL>(x, [](float a, float b) { return a + b; });
}

// ---------------------------------------------- the target's logit of codes

// The matrix cores align eight neighbouring products of codes to the largest
// and cut them 13 bits below it.  That leaves a logit of 4096 products about
// 1e-5 off, where each is exact and FP32 sums would leave 1e-6.  Among the
// exponentials it averages out; the target's logit enters the loss by itself.
// So for codes it is formed in FP32, and the tiles leave it out of their maxima
// and sums: the join adds its exponential, which keeps the loss of a likely
// target (a small difference of the two) right, and finite however far the two
// forms lie apart (a sum that the tile's exponential is taken from again can be
// left with less than nothing).  Loss of 8192 x 32000 x 4096: 2.4e-6 -> 1e-7 of
// it off, for 1% of the time; products in BF16 on the matrix cores, which hold
// FP32, would take twice the time.  The backward pass forms it too: with the
// cut one beside this lse, g of a likely target, p - 1, would be off by what
// the two forms differ in, also where p - 1 is less.
struct TargetDot {
  const uint8_t* x;     // codes, or NULL: not for these inputs
  const uint8_t* w;
  int64_t K;
  float scale2;
};

// The wave's dot product of row `row` of x and row `v` of w, scaled.
__device__ __forceinline__ float target_dot(const TargetDot& d, int64_t row, int64_t v) {
  const int lane = threadIdx.x & 63;
  const uint8_t *x = d.x + row * d.K, *w = d.w + v * d.K;
  float s[4] = {0, 0, 0, 0};
  for (int64_t k = 16 * lane; k < d.K; k += 1024) {
    const uint4 a = *reinterpret_cast<const uint4*>(x + k), b = *reinterpret_cast<const uint4*>(w + k);
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float f[4], g[4];
      e4m3_values4(aw[q], f);
      e4m3_values4(bw[q], g);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[q] = __builtin_fmaf(f[e], g[e], s[q]);
    }
  }
  return lanes_sum<64>((s[0] + s[1]) + (s[2] + s[3])) * d.scale2;
}

// ------------------------------------------------------ rows with a target

struct PrepParams {
  const int64_t* targets;
  const float* d_loss;   // or NULL: no RowInfo
  const float* lse;
  Header* header;
  int32_t* list;         // row of each listed one
  int32_t* place;        // of each row in the list, or -1
  int32_t* target;       // of each listed row, or NULL
  RowInfo* info;         // of each listed row, or NULL
  int64_t M, V;
  float z;
};

// Of row r, by a wave.
__device__ __forceinline__ RowInfo row_info(const PrepParams& p, int64_t r, float d_max, const TargetDot& dot) {
  const float lse = p.lse[r], d = p.d_loss[r] / d_max;
  RowInfo f;
  f.lse2 = lse * kLog2e;
  f.coef = d * __builtin_fmaf(2.0f * p.z, lse, 1.0f);
  f.target = (int32_t)p.targets[r];
  f.hot = dot.x ? f.coef * __builtin_amdgcn_exp2f(target_dot(dot, r, f.target) - f.lse2) - d : d;
  return f;
}

// One block: a running count over 8192 rows at a time, in order.  Row
// 1024 e + t of them is thread t's e-th.
__global__ __launch_bounds__(1024) void prep_kernel(const PrepParams p) {
  constexpr int kEach = 8, kCounts = 16 * kEach;
  __shared__ int32_t before[kCounts + 1];   // rows of the 64s before each
  __shared__ float wave_max[16];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int32_t base = 0;
  float top = 0.0f;
  for (int64_t first = 0; first < p.M; first += 1024 * kEach) {
    int64_t target[kEach];
    float d[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int64_t r = first + 1024 * e + t;
      target[e] = r < p.M ? p.targets[r] : -1;
      d[e] = p.d_loss && r < p.M ? p.d_loss[r] : 0.0f;
    }
    uint64_t lives[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const bool live = target[e] >= 0 && target[e] < p.V;
      lives[e] = __ballot(live);
      top = live ? fmaxf(top, fabsf(d[e])) : top;
      if (lane == 0) before[16 * e + wave] = __popcll(lives[e]);
    }
    __syncthreads();
    if (wave == 0) {   // their running sum, two a lane
      static_assert(kCounts == 128, "two a lane");
      const int32_t a = before[2 * lane], both = a + before[2 * lane + 1];
      int32_t upto = both;
#pragma unroll
      for (int s = 1; s < 64; s *= 2) {
        const int32_t o = __shfl_up(upto, s);
        if (lane >= s) upto += o;
      }
      before[2 * lane] = upto - both;
      before[2 * lane + 1] = upto - both + a;
      if (lane == 63) before[kCounts] = upto;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int64_t r = first + 1024 * e + t;
      if (r >= p.M) continue;
      const bool live = (lives[e] >> lane) & 1;
      const int32_t at = base + before[16 * e + wave] + __popcll(lives[e] & (((uint64_t)1 << lane) - 1));
      p.place[r] = live ? at : -1;
      if (!live) continue;
      p.list[at] = (int32_t)r;
      if (p.target) p.target[at] = (int32_t)target[e];
    }
    base += before[kCounts];
    __syncthreads();   // `before` is read
  }
  if (t == 0) p.header->live = base;
  if (!p.d_loss) return;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) top = fmaxf(top, __shfl_xor(top, s));
  if (lane == 0) wave_max[wave] = top;
  __syncthreads();
  if (t > 0) return;
  for (int w = 0; w < 16; ++w) top = fmaxf(top, wave_max[w]);
  p.header->d_max = top > 0.0f && top <= FLT_MAX ? top : 1.0f;
}

struct GatherParams {
  const uint8_t* x;          // M x K BF16, or codes
  uint16_t* x_bf16;          // listed rows (written), or NULL
  uint8_t* x_codes;          // or NULL
  uint16_t* dx;              // zeros for rows without a target, or NULL
  int64_t K;
  int32_t fp8;
  TargetDot dot;
};

__device__ __forceinline__ uint4 bf16_of_codes(uint2 c) {
  float f[8];
  e4m3_values8(c, f);
  return pack8(f);
}

// Row r of x into its place `at` in the list, codes as BF16 (exact) and as
// they are.
__device__ __forceinline__ void gather_row(const GatherParams& p, int64_t r, int at) {
  const int64_t chunks = p.K / 8;
  if (at < 0) {
    if (p.dx)
      for (int64_t c = threadIdx.x; c < chunks; c += 256)
        *reinterpret_cast<uint4*>(p.dx + r * p.K + 8 * c) = make_uint4(0, 0, 0, 0);
    return;
  }
  for (int64_t c = threadIdx.x; c < chunks; c += 256) {
    if (p.fp8) {
      const uint2 v = load_stream8(p.x + r * p.K + 8 * c);
      if (p.x_codes) *reinterpret_cast<uint2*>(p.x_codes + at * p.K + 8 * c) = v;
      if (p.x_bf16) *reinterpret_cast<uint4*>(p.x_bf16 + at * p.K + 8 * c) = bf16_of_codes(v);
    } else {
      *reinterpret_cast<uint4*>(p.x_bf16 + at * p.K + 8 * c) = load_stream16(p.x + 2 * (r * p.K + 8 * c));
    }
  }
}

__global__ __launch_bounds__(256) void gather_kernel(const PrepParams p, const GatherParams g) {
  const int32_t at = p.place[blockIdx.x];
  if (at >= 0 && threadIdx.x < 64) {
    const RowInfo f = row_info(p, blockIdx.x, p.header->d_max, g.dot);
    if (threadIdx.x == 0) p.info[at] = f;
  }
  gather_row(g, blockIdx.x, at);
}

// Both for at most 64 rows, a block each.
__global__ __launch_bounds__(256) void prep_few_kernel(const PrepParams p, const GatherParams g) {
  const int64_t r = blockIdx.x;
  const int lane = threadIdx.x & 63;
  const int64_t target = lane < p.M ? p.targets[lane] : -1;
  const bool live = target >= 0 && target < p.V;
  const uint64_t lives = __ballot(live);
  float top = live ? fabsf(p.d_loss[lane]) : 0.0f;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) top = fmaxf(top, __shfl_xor(top, s));
  const float d_max = top > 0.0f && top <= FLT_MAX ? top : 1.0f;
  if (r == 0 && threadIdx.x == 0) {
    p.header->live = __popcll(lives);
    p.header->d_max = d_max;
  }
  const int at = (lives >> r) & 1 ? __popcll(lives & (((uint64_t)1 << r) - 1)) : -1;
  if (at >= 0 && threadIdx.x < 64) {
    const RowInfo f = row_info(p, r, d_max, g.dot);
    if (threadIdx.x == 0) {
      p.list[at] = (int32_t)r;
      p.info[at] = f;
    }
  }
  gather_row(g, r, at);
}

// E4M3 codes as BF16, exactly; eight a thread.
__global__ __launch_bounds__(256) void expand_kernel(const uint8_t* codes, int64_t chunks, uint16_t* out) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c < chunks) *reinterpret_cast<uint4*>(out + 8 * c) = bf16_of_codes(load_stream8(codes + 8 * c));
}

// ---------------------------------------------------------------- logits

struct LogitParams {
  const uint8_t* x;         // rows of `stride` bytes; listed ones of them with list
  const uint8_t* w;         // the piece's weights, N rows of `stride` bytes
  const int32_t* list;      // or NULL: row m is row m
  const Header* header;     // or NULL: M rows
  int64_t M, N, V;
  uint32_t stride;
  int32_t steps, n_tiles;
  float scale2;             // log2(e) times what a product is multiplied by
  // loss
  float2* part;             // largest logit and sum of exponentials of each strip and row
  int64_t strip_step, row_step;
  float* at_target;         // the target's logit of each row (BF16)
  const int32_t* target;    // of listed rows, or NULL
  const int64_t* targets;
  // gradient
  const RowInfo* info;
  uint16_t* g;              // rows of ld values
  uint16_t* g_rest;         // what BF16 left of g, or NULL
  int64_t ld;
  int32_t v0;               // first vocabulary row of the piece
};

// Tile order: groups of kGroupM tile rows, column by column inside a group.
__device__ __forceinline__ void tile_at(uint32_t order, uint32_t m_tiles, uint32_t n_tiles, uint32_t& tm, uint32_t& tn) {
  const uint32_t group = order / (kGroupM * n_tiles), first = group * kGroupM;
  const uint32_t rows = m_tiles - first < kGroupM ? m_tiles - first : kGroupM;
  const uint32_t local = order - group * kGroupM * n_tiles;
  tn = local / rows;
  tm = first + local - tn * rows;
}

// How M rows are cut into tiles of n_tiles columns: 256 rows each, but 128 for
// a last row of tiles that holds no more; and the last round of whole tiles in
// halves, where that ends earlier.  In units of half a tile's time, whole
// tiles first: keeping `rem` of them in the last round takes 2 units there and
// leaves room for 2 (units - rem) halves.
struct TilePlan {
  uint32_t rows, whole, halves;   // whole rows of tiles; whole tiles; halves behind them: the last row's, then split ones
  uint32_t last;                  // halves of the last row
  __host__ __device__ TilePlan(int64_t M, uint32_t n_tiles) {
    const uint32_t rest = (uint32_t)(M % Large::kBM);
    rows = (uint32_t)(M / Large::kBM) + (rest > Half::kBM);
    last = rest > 0 && rest <= Half::kBM ? n_tiles : 0;
    whole = rows * n_tiles;
    const uint32_t rem = whole % kUnits;
    const uint32_t split = rem > 0 && last + 2 * rem <= kUnits ? rem : 0;
    whole -= split;
    halves = last + 2 * split;
  }
};

// The tile of block b; false: none.
struct TileAt {
  int64_t m0;
  uint32_t tn;
  bool half;
};

__device__ __forceinline__ bool tile_of(uint32_t b, const TilePlan& p, uint32_t n_tiles, TileAt& t) {
  uint32_t tm;
  if (b < p.whole) {
    tile_at(xcd_contiguous32(b, p.whole), p.rows, n_tiles, tm, t.tn);
    t.m0 = (int64_t)tm * Large::kBM;
    t.half = false;
    return true;
  }
  if (b >= p.whole + p.halves) return false;
  const uint32_t order = xcd_contiguous32(b - p.whole, p.halves);
  t.half = true;
  if (order < p.last) {
    t.m0 = (int64_t)p.rows * Large::kBM;
    t.tn = order;
  } else {
    tile_at(p.whole + ((order - p.last) >> 1), p.rows, n_tiles, tm, t.tn);
    t.m0 = (int64_t)tm * Large::kBM + Half::kBM * ((order - p.last) & 1);
  }
  return true;
}

template <class T, bool kFP8, bool kGrad>
__device__ __forceinline__ void logit_tile(const LogitParams& p, const int64_t live, const int64_t m0, const int64_t n0) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % T::kWM, wn = wave / T::kWM, lr = lane % T::kMf, share = lane / T::kMf;
  // rows and columns past the last re-load it
  uint32_t aoff[T::kLA], boff[T::kLB];
  const uint8_t* a0 = p.list ? p.x : p.x + m0 * p.stride;
  const uint8_t* b0 = p.w + n0 * p.stride;
  minor_offsets(wave, lane, [&](int r) __attribute__((always_inline)) {
    const int64_t m = m0 + r < live ? m0 + r : live - 1;
    return p.list ? (uint32_t)p.list[m] * p.stride : (uint32_t)(m - m0) * p.stride;
  }, aoff);
  minor_offsets(wave, lane, [&](int r) __attribute__((always_inline)) {
    return (uint32_t)(n0 + r < p.N ? r : (int)(p.N - 1 - n0)) * p.stride;
  }, boff);
  typename T::Acc acc;
  mma_zero<T>(acc);
  if constexpr (T::kStages > 2)
    mma_stream<T, kFP8>(acc, p.steps, a0, aoff, b0, boff);
  else
    mma_run<T, kFP8, false, false>(acc, p.steps, [&](int s) { return a0 + 128 * (int64_t)s; }, aoff, 0,
                                   [&](int s) { return b0 + 128 * (int64_t)s; }, boff, 0, [](int) { return 0; });

  const int64_t col0 = n0 + 32 * T::kJ * wn;          // the wave's first column
  const int64_t valid = p.N - col0;                    // of its columns
  if constexpr (!kGrad) {
    if (valid < 32 * T::kJ) {
#pragma unroll
      for (int i = 0; i < T::kRT; ++i)
#pragma unroll
        for (int u = 0; u < T::kRuns; ++u)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            if (4 * T::kL * u + 4 * share + s >= valid) set_quad<T>(acc, i, u, s, -INFINITY);
    }
#pragma unroll
    for (int i = 0; i < T::kRT; ++i) {
      const int64_t row = m0 + 32 * T::kI * wm + T::kMf * i + lr;
      const bool stored = row < live;
      // the target, where it lies in the lane's columns
      int64_t t = -1;
      if (stored) t = p.target ? (int64_t)p.target[row] : p.targets[row];
      const int64_t at = t - col0;
      const bool mine = t >= 0 && t < p.V && at >= 0 && at < 32 * T::kJ && ((at >> 2) & (T::kL - 1)) == share;
      if constexpr (kFP8) {
        if (__any(mine)) {
          // Left out (TargetDot), a quarter of the columns at a time, of which
          // most have none: loss of codes of 8192 x 32000 x 1024 256 us, all at
          // once 261; of 1024 x 32000 x 2048 63.9 and 65.1.
          constexpr int kQuarter = 32 * T::kJ / 4, kQuarterRuns = T::kRuns / 4;
          const int out = mine ? (int)at - 4 * share : -1;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (!__any(mine && out / kQuarter == q)) continue;
#pragma unroll
            for (int u = q * kQuarterRuns; u < (q + 1) * kQuarterRuns; ++u)
#pragma unroll
              for (int s = 0; s < 4; ++s) set_quad<T>(acc, i, u, s, 4 * T::kL * u + s == out ? -INFINITY : quad<T>(acc, i, u, s));
          }
        }
      }
      // (a NaN is left to the sum)
      float top = -FLT_MAX;
#pragma unroll
      for (int u = 0; u < T::kRuns; ++u)
#pragma unroll
        for (int s = 0; s < 4; s += 2) top = fmaxf(fmaxf(top, quad<T>(acc, i, u, s)), quad<T>(acc, i, u, s + 1));
      top = fmaxf(row_max<T::kL>(top) * p.scale2, -FLT_MAX);
      float sum[4] = {0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < T::kRuns; ++u)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          sum[s] += __builtin_amdgcn_exp2f(__builtin_fmaf(quad<T>(acc, i, u, s), p.scale2, -top));
      float all = row_sum<T::kL>((sum[0] + sum[1]) + (sum[2] + sum[3]));
      int strip = wn;
      if constexpr (32 * T::kJ < kStrip && T::kStages == 2) {
        // two waves share a strip: the odd one hands its part over
        static_assert(64 * T::kJ == kStrip, "two waves");
        float2* shared = reinterpret_cast<float2*>(mma_part<T, 0>()) + 32 * T::kI * wm + T::kMf * i + lr + T::kBM * (wn >> 1);
        if ((wn & 1) && share == 0) *shared = make_float2(top, all);
        __syncthreads();
        if (!(wn & 1)) {
          const float2 o = *shared;
          const float m = fmaxf(top, o.x);
          all = all * __builtin_amdgcn_exp2f(top - m) + o.y * __builtin_amdgcn_exp2f(o.x - m);
          top = m;
        }
        strip = wn & 1 ? -1 : wn >> 1;
      }
      if (stored && share == 0 && strip >= 0)
        p.part[(n0 / (T::kStages == 2 ? kStrip : 32 * T::kJ) + strip) * p.strip_step + row * p.row_step] = make_float2(top, all);
      if constexpr (!kFP8) {
        if (__any(mine)) {
          const float v = value_at<T>(acc, i, (int)at);
          if (mine) p.at_target[row] = v * p.scale2;
        }
      }
    }
  } else {
    const int64_t padded = (live + 63) / 64 * 64;   // rows of g that the products read
    RowInfo f[T::kRT];
#pragma unroll
    for (int i = 0; i < T::kRT; ++i) {
      const int64_t row = m0 + 32 * T::kI * wm + T::kMf * i + lr;
      f[i] = row < live ? p.info[row] : RowInfo{0.0f, 0.0f, 0.0f, -1};
    }
    auto part_of = [&](int i, float product) __attribute__((always_inline)) {
      return f[i].coef * __builtin_amdgcn_exp2f(__builtin_fmaf(product, p.scale2, -f[i].lse2));
    };
    // kRest: what BF16 leaves of the value
    auto pair = [](float a, float b, auto kRest) __attribute__((always_inline)) {
      const uint32_t w = bf16_pack2(a, b);
      if constexpr (!decltype(kRest)::value) return w;
      return bf16_pack2(a - bf16_lo(w), b - bf16_hi(w));
    };
    auto write = [&](uint16_t* g, auto kRest) __attribute__((always_inline)) {
      tile_out_bf16<T>(
          [&](int i, int u) __attribute__((always_inline)) {
            const float v0 = part_of(i, quad<T>(acc, i, u, 0)), v1 = part_of(i, quad<T>(acc, i, u, 1));
            const float v2 = part_of(i, quad<T>(acc, i, u, 2)), v3 = part_of(i, quad<T>(acc, i, u, 3));
            return make_uint2(pair(v0, v1, kRest), pair(v2, v3, kRest));
          },
          // rows and columns past the last are zero
          [&](int row, int c, uint4 v) __attribute__((always_inline)) {
            const int64_t m = m0 + row, n = n0 + 8 * c;
            if (m >= padded || n >= p.ld) return;
            const int64_t left = m < live ? p.N - n : 0;
            if (left < 8) {
              auto keep = [&](int at, uint32_t w) { return left > at + 1 ? w : left > at ? w & 0xFFFFu : 0u; };
              v = make_uint4(keep(0, v.x), keep(2, v.y), keep(4, v.z), keep(6, v.w));
            }
            store_stream16(g + m * p.ld + n, v);
          },
          // the target's value, where it lies in the lane's columns
          [&](int i, auto set) __attribute__((always_inline)) {
            const int64_t at = (int64_t)f[i].target - p.v0 - col0;
            const bool mine = f[i].target >= 0 && at >= 0 && at < 32 * T::kJ && ((at >> 2) & (T::kL - 1)) == share;
            if (!__any(mine)) return;
            float v = f[i].hot;
            if constexpr (!kFP8) v = part_of(i, value_at<T>(acc, i, (int)at)) - v;
            if (mine) set((int)at + 32 * T::kJ * wn, pair(v, 0.0f, kRest) & 0xFFFFu);
          });
    };
    write(p.g, std::false_type{});
    if (p.g_rest) {
      __syncthreads();
      // (values are formed again: kept since the first pass they would not fit
      // the registers)
#pragma unroll
      for (int i = 0; i < T::kRT; ++i) asm volatile("" : "+v"(f[i].lse2));
      write(p.g_rest, std::true_type{});
    }
  }
}

// The grid is that of all M rows; blocks past the last tile of the live ones
// end.  (A block a tile: blocks that stay and fetch the next tile's first panels
// beside this one's end spill registers where the loop's versions meet, 1686 us
// where this took 1603; that stay without it, 1630.  Groups of 2, 8 or 16 tile
// rows, and tiles of four waves of 128 x 128 for the gradients, which spill,
// are slower too.)
template <bool kFP8, bool kGrad>
__global__ __launch_bounds__(Large::kThreads) void logit_large_kernel(const LogitParams p) {
  const int64_t live = p.header ? p.header->live : p.M;
  TileAt t;
  if (!tile_of(blockIdx.x, TilePlan(live, (uint32_t)p.n_tiles), (uint32_t)p.n_tiles, t)) return;
  if (!t.half) logit_tile<LargeOf<kFP8>, kFP8, kGrad>(p, live, t.m0, (int64_t)t.tn * Large::kBN);
  else if (t.m0 < live) logit_tile<HalfOf<kFP8>, kFP8, kGrad>(p, live, t.m0, (int64_t)t.tn * Large::kBN);
}

// Smaller tiles where whole ones would be few.
template <class T, bool kFP8, bool kGrad>
__device__ __forceinline__ void logit_tiles(const LogitParams& p) {
  const int64_t live = p.header ? p.header->live : p.M;
  const uint32_t m_tiles = (uint32_t)((live + T::kBM - 1) / T::kBM), tiles = m_tiles * (uint32_t)p.n_tiles;
  if (blockIdx.x >= tiles) return;
  uint32_t tm, tn;
  tile_at(xcd_contiguous32(blockIdx.x, tiles), m_tiles, (uint32_t)p.n_tiles, tm, tn);
  logit_tile<T, kFP8, kGrad>(p, live, (int64_t)tm * T::kBM, (int64_t)tn * T::kBN);
}

template <bool kFP8, bool kGrad>
__global__ __launch_bounds__(Small::kThreads) void logit_small_kernel(const LogitParams p) {
  logit_tiles<SmallOf<kFP8>, kFP8, kGrad>(p);
}

template <bool kFP8, bool kGrad, int kI>
__global__ __launch_bounds__(128) void logit_thin_kernel(const LogitParams p) {
  logit_tiles<Thin<kI>, kFP8, kGrad>(p);
}

struct JoinParams {
  const float2* part;
  int64_t strip_step, row_step;
  float* at_target;         // as the tiles write it, or for codes target_kernel
  TargetDot dot;
  const int32_t* place;     // of each row in the list, or NULL
  const int64_t* targets;
  float* loss;
  float* lse;               // or NULL
  int64_t M, V;
  int32_t strips;
  float z;
};

// Joins strips g, g + kBy, .. of a row, eight loads in flight.
template <int kBy>
__device__ __forceinline__ float2 join_strips(const JoinParams& p, int64_t at, int g) {
  const float2* part = p.part + at * p.row_step;
  float top = -FLT_MAX, sum = 0.0f;
  for (int s = g; s < p.strips; s += 8 * kBy) {
    float2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = s + i * kBy < p.strips ? part[(s + i * kBy) * p.strip_step] : make_float2(-FLT_MAX, 0.0f);
    float m = top;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, v[i].x);
    sum *= __builtin_amdgcn_exp2f(top - m);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += v[i].y * __builtin_amdgcn_exp2f(v[i].x - m);
    top = m;
  }
  return make_float2(top, sum);
}

// target: its logit, for codes not among those of top and sum.
__device__ __forceinline__ void store_loss(const JoinParams& p, int64_t row, int64_t at, float top, float sum, float target) {
  float loss = 0.0f, lse = 0.0f;
  if (at >= 0) {
    if (p.dot.x) {
      const float m = fmaxf(top, target);
      sum = sum * __builtin_amdgcn_exp2f(top - m) + __builtin_amdgcn_exp2f(target - m);
      top = m;
    }
    const float log2s = __builtin_amdgcn_logf(sum);
    lse = kLn2 * (top + log2s);
    loss = kLn2 * ((top - target) + log2s) + p.z * lse * lse;
  }
  p.loss[row] = loss;
  if (p.lse) p.lse[row] = lse;
}

__device__ __forceinline__ int64_t place_of(const JoinParams& p, int64_t row) {
  const int64_t target = p.targets[row];
  if (target < 0 || target >= p.V) return -1;
  return p.place ? p.place[row] : row;
}

// A wave each row, for codes.
__global__ __launch_bounds__(256) void target_kernel(const JoinParams p) {
  const int64_t row = 4 * (int64_t)blockIdx.x + (threadIdx.x >> 6);
  const int64_t at = row < p.M ? place_of(p, row) : -1;
  if (at < 0) return;
  const float v = target_dot(p.dot, row, p.targets[row]);
  if ((threadIdx.x & 63) == 0) p.at_target[at] = v;
}

// 16 rows, 16 threads each.
__global__ __launch_bounds__(256) void loss_join_kernel(const JoinParams p) {
  __shared__ float2 part[16][17];
  const int t = threadIdx.x, r16 = t & 15, g = t >> 4;
  const int64_t row = (int64_t)blockIdx.x * 16 + r16;
  const int64_t at = row < p.M ? place_of(p, row) : -1;
  part[r16][g] = at >= 0 ? join_strips<16>(p, at, g) : make_float2(-FLT_MAX, 0.0f);
  __syncthreads();
  if (t >= 16 || row >= p.M) return;
  float top = -FLT_MAX, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, part[r16][i].x);
#pragma unroll
  for (int i = 0; i < 16; ++i) sum += part[r16][i].y * __builtin_amdgcn_exp2f(part[r16][i].x - top);
  store_loss(p, row, at, top, sum, at >= 0 ? p.at_target[at] : 0.0f);
}

// Few rows: a wave each.
__global__ __launch_bounds__(64) void loss_join_few_kernel(const JoinParams p) {
  const int64_t row = blockIdx.x, at = place_of(p, row);
  float top = -FLT_MAX, sum = 0.0f, target = 0.0f;
  if (at >= 0) {
    target = p.dot.x ? target_dot(p.dot, row, p.targets[row]) : p.at_target[at];
    const float2 v = join_strips<64>(p, at, threadIdx.x);
    top = v.x;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) top = fmaxf(top, __shfl_xor(top, s));
    sum = lanes_sum<64>(v.y * __builtin_amdgcn_exp2f(v.x - top));
  }
  if (threadIdx.x == 0) store_loss(p, row, at, top, sum, target);
}

// -------------------------------------------------- products with g

enum Out { kBF16 = 0, kF32 = 1, kF32Add = 2 };

// How a product's contraction is split where its tiles leave compute units
// empty: into parts of partial sums.  A function of the rows (M, or the live
// ones) alone, on the device too.
struct Splits {
  int32_t most;        // by the steps: eight to a part at least
  int32_t always;      // partial sums even of one part (joined over pieces)
  int64_t room;        // rows that the partial sums have room for
  int32_t tile_rows, n_tiles, blocks;   // of the tiles; blocks that fill the device
  __host__ __device__ int32_t parts(int64_t rows) const {
    const int64_t tiles = (rows + tile_rows - 1) / tile_rows * n_tiles;
    if (tiles == 0 || tiles > blocks / 2) return 1;
    int64_t s = blocks / tiles;
    s = s < most ? s : most;
    s = s < room / rows ? s : room / rows;
    return (int32_t)(s < 1 ? 1 : s);
  }
};

struct ProductParams {
  const uint8_t* a;         // g: rows of lda bytes
  const uint8_t* a_rest;    // its second part, or NULL
  const uint8_t* b;         // k rows of ldb bytes
  const Header* header;
  const int32_t* list;      // C's row m goes to row list[m], or NULL
  void* out;                // BF16 or FP32, rows of N values
  float* partial;           // FP32 sums, [split][row][N], or NULL
  int64_t M, N;
  Splits splits;
  uint32_t lda, ldb;
  int32_t k_rows;           // contracted rows of b; those of a are padded with zeros to a multiple of 64
  int32_t mode;             // of out
  int32_t add;              // the partial sums are added to
  float scale;              // of out, times the header's d_max
  uint32_t n_tiles;
};

// kGT: C = g^T x (A slow, the contracted rows are the live ones); else g W.
// Both in the layouts as they lie.  8192 x 32000 x 4096: g W 1500 us (1.43
// PFLOP/s; the library 1550), g^T x 1610 (1.33; the library 1940, whose operands
// lie the wrong way round for it).
template <class T, bool kGT>
__device__ __forceinline__ void product_tile(const ProductParams& p, const int64_t live, const int64_t m0, const int64_t n0,
                                             const int part, const int parts) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % T::kWM, wn = wave / T::kWM, lr = lane % T::kMf, share = lane / T::kMf;
  const int64_t M = kGT ? p.M : live;
  const int k_rows = kGT ? (int)live : p.k_rows;
  const int each = (k_rows + 63) / 64, all = p.a_rest ? 2 * each : each;
  const int first = (int)((int64_t)all * part / parts), last = (int)((int64_t)all * (part + 1) / parts);
  uint32_t aoff[kGT ? kSlowDistinct<T::kLA, T::kBM> : T::kLA], boff[kSlowDistinct<T::kLB, T::kBN>];
  if constexpr (kGT) {
    slow_offsets<T::kLA, T::kBM>(wave, lane, p.lda, p.lda / 2 - m0, aoff);
  } else {
    minor_offsets(wave, lane, [&](int r) __attribute__((always_inline)) {
      return (uint32_t)(m0 + r < M ? r : (int)(M - 1 - m0)) * p.lda;
    }, aoff);
  }
  slow_offsets<T::kLB, T::kBN>(wave, lane, p.ldb, p.N - n0, boff);
  typename T::Acc acc;
  mma_zero<T>(acc);
  const uint8_t* a0 = kGT ? p.a + 2 * m0 : p.a + m0 * p.lda;
  const uint8_t* a1 = kGT ? p.a_rest + 2 * m0 : p.a_rest + m0 * p.lda;
  const uint8_t* b0 = p.b + 2 * n0;
  const int64_t a_step = kGT ? 64 * (int64_t)p.lda : 128, b_step = 64 * (int64_t)p.ldb;
  // the last panel's rows (b0 is not at their first column)
  const uint32_t last_bytes = (uint32_t)(k_rows - 64 * (each - 1)) * p.ldb - 2 * (uint32_t)n0;
  mma_run<T, false, kGT, true>(
      acc, last - first,
      [&](int s) { return first + s < each ? a0 + (first + s) * a_step : a1 + (first + s - each) * a_step; }, aoff, p.lda,
      [&](int s) { return b0 + (first + s < each ? first + s : first + s - each) * b_step; }, boff, p.ldb,
      [&](int s) { return first + s == each - 1 || first + s == 2 * each - 1 ? last_bytes : 0xFFFFFFFFu; });
  const bool partial = parts > 1 || p.splits.always;
  if (partial || p.mode != kBF16) {
    const float scale = partial ? 1.0f : p.scale * p.header->d_max;
    const bool add = partial ? p.add : p.mode == kF32Add;
    float* out = partial ? p.partial + part * M * p.N : (float*)p.out;
#pragma unroll
    for (int i = 0; i < T::kRT; ++i) {
      const int64_t row = m0 + 32 * T::kI * wm + T::kMf * i + lr;
      if (row >= M) continue;
#pragma unroll
      for (int u = 0; u < T::kRuns; ++u) {
        const int64_t col = n0 + 32 * T::kJ * wn + 4 * T::kL * u + 4 * share;
        if (col >= p.N) continue;
        float4* dst = reinterpret_cast<float4*>(out + row * p.N + col);
        float4 v = make_float4(quad<T>(acc, i, u, 0) * scale, quad<T>(acc, i, u, 1) * scale, quad<T>(acc, i, u, 2) * scale,
                               quad<T>(acc, i, u, 3) * scale);
        if (add) {
          const float4 o = *dst;
          v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
        }
        *dst = v;
      }
    }
    return;
  }
  const float scale = p.scale * p.header->d_max;
  tile_out_bf16<T>([&](int i, int u) __attribute__((always_inline)) {
    return make_uint2(bf16_pack2(quad<T>(acc, i, u, 0) * scale, quad<T>(acc, i, u, 1) * scale),
                      bf16_pack2(quad<T>(acc, i, u, 2) * scale, quad<T>(acc, i, u, 3) * scale));
  }, [&](int row, int c, uint4 v) __attribute__((always_inline)) {
    const int64_t m = m0 + row, n = n0 + 8 * c;
    if (m < M && n < p.N) store_stream16((uint16_t*)p.out + (p.list ? (int64_t)p.list[m] : m) * p.N + n, v);
  });
}

template <bool kGT>
__global__ __launch_bounds__(Large::kThreads) void product_kernel(const ProductParams p) {
  const int64_t live = p.header->live, M = kGT ? p.M : live;
  const int parts = p.splits.parts(M);
  TileAt t;
  if (parts > 1) {
    const uint32_t m_tiles = (uint32_t)((M + Large::kBM - 1) / Large::kBM), tiles = m_tiles * p.n_tiles;
    if (blockIdx.x >= tiles * parts) return;
    const uint32_t order = xcd_contiguous32(blockIdx.x, tiles * parts), part = order / tiles;
    uint32_t tm;
    tile_at(order - part * tiles, m_tiles, p.n_tiles, tm, t.tn);
    product_tile<Large, kGT>(p, live, (int64_t)tm * Large::kBM, (int64_t)t.tn * Large::kBN, (int)part, parts);
    return;
  }
  if (!tile_of(blockIdx.x, TilePlan(M, p.n_tiles), p.n_tiles, t)) return;
  if (!t.half) product_tile<Large, kGT>(p, live, t.m0, (int64_t)t.tn * Large::kBN, 0, 1);
  else if (t.m0 < M) product_tile<Half, kGT>(p, live, t.m0, (int64_t)t.tn * Large::kBN, 0, 1);
}

// g W for at most 64 rows: g's two parts are rows 0 to 63 and 64 to 127 of a
// tile, and are added where they meet, in the registers.
__global__ __launch_bounds__(ThinDx::kThreads) void product_thin_kernel(const ProductParams p) {
  using T = ThinDx;
  const int64_t live = p.header->live;
  const int parts = p.splits.parts(live);
  const uint32_t blocks = (uint32_t)(p.splits.n_tiles * parts);
  if (live == 0 || blockIdx.x >= blocks) return;
  const uint32_t order = xcd_contiguous32(blockIdx.x, blocks), part = order / p.splits.n_tiles;
  const int64_t n0 = (int64_t)(order - part * p.splits.n_tiles) * T::kBN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int all = (p.k_rows + 63) / 64;
  const int first = (int)((int64_t)all * part / parts), last = (int)((int64_t)all * (part + 1) / parts);
  uint32_t aoff[T::kLA], boff[kSlowDistinct<T::kLB, T::kBN>];
  minor_offsets(wave, lane, [&](int r) __attribute__((always_inline)) { return (uint32_t)r * p.lda; }, aoff);
  slow_offsets<T::kLB, T::kBN>(wave, lane, p.ldb, p.N - n0, boff);
  typename T::Acc acc;
  mma_zero<T>(acc);
  const uint8_t* b0 = p.b + 2 * n0;
  const int64_t b_step = 64 * (int64_t)p.ldb;
  const uint32_t last_bytes = (uint32_t)(p.k_rows - 64 * (all - 1)) * p.ldb - 2 * (uint32_t)n0;
  mma_run<T, false, false, true>(acc, last - first, [&](int s) { return p.a + 128 * (int64_t)(first + s); }, aoff, 0,
                                 [&](int s) { return b0 + (first + s) * b_step; }, boff, p.ldb,
                                 [&](int s) { return first + s == all - 1 ? last_bytes : 0xFFFFFFFFu; });
  const bool partial = parts > 1 || p.splits.always;
  const float scale = p.scale * p.header->d_max;
#pragma unroll
  for (int i = 0; i < T::kRT / 2; ++i) {
    const int64_t row = T::kMf * i + lane % T::kMf;
    if (row >= live) continue;
#pragma unroll
    for (int u = 0; u < T::kRuns; ++u) {
      const int64_t col = n0 + 32 * wave + 4 * T::kL * u + 4 * (lane / T::kMf);
      if (col >= p.N) continue;
      auto both = [&](int s) __attribute__((always_inline)) { return quad<T>(acc, i, u, s) + quad<T>(acc, i + T::kRT / 2, u, s); };
      float4 v = make_float4(both(0), both(1), both(2), both(3));
      if (partial) {
        float4* dst = reinterpret_cast<float4*>(p.partial + (part * live + row) * p.N + col);
        if (p.add) {
          const float4 o = *dst;
          v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
        }
        *dst = v;
      } else {
        *reinterpret_cast<uint2*>((uint16_t*)p.out + (int64_t)p.list[row] * p.N + col) =
            make_uint2(bf16_pack2(v.x * scale, v.y * scale), bf16_pack2(v.z * scale, v.w * scale));
      }
    }
  }
}

struct FinishParams {
  const float* partial;     // [split][row][N]
  const Header* header;
  const int32_t* list;      // rows of out, and the live rows alone; or NULL: M rows
  void* out;
  int64_t M, N;
  Splits splits;
  int32_t mode;
  float scale;
};

// Sums of the splits, scaled; four columns a thread, and with kBy > 1 every
// kBy-th split a thread, joined in a fixed order.
template <int kBy>
__device__ __forceinline__ void finish_block(const FinishParams& p, const int64_t block) {
  __shared__ float4 part[kBy][256 / kBy];
  const int64_t rows = p.list ? (int64_t)p.header->live : p.M, quads = p.N / 4;
  const int parts = rows > 0 ? p.splits.parts(rows) : 1;
  if (rows == 0 || (parts == 1 && !p.splits.always)) return;   // the product wrote the result
  const int t = threadIdx.x % (256 / kBy), by = threadIdx.x / (256 / kBy);
  const int64_t at = block * (256 / kBy) + t, row = at / quads, col = 4 * (at - row * quads);
  float4 v = make_float4(0, 0, 0, 0);
  if (row < rows) {
    const float* src = p.partial + row * p.N + col;
#pragma unroll 8
    for (int s = by; s < parts; s += kBy) {
      const float4 o = *reinterpret_cast<const float4*>(src + s * rows * p.N);
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
  }
  if constexpr (kBy > 1) {
    part[by][t] = v;
    __syncthreads();
    if (by > 0) return;
#pragma unroll
    for (int s = 1; s < kBy; ++s) {
      const float4 o = part[s][t];
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
  }
  if (row >= rows) return;
  const float scale = p.scale * p.header->d_max;
  v.x *= scale, v.y *= scale, v.z *= scale, v.w *= scale;
  const int64_t to = (p.list ? (int64_t)p.list[row] : row) * p.N + col;
  if (p.mode == kBF16) {
    *reinterpret_cast<uint2*>((uint16_t*)p.out + to) = make_uint2(bf16_pack2(v.x, v.y), bf16_pack2(v.z, v.w));
  } else {
    float4* dst = reinterpret_cast<float4*>((float*)p.out + to);
    if (p.mode == kF32Add) {
      const float4 o = *dst;
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    *dst = v;
  }
}

template <int kBy>
__global__ __launch_bounds__(256) void finish_kernel(const FinishParams p) {
  finish_block<kBy>(p, blockIdx.x);
}

// g^T x of one or two steps: a tile is its first loads and its stores.  With up
// to 2048 columns small tiles, two blocks to a compute unit, so that one's run
// beside the other's (gradients of 61 x 32000 x 1024: 65.2 us, 66.5 in whole
// tiles; of 128 x 50001 x 2048 187.5 and 189.1); rows of more columns are
// written faster in whole ones' longer pieces (64 x 32000 x 4096: 219.6 small,
// 213.9 whole), and more steps go faster there (200 x 32000 x 2048, four steps:
// 165.4 and 159.5).
//
// The blocks ahead of the tiles', if there are any, finish dx (f): neither reads
// what the other writes, and dx's needs no launch of its own (61 x 32000 x 1024:
// 64.4 us with one, 63.1 with the blocks behind the tiles', 61.7 so).
__global__ __launch_bounds__(Small::kThreads) void product_small_kernel(const ProductParams p, const FinishParams f) {
  static_assert(Small::kThreads == 256, "of a block that finishes too");
  const uint32_t n_tiles = (uint32_t)((p.N + Small::kBN - 1) / Small::kBN), m_tiles = (uint32_t)((p.M + Small::kBM - 1) / Small::kBM);
  const uint32_t ahead = gridDim.x - m_tiles * n_tiles;
  if (blockIdx.x < ahead) {
    finish_block<8>(f, blockIdx.x);
    return;
  }
  uint32_t tm, tn;
  tile_at(xcd_contiguous32(blockIdx.x - ahead, m_tiles * n_tiles), m_tiles, n_tiles, tm, tn);
  product_tile<Small, true>(p, p.header->live, (int64_t)tm * Small::kBM, (int64_t)tn * Small::kBN, 0, 1);
}

// No rows: a gradient of zeros.
__global__ __launch_bounds__(256) void zero_kernel(uint8_t* p, int64_t bytes) {
  for (int64_t at = 16 * ((int64_t)blockIdx.x * 256 + threadIdx.x); at < bytes; at += 4096 * (int64_t)gridDim.x)
    *reinterpret_cast<uint4*>(p + at) = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ host

constexpr int64_t kMaxRows = 1 << 23, kMaxVocab = 1 << 22, kMaxCols = 1 << 16;   // (a launch has less than 2^32 threads)
int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return up(a, b) * b; }

// Cuts a workspace into arrays at multiples of 256 bytes; without a base it
// counts them.
struct Cutter {
  uint8_t* base;
  int64_t used = 0;
  template <class P>
  P* take(int64_t bytes) {
    P* p = base ? reinterpret_cast<P*>(base + used) : nullptr;
    used += round_up(bytes, 256);
    return p;
  }
};

// The logits' tiles.  Where whole ones are few, most of the device is idle and
// each waits for its loads: up to an eighth of the compute units thin ones are
// faster (155 rows x 3070 x 4288: 24 us, 47 in small and 60 in whole tiles;
// with 64 whole tiles, 1000 x 4000 x 2048, 34, 32 and 36), up to a half small
// ones (129 x 32000 x 4096, 125 whole tiles: 82 us against 90; 144 of them,
// 1500 x 6000 x 4096: 99 against 82).
enum Tiles { kThinTiles, kSmallTiles, kLargeTiles };

Tiles tiles_for(int64_t M, int64_t N) {
  const int64_t large = up(M, Large::kBM) * up(N, Large::kBN);
  if (M <= kThinRows || large <= kUnits / 8) return kThinTiles;
  return M <= kFewRows || large <= kUnits / 2 ? kSmallTiles : kLargeTiles;
}

struct LossSpace {
  Header* header;
  int32_t *list, *place, *target;
  float* at_target;
  float2* part;
  int64_t strip_step, row_step, bytes;
  int32_t strips;
};

// Rows of x that the forward pass takes at a time: offsets into them have 32 bits.
int64_t loss_rows(int64_t M, int64_t K) {
  const int64_t most = ((int64_t)0xFFFFFFFF / (2 * K)) / 256 * 256;
  return M < most ? M : most;
}

LossSpace loss_space(void* base, int64_t M, int64_t V) {
  Cutter c{(uint8_t*)base};
  LossSpace s;
  memset(&s, 0, sizeof(s));
  const bool few = M <= kFewRows;
  const Tiles tiles = tiles_for(M, V);
  s.at_target = c.take<float>(4 * M);
  if (!few) {
    s.header = c.take<Header>(sizeof(Header));
    s.list = c.take<int32_t>(4 * M);
    s.place = c.take<int32_t>(4 * M);
    s.target = c.take<int32_t>(4 * M);
  }
  s.strips = (int32_t)(tiles == kThinTiles    ? up(V, kThinCols) * (kThinCols / kThinStrip)
                       : tiles == kSmallTiles ? up(V, kStrip)
                                              : up(V, Large::kBN) * (Large::kBN / kStrip));
  s.row_step = few ? s.strips : 1;
  s.strip_step = few ? 1 : round_up(M, 16);
  s.part = c.take<float2>(8 * (few ? M : s.strip_step) * s.strips);
  s.bytes = c.used;
  return s;
}

// Splits of a product of up to `rows` rows and `cols` columns over `steps`.
// room: rows that the parts of any number of rows take at most.
Splits splits_for(int64_t rows, int64_t cols, int64_t steps, bool always, bool thin) {
  Splits s;
  s.tile_rows = thin ? (int32_t)kThinRows : Large::kBM;
  s.n_tiles = (int32_t)up(cols, thin ? ThinDx::kBN : Large::kBN);
  s.blocks = (int32_t)(thin ? 2 * kUnits : kUnits);
  const int64_t by_steps = steps / 8, by_tiles = s.blocks / s.n_tiles;
  s.most = (int32_t)(by_steps < by_tiles ? by_steps : by_tiles);
  s.always = always;
  s.room = 0;
  if (s.most > 1 && up(rows, s.tile_rows) * s.n_tiles <= s.blocks) {
    const int64_t all = (int64_t)s.tile_rows * s.blocks / s.n_tiles;
    s.room = s.most * rows < all ? s.most * rows : all;
  }
  if (always && s.room < rows) s.room = rows;
  return s;
}

struct GradSpace {
  Header* header;
  int32_t *list, *place;
  RowInfo* info;
  uint16_t* x_bf16;
  uint8_t* x_codes;
  uint16_t *g, *w_bf16;
  float *dx_sum, *dw_sum;
  int64_t pieces, piece, bytes;   // piece: vocabulary rows, a multiple of 256
  Splits dx_splits, dw_splits;
};

struct GradShape {
  int64_t M, V, K;
  bool fp8, dx, dw, f32;
};

GradSpace grad_space_of(void* base, const GradShape& h, int64_t pieces) {
  Cutter c{(uint8_t*)base};
  GradSpace s;
  memset(&s, 0, sizeof(s));
  s.piece = round_up(up(h.V, pieces), 256);
  s.pieces = up(h.V, s.piece);
  const int64_t rows = round_up(h.M, 64), p = s.piece;
  const bool thin = h.M <= kThinRows, two = thin || h.f32;   // two: g in two parts
  s.dx_splits = splits_for(h.M, h.K, p / 64, s.pieces > 1, thin);
  s.dw_splits = splits_for(p, h.K, (two ? 2 : 1) * rows / 64, false, false);
  s.header = c.take<Header>(sizeof(Header));
  s.list = c.take<int32_t>(4 * h.M);
  s.place = c.take<int32_t>(4 * h.M);
  s.info = c.take<RowInfo>(sizeof(RowInfo) * h.M);
  if (!h.fp8 || h.dw) s.x_bf16 = c.take<uint16_t>(2 * h.M * h.K);
  if (h.fp8) s.x_codes = c.take<uint8_t>(h.M * h.K);
  s.g = c.take<uint16_t>((two ? 4 : 2) * rows * p);
  if (h.fp8 && h.dx) s.w_bf16 = c.take<uint16_t>(2 * p * h.K);
  const int64_t dx_room = h.dx ? s.dx_splits.room : 0, dw_room = h.dw ? s.dw_splits.room : 0;
  if (s.pieces == 1) {   // dx is done before dw begins: one array for both
    float* sums = c.take<float>(4 * (dx_room > dw_room ? dx_room : dw_room) * h.K);
    s.dx_sum = dx_room > 0 ? sums : nullptr;
    s.dw_sum = dw_room > 0 ? sums : nullptr;
  } else {
    if (dx_room > 0) s.dx_sum = c.take<float>(4 * dx_room * h.K);
    if (dw_room > 0) s.dw_sum = c.take<float>(4 * dw_room * h.K);
  }
  s.bytes = c.used;
  return s;
}

// The next number of pieces that makes them smaller than those of s, past
// 256-row ones more than there are.
int64_t next_pieces(const GradShape& h, const GradSpace& s) {
  return s.piece > 256 ? up(h.V, s.piece - 256) : up(h.V, 256) + 1;
}

// The space of as few pieces as `bytes` hold; pieces 0 if none fit.
GradSpace grad_space(void* base, int64_t bytes, const GradShape& h) {
  const int64_t most = up(h.V, 256);
  GradSpace s;
  for (int64_t n = 1; n <= most; n = next_pieces(h, s)) {
    s = grad_space_of(base, h, n);
    if (s.bytes <= bytes) return s;
  }
  s.pieces = 0;
  return s;
}

// The least space that `most` pieces or fewer take.  (Fewer may take less: one
// piece has no sums of dx to keep, and splits of dw go by a piece's tiles.)
int64_t least_space(const GradShape& h, int64_t most) {
  GradSpace s = grad_space_of(nullptr, h, 1);
  int64_t least = s.bytes;
  for (int64_t n = next_pieces(h, s); n <= most; n = next_pieces(h, s)) {
    s = grad_space_of(nullptr, h, n);
    if (s.bytes < least) least = s.bytes;
  }
  return least;
}

bool loss_sizes_ok(int64_t M, int64_t V, int64_t K, bool fp8) {
  return M >= 0 && M <= kMaxRows && V >= 0 && V <= kMaxVocab && K >= 0 && K <= kMaxCols && K % (fp8 ? 128 : 64) == 0 &&
         M * K <= (int64_t)1 << 33 && V * K <= (int64_t)1 << 34 && up(M, Large::kBM) * up(V, Large::kBN) <= (int64_t)1 << 22;
}

bool scale_ok(float s) { return s >= FLT_MIN && s <= FLT_MAX; }

// Products of scales, rounded once.
float times(float a, float b, float c = 1.0f) { return (float)((double)a * b * c); }

// What the forward and the backward call check alike.
template <class Args>
coat_status_t check_common(const Args* a, bool& fp8) {
  fp8 = a->x_codes || a->weight_codes;
  if (!loss_sizes_ok(a->rows, a->vocab, a->cols, fp8)) return COAT_ERR_INVALID_VALUE;
  if (fp8 && (a->x || a->weight)) return COAT_ERR_INVALID_VALUE;
  if (!scale_ok(a->x_scale) || !scale_ok(a->weight_scale) || !scale_ok(a->logit_scale) ||
      !scale_ok(times(a->x_scale, a->weight_scale, a->logit_scale)) || !scale_ok(times(a->x_scale, a->logit_scale)) ||
      !scale_ok(times(a->weight_scale, a->logit_scale)) ||
      !scale_ok(times(a->x_scale, a->weight_scale, a->logit_scale) * kLog2e) || !(fabsf(a->z_loss) <= FLT_MAX))
    return COAT_ERR_INVALID_VALUE;
  return COAT_OK;
}

template <class Args>
bool operands_missing(const Args* a, bool fp8) {
  return fp8 ? !a->x_codes || !a->weight_codes : !a->x || !a->weight;
}

hipError_t launch(const void* fn, int64_t blocks, int threads, void* params, hipStream_t stream) {
  void* args[] = {params};
  return hipLaunchKernel(fn, dim3((unsigned)blocks), dim3((unsigned)threads), args, 0, stream);
}

template <bool kGrad>
hipError_t launch_logits(LogitParams& p, bool fp8, hipStream_t stream) {
  const Tiles tiles = tiles_for(p.M, p.N);
  if (tiles == kThinTiles) {
    // (g has 64 rows for the products at least)
    constexpr int kLeast = kGrad ? 2 : 1;
    const void* fns[] = {reinterpret_cast<const void*>(&logit_thin_kernel<false, kGrad, kLeast>),
                         reinterpret_cast<const void*>(&logit_thin_kernel<false, kGrad, 2>),
                         reinterpret_cast<const void*>(&logit_thin_kernel<true, kGrad, kLeast>),
                         reinterpret_cast<const void*>(&logit_thin_kernel<true, kGrad, 2>)};
    p.n_tiles = (int32_t)up(p.N, kThinCols);
    return launch(fns[2 * fp8 + (p.M > 32)], up(p.M, kThinRows) * p.n_tiles, 128, &p, stream);
  }
  if (tiles == kSmallTiles) {
    const void* fn = fp8 ? reinterpret_cast<const void*>(&logit_small_kernel<true, kGrad>)
                         : reinterpret_cast<const void*>(&logit_small_kernel<false, kGrad>);
    p.n_tiles = (int32_t)up(p.N, Small::kBN);
    return launch(fn, up(p.M, Small::kBM) * p.n_tiles, Small::kThreads, &p, stream);
  }
  const void* fn = fp8 ? reinterpret_cast<const void*>(&logit_large_kernel<true, kGrad>)
                       : reinterpret_cast<const void*>(&logit_large_kernel<false, kGrad>);
  p.n_tiles = (int32_t)up(p.N, Large::kBN);
  return launch(fn, up(p.M, Large::kBM) * p.n_tiles + kUnits / 2, Large::kThreads, &p, stream);
}

// Whether g^T x takes small tiles; two: g in two parts.
bool small_product(const Splits& s, int64_t cols, int64_t rows, bool two) {
  return s.room == 0 && cols <= kSmallCols && up(rows, 64) * (two ? 2 : 1) <= kSmallSteps;
}

int64_t few_finish_blocks(const FinishParams& p) { return up(p.M * (p.N / 4), 32); }

// f: dx to be finished beside a product of small tiles, or NULL.
hipError_t launch_product(ProductParams& p, bool gt, int64_t rows, hipStream_t stream, FinishParams* f = nullptr) {
  if (!gt && rows <= kThinRows)
    return launch(reinterpret_cast<const void*>(&product_thin_kernel),
                  (int64_t)p.splits.n_tiles * (p.splits.most > 1 ? p.splits.most : 1), ThinDx::kThreads, &p, stream);
  if (gt && small_product(p.splits, p.N, rows, p.a_rest)) {
    FinishParams none;
    memset(&none, 0, sizeof(none));
    void* args[] = {&p, f ? f : &none};
    const int64_t blocks = up(p.M, Small::kBM) * up(p.N, Small::kBN) + (f ? few_finish_blocks(*f) : 0);
    return hipLaunchKernel(reinterpret_cast<const void*>(&product_small_kernel), dim3((unsigned)blocks),
                           dim3((unsigned)Small::kThreads), args, 0, stream);
  }
  p.n_tiles = (uint32_t)up(p.N, Large::kBN);
  // (parts times tiles are at most kUnits)
  const int64_t tiles = up(p.M, Large::kBM) * p.n_tiles + kUnits / 2;
  const void* fn = gt ? reinterpret_cast<const void*>(&product_kernel<true>) : reinterpret_cast<const void*>(&product_kernel<false>);
  return launch(fn, tiles > kUnits ? tiles : kUnits, Large::kThreads, &p, stream);
}

// rows: at most.
hipError_t launch_finish(FinishParams& p, int64_t rows, hipStream_t stream) {
  if (rows <= kThinRows)
    return launch(reinterpret_cast<const void*>(&finish_kernel<8>), few_finish_blocks(p), 256, &p, stream);
  return launch(reinterpret_cast<const void*>(&finish_kernel<1>), up(rows * (p.N / 4), 256), 256, &p, stream);
}

}  // namespace

extern "C" {

int64_t coat_fp8_cross_entropy_workspace(int64_t rows, int64_t vocab, int64_t cols) {
  if (!loss_sizes_ok(rows, vocab, cols, false)) return -1;
  return rows == 0 || vocab == 0 || cols == 0 ? 0 : loss_space(nullptr, loss_rows(rows, cols), vocab).bytes;
}

coat_status_t coat_fp8_cross_entropy(const coat_cross_entropy_args_t* a, hipStream_t stream) {
  if (!a) return COAT_ERR_NULL_POINTER;
  bool fp8;
  const coat_status_t st = check_common(a, fp8);
  if (st != COAT_OK) return st;
  const int64_t M = a->rows, V = a->vocab, K = a->cols;
  if (M == 0) return COAT_OK;
  if (V == 0 || K == 0) return COAT_ERR_INVALID_VALUE;
  if (operands_missing(a, fp8) || !a->targets || !a->loss || !a->workspace) return COAT_ERR_NULL_POINTER;
  const uint8_t* x = fp8 ? a->x_codes : (const uint8_t*)a->x;
  const uint8_t* w = fp8 ? a->weight_codes : (const uint8_t*)a->weight;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(a->targets, 8) || !aligned(a->loss, 4) || !aligned(a->lse, 4) ||
      !aligned(a->workspace, 16))
    return COAT_ERR_MISALIGNED;
  const int64_t each = loss_rows(M, K);
  if (a->workspace_bytes < loss_space(nullptr, each, V).bytes) return COAT_ERR_INVALID_VALUE;
  hipError_t e = hipSuccess;
  for (int64_t m0 = 0; m0 < M && e == hipSuccess; m0 += each) {
    const int64_t rows = M - m0 < each ? M - m0 : each;
    const LossSpace s = loss_space(a->workspace, rows, V);
    LogitParams p;
    memset(&p, 0, sizeof(p));
    p.stride = (uint32_t)(fp8 ? K : 2 * K);
    p.x = x + m0 * p.stride;
    p.w = w;
    p.M = rows;
    p.N = p.V = V;
    p.steps = (int32_t)(p.stride / 128);
    p.scale2 = times(a->x_scale, a->weight_scale, a->logit_scale) * kLog2e;
    p.part = s.part;
    p.at_target = s.at_target;
    p.targets = a->targets + m0;
    p.target = s.target;
    p.list = s.list;
    p.header = s.header;
    p.strip_step = s.strip_step;
    p.row_step = s.row_step;
    if (s.list) {
      PrepParams q;
      memset(&q, 0, sizeof(q));
      q.targets = p.targets;
      q.header = s.header;
      q.list = s.list;
      q.place = s.place;
      q.target = s.target;
      q.M = rows;
      q.V = V;
      e = launch(reinterpret_cast<const void*>(&prep_kernel), 1, 1024, &q, stream);
    }
    if (e == hipSuccess) e = launch_logits<false>(p, fp8, stream);
    if (e == hipSuccess) {
      JoinParams j;
      memset(&j, 0, sizeof(j));
      j.part = s.part;
      j.at_target = s.at_target;
      j.place = s.place;
      j.targets = p.targets;
      j.loss = a->loss + m0;
      j.lse = a->lse ? a->lse + m0 : nullptr;
      j.M = rows;
      j.V = V;
      j.strip_step = s.strip_step;
      j.row_step = s.row_step;
      j.strips = s.strips;
      j.z = a->z_loss;
      if (fp8) j.dot = TargetDot{p.x, w, K, p.scale2};
      if (fp8 && s.list) e = launch(reinterpret_cast<const void*>(&target_kernel), up(rows, 4), 256, &j, stream);
      if (e == hipSuccess)
        e = s.list ? launch(reinterpret_cast<const void*>(&loss_join_kernel), up(rows, 16), 256, &j, stream)
                   : launch(reinterpret_cast<const void*>(&loss_join_few_kernel), rows, 64, &j, stream);
    }
  }
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

int64_t coat_fp8_cross_entropy_bwd_workspace(int64_t rows, int64_t vocab, int64_t cols, int64_t piece,
                                             int32_t codes, int32_t f32) {
  if (!loss_sizes_ok(rows, vocab, cols, codes != 0) || piece < 1) return -1;
  if (rows == 0 || vocab == 0 || cols == 0) return 0;
  const GradShape h = {rows, vocab, cols, codes != 0, true, true, f32 != 0};
  return least_space(h, up(vocab, piece < vocab ? round_up(piece, 256) : vocab));
}

coat_status_t coat_fp8_cross_entropy_bwd(const coat_cross_entropy_bwd_args_t* a, hipStream_t stream) {
  if (!a) return COAT_ERR_NULL_POINTER;
  bool fp8;
  const coat_status_t st = check_common(a, fp8);
  if (st != COAT_OK) return st;
  if (a->dw_bf16 && (a->dw_f32 || a->accumulate)) return COAT_ERR_INVALID_VALUE;
  const int64_t M = a->rows, V = a->vocab, K = a->cols;
  if (V == 0 || K == 0) return M == 0 ? COAT_OK : COAT_ERR_INVALID_VALUE;
  const bool dw = a->dw_bf16 || a->dw_f32;
  if (!dw && !a->dx) return M == 0 ? COAT_OK : COAT_ERR_NULL_POINTER;
  if (M > 0 && (operands_missing(a, fp8) || !a->targets || !a->lse || !a->d_loss)) return COAT_ERR_NULL_POINTER;
  if (M > 0 && !a->workspace) return COAT_ERR_NULL_POINTER;
  const uint8_t* x = fp8 ? a->x_codes : (const uint8_t*)a->x;
  const uint8_t* w = fp8 ? a->weight_codes : (const uint8_t*)a->weight;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(a->targets, 8) || !aligned(a->lse, 4) || !aligned(a->d_loss, 4) ||
      !aligned(a->dx, 16) || !aligned(a->dw_bf16, 16) || !aligned(a->dw_f32, 16) || !aligned(a->workspace, 16))
    return COAT_ERR_MISALIGNED;
  if (M == 0) {
    if (!dw || a->accumulate) return COAT_OK;
    uint8_t* dst = a->dw_bf16 ? (uint8_t*)a->dw_bf16 : (uint8_t*)a->dw_f32;
    int64_t bytes = V * K * (a->dw_bf16 ? 2 : 4);
    const int64_t blocks = up(bytes, 4096);
    void* args[] = {&dst, &bytes};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&zero_kernel),
                                         dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), args, 0, stream);
    return e == hipSuccess ? COAT_OK : hip_fail(e);
  }
  const GradShape h = {M, V, K, fp8, a->dx != nullptr, dw, a->dw_f32 != nullptr};
  const GradSpace s = grad_space(a->workspace, a->workspace_bytes, h);
  if (s.pieces == 0) return COAT_ERR_INVALID_VALUE;

  PrepParams q;
  memset(&q, 0, sizeof(q));
  q.targets = a->targets;
  q.d_loss = a->d_loss;
  q.lse = a->lse;
  q.header = s.header;
  q.list = s.list;
  q.place = s.place;
  q.info = s.info;
  q.M = M;
  q.V = V;
  q.z = a->z_loss;
  GatherParams g;
  memset(&g, 0, sizeof(g));
  g.x = x;
  g.x_bf16 = s.x_bf16;
  g.x_codes = s.x_codes;
  g.dx = a->dx;
  g.K = K;
  g.fp8 = fp8;
  const float scale = times(a->x_scale, a->weight_scale, a->logit_scale);
  if (fp8) g.dot = TargetDot{x, w, K, scale * kLog2e};
  void* both[] = {&q, &g};
  hipError_t e = hipSuccess;
  if (M > kThinRows) e = launch(reinterpret_cast<const void*>(&prep_kernel), 1, 1024, &q, stream);
  if (e == hipSuccess)
    e = hipLaunchKernel(M > kThinRows ? reinterpret_cast<const void*>(&gather_kernel)
                                      : reinterpret_cast<const void*>(&prep_few_kernel),
                        dim3((unsigned)M), dim3(256), both, 0, stream);
  const bool thin = M <= kThinRows, two = thin || h.f32;
  for (int64_t n = 0; n < s.pieces && e == hipSuccess; ++n) {
    const int64_t v0 = n * s.piece, rows = V - v0 < s.piece ? V - v0 : s.piece, ld = round_up(rows, 64);
    const uint8_t* wp = w + v0 * K * (fp8 ? 1 : 2);
    {
      LogitParams p;
      memset(&p, 0, sizeof(p));
      p.x = fp8 ? s.x_codes : (const uint8_t*)s.x_bf16;
      p.w = wp;
      p.header = s.header;
      p.M = M;
      p.N = rows;
      p.V = V;
      p.stride = (uint32_t)(fp8 ? K : 2 * K);
      p.steps = (int32_t)(p.stride / 128);
      p.scale2 = scale * kLog2e;
      p.ld = ld;
      p.info = s.info;
      p.g = s.g;
      p.g_rest = two ? s.g + round_up(M, 64) * ld : nullptr;
      p.v0 = (int32_t)v0;
      e = launch_logits<true>(p, fp8, stream);
    }
    FinishParams f;        // dx's
    memset(&f, 0, sizeof(f));
    bool beside = false;   // finished beside dW's product
    if (e == hipSuccess && a->dx) {
      if (fp8) {
        const int64_t chunks = rows * K / 8;
        void* args[] = {(void*)&wp, (void*)&chunks, (void*)&s.w_bf16};
        e = hipLaunchKernel(reinterpret_cast<const void*>(&expand_kernel), dim3((unsigned)up(chunks, 256)), dim3(256), args,
                            0, stream);
      }
      ProductParams p;
      memset(&p, 0, sizeof(p));
      p.a = (const uint8_t*)s.g;
      p.b = fp8 ? (const uint8_t*)s.w_bf16 : wp;
      p.header = s.header;
      p.list = s.list;
      p.out = a->dx;
      p.partial = s.dx_sum;
      p.M = M;
      p.N = K;
      p.lda = (uint32_t)(2 * ld);
      p.ldb = (uint32_t)(2 * K);
      p.k_rows = (int32_t)rows;
      p.splits = s.dx_splits;
      p.mode = kBF16;
      p.add = n > 0;
      p.scale = times(a->weight_scale, a->logit_scale);
      if (e == hipSuccess) e = launch_product(p, false, M, stream);
      if (e == hipSuccess && s.dx_sum && n == s.pieces - 1) {
        f.partial = s.dx_sum;
        f.header = s.header;
        f.list = s.list;
        f.out = a->dx;
        f.M = M;
        f.N = K;
        f.splits = s.dx_splits;
        f.mode = kBF16;
        f.scale = times(a->weight_scale, a->logit_scale);
        beside = M <= kThinRows && dw && small_product(s.dw_splits, K, M, two);
        if (!beside) e = launch_finish(f, M, stream);
      }
    }
    if (e == hipSuccess && dw) {
      const int out = a->dw_bf16 ? kBF16 : a->accumulate ? kF32Add : kF32;
      void* dst = a->dw_bf16 ? (void*)(a->dw_bf16 + v0 * K) : (void*)(a->dw_f32 + v0 * K);
      ProductParams p;
      memset(&p, 0, sizeof(p));
      p.a = (const uint8_t*)s.g;
      p.a_rest = two ? (const uint8_t*)(s.g + round_up(M, 64) * ld) : nullptr;
      p.b = (const uint8_t*)s.x_bf16;
      p.header = s.header;
      p.out = dst;
      p.partial = s.dw_sum;
      p.M = rows;
      p.N = K;
      p.lda = (uint32_t)(2 * ld);
      p.ldb = (uint32_t)(2 * K);
      p.splits = s.dw_splits;
      p.mode = out;
      p.scale = times(a->x_scale, a->logit_scale);
      e = launch_product(p, true, M, stream, beside ? &f : nullptr);
      if (e == hipSuccess && s.dw_sum) {
        FinishParams q;
        memset(&q, 0, sizeof(q));
        q.partial = s.dw_sum;
        q.header = s.header;
        q.out = dst;
        q.M = rows;
        q.N = K;
        q.splits = s.dw_splits;
        q.mode = out;
        q.scale = p.scale;
        e = launch_finish(q, rows, stream);
      }
    }
  }
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

}  // extern "C"
