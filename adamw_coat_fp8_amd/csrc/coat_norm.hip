// coat_norm.hip -- gfx950 kernels and C ABI of the RMS norm with an E4M3
// checkpoint of its input, and of its backward pass.
//
// Sources (see include/coat_fp8.h for the full citations):
//   [P1] COAT paper review (xllm-io.github.io), section 三: the input of a
//        non-linear layer is kept in E4M3 per 1xG group for the backward
//        pass (混合粒度激活量化); the input of a linear layer is E4M3 under
//        one scale per tensor; COAT LLaMA's BeforeAttention and MLPResidual
//        take the residual sum and the norm together.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "coat_elem.h"

using namespace coat;

namespace {

// ------------------------------------------------------------ forward
//
//   h = bf16(x + residual),  rstd = (mean(h^2) + eps)^-1/2,  y = h rstd w
//
// One block takes one row at a time and keeps it in registers: chunk i of
// thread t is the eight columns from 8 (t + blockDim i), so every byte is
// read and written once (past 16384 columns the row no longer fits, and is
// read again from the L2).  A block has as many waves as kC chunks a thread
// need for the row (kMost: the most threads of an instance).  The weight's chunks stay in registers over the
// rows of a block, and the next row is loaded before the current one is
// reduced.  The sum of squares is FP32: eight values of a lane in order,
// then lanes, then waves (LDS, two slots in turn, one barrier a row).  A
// checkpoint group lies on G/8 neighbouring lanes of one 16-lane DPP row.
//
// Bound by HBM: 8192 x 4096 with residual, E4M3 output and checkpoint (8.03
// bytes a value) takes 48.5 to 49.0 us, 5.5 TB/s, raising a maximum 0.7 more;
// vector instructions issue in 39% of the cycles.  A grid of one block a row,
// without the loads ahead, took 51.5.  4096 x 8192 5.7 TB/s, 2048 x 16384 5.5;
// past 16384 columns, where the chunks of a row spill from the registers (108
// bytes a lane), 3 TB/s (1000 x 32768: 85 us).

constexpr int64_t kMaxCols = 32768;

struct NormParams {
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* weight;
  uint16_t* sum;
  uint16_t* y;
  uint8_t* y_codes;
  float* y_amax;
  uint8_t* codes;
  float* scales;
  float* rstd;
  int64_t rows;
  int32_t cols;
  int32_t group_shift;   // log2(group_size)
  float eps, inv_y_scale, inv_cols;
};

// Element `col` of a row that starts at the uniform address `row`: a scalar
// base and a 32-bit offset, which takes one register a lane and not two for
// each array.
template <class V>
__device__ __forceinline__ V* at(V* row, int col) {
  return reinterpret_cast<V*>(reinterpret_cast<uintptr_t>(row) + (uint32_t)col * (uint32_t)sizeof(V));
}

// Chunks of a row that is read once, or twice (then the second time is from
// the L2).
template <bool kOnce>
__device__ __forceinline__ uint4 load_row16(const void* p) {
  return kOnce ? load_stream16(p) : *reinterpret_cast<const uint4*>(p);
}

template <bool kOnce>
__device__ __forceinline__ uint2 load_row8(const void* p) {
  return kOnce ? load_stream8(p) : *reinterpret_cast<const uint2*>(p);
}

// The block's sum of v (every thread gets it).  `slot` alternates between
// calls: a wave can be at most one barrier ahead of another.
template <int kMost>
__device__ __forceinline__ float block_sum(float v, int slot) {
  v = lanes_sum<64>(v);
  if constexpr (kMost > 64) {
    constexpr int kWaves = kMost / 64;
    __shared__ float part[2][kWaves];
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[slot][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += w < waves ? part[slot][w] : 0.0f;
  }
  return v;
}

// kRows: rows that a block takes at once, one wave each (they need no barrier).
template <int kMost, int kC, int kRows = 1>
__global__ __launch_bounds__(kMost * kRows) void rms_norm_kernel(const NormParams p) {
  static_assert(kRows == 1 || kMost == 64, "a row of one wave");
  const int t = kRows > 1 ? threadIdx.x & 63 : threadIdx.x, threads = kRows > 1 ? 64 : blockDim.x;
  const int cols = p.cols, lanes = 1 << (p.group_shift - 3);
  bool ok[kC];
  int col[kC];
  uint4 w[kC], next[kC], nres[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    col[i] = 8 * (t + threads * i);
    ok[i] = col[i] < cols;
    w[i] = next[i] = nres[i] = make_uint4(0, 0, 0, 0);
  }
  constexpr bool kKeep = kC <= 2;   // else each phase loads a chunk when it comes to it
  auto load = [&](int64_t row, int i) __attribute__((always_inline)) {
    if (!ok[i]) return;
    next[i] = load_row16<kKeep>(at(p.x + row * cols, col[i]));
    if (p.residual) nres[i] = load_row16<kKeep>(at(p.residual + row * cols, col[i]));
  };
  auto load_weight = [&](int i) __attribute__((always_inline)) {
    if (ok[i]) w[i] = *reinterpret_cast<const uint4*>(at(p.weight, col[i]));
  };
  // the chunk as everything but the sum reads it: as it is stored
  auto stored = [&](int i) __attribute__((always_inline)) {
    if (!p.residual) return next[i];
    float f[8], r[8];
    unpack8(next[i], f);
    unpack8(nres[i], r);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += r[e];
    return pack8(f);
  };
  const int64_t stride = (int64_t)gridDim.x * kRows;
  int64_t row = blockIdx.x;
  if constexpr (kRows > 1) row = row * kRows + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if (kKeep && (kRows == 1 || row < p.rows)) {
#pragma unroll
    for (int i = 0; i < kC; ++i) load(row, i), load_weight(i);
  }

  float top = 0.0f;
  int slot = 0;
  for (; row < p.rows; row += stride, slot ^= 1) {
    uint4 raw[kC];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float f[8];
      if (!kKeep) load(row, i);
      raw[i] = stored(i);
      unpack8(raw[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(f[e], f[e], ss);
    }
    if (kKeep && row + stride < p.rows) {
#pragma unroll
      for (int i = 0; i < kC; ++i) load(row + stride, i);
    }
    const float rstd = inv_sqrt(__builtin_fmaf(block_sum<kMost>(ss, slot), p.inv_cols, p.eps));
    if (p.rstd && t == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int64_t start = row * cols;
      if (!kKeep) {
        load(row, i), load_weight(i);
        raw[i] = stored(i);
      }
      if (p.codes) {   // all lanes: groups exchange their maxima
        float scale;
        const uint2 c = checkpoint8(raw[i], lanes, scale);
        if (ok[i]) {
          store_stream8(at(p.codes + start, col[i]), c);
          if (((t + threads * i) & (lanes - 1)) == 0)
            *at(p.scales + (start >> p.group_shift), col[i] >> p.group_shift) = scale;
        }
      }
      if (!ok[i]) continue;
      if (p.sum) store_stream16(at(p.sum + start, col[i]), raw[i]);
      float f[8], g[8];
      unpack8(raw[i], f);
      unpack8(w[i], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * g[e];
      if (p.y) store_stream16(at(p.y + start, col[i]), pack8(f));
      if (p.y_codes) {
        const float m = max_mag(f);
        top = fmaxf(top, m);
        uint32_t c[2];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= p.inv_y_scale;
        e4m3_pack(f, m * p.inv_y_scale, c);
        store_stream8(at(p.y_codes + start, col[i]), make_uint2(c[0], c[1]));
      }
    }
  }
  if (p.y_amax) raise_amax(p.y_amax, top);
}

// ----------------------------------------------------------- backward
//
// With n = code scale rstd (the normalised input as the checkpoint holds it)
// and dn = dy w:
//   dx = rstd (dn - n mean(dn n)) (+ d_residual),   dw = sum over rows of dy n
//
// The same layout; a block walks rows with a stride and adds dy n of its
// columns up in registers, in FP32, writing one row of partial sums at its
// end.  A second launch adds those up in a fixed order, so the result does
// not depend on timing.
//
// 8192 x 4096 with d_residual: 42.5 us (5.5 TB/s) and 4.5 for the second
// launch, most of it latency.  One row is in flight a unit, so shorter ones
// without d_residual reach less: 4097 x 5120 24.0 + 4.6 us, 4.5 TB/s.  Two rows
// at a time need twice the registers and took 62.8 us where one takes 45.8.
// Past 16384 columns the chunks of a row spill (368 bytes a lane), and each
// phase waits for its loads: 1000 x 32768 with d_residual 197 us, 1.2 TB/s.

struct NormBwdParams {
  const uint16_t* dy;
  const uint8_t* codes;
  const float* scales;
  const float* rstd;
  const uint16_t* weight;
  const uint16_t* d_residual;
  uint16_t* dx;
  float* partials;   // a row of cols for each block, or NULL
  float* dw;         // few rows: the weight gradient itself
  int64_t rows;
  int32_t cols;
  int32_t group_shift;
  int32_t accumulate;
  float inv_cols;
};

// Rows first, first + stride, ...
template <int kMost, int kC>
__device__ __forceinline__ void rms_norm_bwd_rows(const NormBwdParams& p, const int64_t first, const int64_t stride) {
  const int t = threadIdx.x, threads = blockDim.x;
  const int cols = p.cols;
  bool ok[kC];
  int col[kC];
  uint4 w[kC], dyn[kC], drn[kC];
  uint2 cn[kC];
  float sn[kC], rn = 0.0f, dw[kC][8];
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    col[i] = 8 * (t + threads * i);
    ok[i] = col[i] < cols;
    w[i] = dyn[i] = drn[i] = make_uint4(0, 0, 0, 0);
    cn[i] = make_uint2(0, 0);
    sn[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
  }
  constexpr bool kKeep = kC <= 2;   // else each phase loads a chunk when it comes to it
  auto load = [&](int64_t row, int i) __attribute__((always_inline)) {
    if (!ok[i]) return;
    const int64_t start = row * cols;
    dyn[i] = load_row16<kKeep>(at(p.dy + start, col[i]));
    cn[i] = load_row8<kKeep>(at(p.codes + start, col[i]));
    sn[i] = *at(p.scales + (start >> p.group_shift), col[i] >> p.group_shift);
  };
  auto load_residual = [&](int64_t row, int i) __attribute__((always_inline)) {
    if (ok[i] && p.d_residual) drn[i] = load_stream16(at(p.d_residual + row * cols, col[i]));
  };
  auto load_weight = [&](int i) __attribute__((always_inline)) {
    if (ok[i]) w[i] = *reinterpret_cast<const uint4*>(at(p.weight, col[i]));
  };
  int64_t row = first;
  rn = p.rstd[row];
  if (kKeep) {
#pragma unroll
    for (int i = 0; i < kC; ++i) load(row, i), load_residual(row, i), load_weight(i);
  }

  int slot = 0;
  for (; row < p.rows; row += stride, slot ^= 1) {
    // kept as they came: n and dn are formed twice, which costs less than the
    // registers to hold them
    uint4 dy[kC], dr[kC];
    uint2 code[kC];
    float scale[kC], dot = 0.0f;
    const float rstd = rn;
    auto terms = [&](int i, float (&d)[8], float (&n)[8]) __attribute__((always_inline)) {
      unpack8(dy[i], d);
      e4m3_values8(code[i], n);
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] *= scale[i];
    };
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      if (!kKeep) load(row, i), load_weight(i);
      dy[i] = dyn[i];
      dr[i] = drn[i];
      code[i] = cn[i];
      scale[i] = sn[i] * rstd;
      float d[8], n[8], g[8];
      terms(i, d, n);
      unpack8(w[i], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dyn_e = d[e] * n[e];
        dw[i][e] += dyn_e;
        dot = __builtin_fmaf(dyn_e, g[e], dot);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (row + stride < p.rows) {
      rn = p.rstd[row + stride];
      if (kKeep) {
#pragma unroll
        for (int i = 0; i < kC; ++i) load(row + stride, i), load_residual(row + stride, i);
      }
    }
    const float mean = block_sum<kMost>(dot, slot) * p.inv_cols;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      if (!ok[i]) continue;
      if (kKeep) {
        // (opaque, or the compiler keeps the expanded values after all)
        asm volatile("" : "+v"(dy[i].x), "+v"(dy[i].y), "+v"(dy[i].z), "+v"(dy[i].w), "+v"(code[i].x), "+v"(code[i].y));
        asm volatile("" : "+v"(w[i].x), "+v"(w[i].y), "+v"(w[i].z), "+v"(w[i].w));
      } else {
        load(row, i), load_residual(row, i), load_weight(i);
        dy[i] = dyn[i], dr[i] = drn[i], code[i] = cn[i], scale[i] = sn[i] * rstd;
      }
      float d[8], n[8], g[8];
      terms(i, d, n);
      unpack8(w[i], g);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = rstd * __builtin_fmaf(-n[e], mean, d[e] * g[e]);
      if (p.d_residual) {
        unpack8(dr[i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] += g[e];
      }
      store_stream16(at(p.dx + row * cols, col[i]), pack8(d));
    }
  }
  if (p.partials) {
    float* out = p.partials + (int64_t)blockIdx.x * cols;
#pragma unroll
    for (int i = 0; i < kC; ++i)
      if (ok[i]) {
        *reinterpret_cast<float4*>(out + col[i]) = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
        *reinterpret_cast<float4*>(out + col[i] + 4) = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
      }
  }
}

template <int kMost, int kC>
__global__ __launch_bounds__(kMost) void rms_norm_bwd_kernel(const NormBwdParams p) {
  rms_norm_bwd_rows<kMost, kC>(p, blockIdx.x, gridDim.x);
}

// Few rows: one launch and no partial sums.  Blocks 0 .. rows - 1 take a row
// each; every block behind them takes the weight gradient of 128 columns: 16
// threads of eight columns, blockDim / 16 slices of the rows, which join in
// the LDS in a fixed order.  The rows are read a second time, on other XCDs
// than the first for the most part, so from behind the L2s; and by blocks that
// may run before or after the row's own, so dx must not be dy.  A call this
// small is as long as its launches: 1 to 512 rows of 4096 take 7.7 us, with two
// launches 10.7.  At more than about 32 rows a slice the second reading shows
// (256 x 512, 64 rows a slice: 13.2 us against 11.0).  (The workspace is asked
// for all the same: its size is one function of the rows and columns.)
constexpr int kFewCols = 128;
constexpr int64_t kFewRows = 512;

bool few_rows(int64_t rows, int threads) { return rows <= kFewRows && rows <= 2 * threads; }

template <int kMost, int kC>
__global__ __launch_bounds__(kMost) void rms_norm_bwd_few_kernel(const NormBwdParams p) {
  if (blockIdx.x < p.rows) {
    rms_norm_bwd_rows<kMost, kC>(p, blockIdx.x, p.rows);
    return;
  }
  __shared__ float part[kMost / 16][kFewCols + 4];
  const int c = threadIdx.x & 15, slice = threadIdx.x >> 4, slices = blockDim.x >> 4;
  const int col = (int)(blockIdx.x - p.rows) * kFewCols + 8 * c;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
  if (col < p.cols) {
#pragma unroll 4
    for (int64_t row = slice; row < p.rows; row += slices) {
      const int64_t from = row * p.cols + col;
      const uint4 dy = *reinterpret_cast<const uint4*>(p.dy + from);
      const uint2 code = *reinterpret_cast<const uint2*>(p.codes + from);
      const float scale = p.scales[from >> p.group_shift] * p.rstd[row];
      float d[8], n[8];
      unpack8(dy, d);
      e4m3_values8(code, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = __builtin_fmaf(d[e], n[e] * scale, sum[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) part[slice][8 * c + e] = sum[e];
  __syncthreads();
  for (int n = kMost / 32; n > 0; n /= 2) {
    if (slice < n && slice + n < slices) {
#pragma unroll
      for (int e = 0; e < 8; ++e) part[slice][8 * c + e] += part[slice + n][8 * c + e];
    }
    __syncthreads();
  }
  if (slice == 0 && col < p.cols) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = part[0][8 * c + e];
      p.dw[col + e] = p.accumulate ? p.dw[col + e] + v : v;
    }
  }
}

// Sums `parts` rows of partial sums by column: a block takes 16 columns (64
// bytes of a row), its 64 slices add every 64th row, and the slices join in
// the LDS in a fixed order.
constexpr int kSumCols = 16, kSumSlices = 64;

__global__ __launch_bounds__(kSumCols* kSumSlices) void sum_partials_kernel(const float* partials, int parts,
                                                                          int64_t cols, float* dst0, int64_t split,
                                                                          float* dst1, int accumulate) {
  __shared__ float part[kSumSlices][kSumCols + 1];
  const int c = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
  const int64_t col = (int64_t)blockIdx.x * kSumCols + c;
  float v = 0.0f;
  if (col < cols) {
    // eight rows' loads in flight at a time
    for (int r = slice; r < parts; r += 8 * kSumSlices) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = r + i * kSumSlices;
        x[i] = at < parts ? partials[at * cols + col] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v += x[i];
    }
  }
  part[slice][c] = v;
  __syncthreads();
#pragma unroll
  for (int n = kSumSlices / 2; n > 0; n /= 2) {
    if (slice < n) part[slice][c] += part[slice + n][c];
    __syncthreads();
  }
  if (slice == 0 && col < cols) {
    float* dst = col < split ? dst0 + col : dst1 + (col - split);
    *dst = accumulate ? *dst + part[0][c] : part[0][c];
  }
}

// Blocks for rows, at most `most`, that all take as many rows as the busiest.
int64_t balanced(int64_t rows, int64_t most) {
  if (rows <= most) return rows;
  const int64_t each = (rows + most - 1) / most;
  return (rows + each - 1) / each;
}

// The instance for a row, and its threads: whole waves, as few as hold the
// row.  One chunk a thread up to 8192 columns: as many bytes in flight from
// twice the waves, which hide more of each other (backward, 4097 x 5120, one
// block a unit: 34 us with two chunks and five waves, 28 with one and ten).
// Only the forward pass of 2049 to 4096 columns is better with two chunks, in
// half the waves, of which a CU then holds more rows: 8192 rows with residual,
// checkpoint and E4M3 output 28.3 us against 32.9 at 2176 columns, 32.2 : 36.1
// at 2560, 35.4 : 39.4 at 2816, 39.5 : 44.7 at 3328, 42.0 : 47.1 at 3584,
// 48.3 : 49.4 at 4096; 1024 rows 5.5 : 5.2, 5.7 : 5.3, 5.8 : 6.9, 6.1 : 7.4,
// 6.2 : 8.0, 7.2 : 7.4; one row 3.1 : 2.9 throughout.
struct NormShape {
  int most, chunks, threads;
};

NormShape norm_shape(int64_t cols, bool backward) {
  NormShape s = cols <= 512     ? NormShape{64, 1, 0}
                : cols <= 2048  ? NormShape{256, 1, 0}
                : cols <= 4096 && !backward ? NormShape{256, 2, 0}
                : cols <= 8192  ? NormShape{1024, 1, 0}
                : cols <= 16384 ? NormShape{1024, 2, 0}
                                : NormShape{1024, 4, 0};
  s.threads = (int)((cols / 8 + 64 * s.chunks - 1) / (64 * s.chunks)) * 64;
  return s;
}

enum NormKernel { kForward, kBackward, kBackwardFew };

// Rows of one wave with a maximum to raise: four to a block where there are
// many, a quarter of the atomics (16384 x 512: 10.0 us against 13.4, 300 x 256: 4.0
// against 5.6; up to 128 blocks, or without a maximum, one to a block is 0.2
// to 0.4 us better).
constexpr int kWaveRows = 4;

const void* norm_kernel_for(NormShape s, NormKernel which) {
#define COAT_NORM(T, C)                                                                       \
  if (s.most == T && s.chunks == C)                                                           \
    return which == kForward    ? reinterpret_cast<const void*>(&rms_norm_kernel<T, C>)       \
           : which == kBackward ? reinterpret_cast<const void*>(&rms_norm_bwd_kernel<T, C>)   \
                                : reinterpret_cast<const void*>(&rms_norm_bwd_few_kernel<T, C>);
  COAT_NORM(64, 1)
  COAT_NORM(256, 1)
  COAT_NORM(1024, 1)
  COAT_NORM(1024, 2)
  COAT_NORM(1024, 4)
#undef COAT_NORM
  if (which == kForward && s.most == 256 && s.chunks == 2) return reinterpret_cast<const void*>(&rms_norm_kernel<256, 2>);
  return nullptr;
}

// Rows of partial sums of the backward pass: a block for each of 256 compute
// units, more where a block is less than eight waves.  No property of the
// device, so that the workspace and the order of the sums are not either.
int64_t norm_parts(int64_t rows, int64_t cols) {
  const int threads = norm_shape(cols, true).threads;
  return balanced(rows, 256 * (threads >= 512 ? 1 : threads >= 128 ? 512 / threads : 4));
}

bool norm_sizes_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && cols <= kMaxCols && rows <= INT64_MAX / 8 / kMaxCols;
}

coat_status_t check_norm_shape(int64_t rows, int64_t cols, int32_t group_size) {
  if (rows < 0 || cols < 0) return COAT_ERR_INVALID_VALUE;
  if (!valid_group_size(group_size)) return COAT_ERR_GROUP_SIZE;
  if (cols % group_size != 0 || !norm_sizes_ok(rows, cols)) return COAT_ERR_INVALID_VALUE;
  return COAT_OK;
}

}  // namespace

namespace coat {

hipError_t launch_sum_partials(const float* partials, int parts, int64_t cols, float* dst0, int64_t split,
                               float* dst1, bool accumulate, hipStream_t stream) {
  int acc = accumulate ? 1 : 0;
  void* args[] = {&partials, &parts, &cols, &dst0, &split, &dst1, &acc};
  return hipLaunchKernel(reinterpret_cast<const void*>(&sum_partials_kernel),
                         dim3((unsigned)((cols + kSumCols - 1) / kSumCols)), dim3(kSumCols * kSumSlices), args, 0,
                         stream);
}

}  // namespace coat

extern "C" {

coat_status_t coat_fp8_rms_norm(const coat_rms_norm_args_t* a, hipStream_t stream) {
  if (!a) return COAT_ERR_NULL_POINTER;
  const coat_status_t st = check_norm_shape(a->rows, a->cols, a->group_size);
  if (st != COAT_OK) return st;
  if (!isfinite(a->eps) || a->eps < 0x1p-126f) return COAT_ERR_INVALID_VALUE;
  if (a->y_codes && !(a->y_scale > 0.0f && isfinite(a->y_scale) && isfinite(1.0f / a->y_scale)))
    return COAT_ERR_INVALID_VALUE;
  if (a->y_amax && !a->y_codes) return COAT_ERR_INVALID_VALUE;
  if (a->rows == 0 || a->cols == 0) return COAT_OK;
  if (!a->x || !a->weight || (!a->y && !a->y_codes)) return COAT_ERR_NULL_POINTER;
  if (!a->residual != !a->residual_out || !a->codes != !a->scales) return COAT_ERR_NULL_POINTER;
  if (!aligned(a->x, 16) || !aligned(a->weight, 16) || !aligned(a->residual, 16) || !aligned(a->residual_out, 16) ||
      !aligned(a->y, 16) || !aligned(a->y_codes, 16) || !aligned(a->codes, 16) || !aligned(a->scales, 4) ||
      !aligned(a->rstd, 4) || !aligned(a->y_amax, 4))
    return COAT_ERR_MISALIGNED;
  NormParams p;
  memset(&p, 0, sizeof(p));
  p.x = a->x;
  p.residual = a->residual;
  p.weight = a->weight;
  p.sum = a->residual_out;
  p.y = a->y;
  p.y_codes = a->y_codes;
  p.y_amax = a->y_amax;
  p.codes = a->codes;
  p.scales = a->scales;
  p.rstd = a->rstd;
  p.rows = a->rows;
  p.cols = (int32_t)a->cols;
  p.group_shift = __builtin_ctz((unsigned)a->group_size);
  p.eps = a->eps;
  p.inv_y_scale = a->y_codes ? 1.0f / a->y_scale : 0.0f;
  p.inv_cols = (float)(1.0 / (double)a->cols);
  int cus = 0;
  hipError_t e = current_cu_count(&cus);
  if (e != hipSuccess) return hip_fail(e);
  const NormShape s = norm_shape(a->cols, false);
  // as many blocks as the registers let a CU hold, all with as many rows:
  // 28 waves with one chunk a thread, 16 with more
  const int64_t blocks = balanced(a->rows, (int64_t)cus * ((s.chunks == 1 ? 28 : 16) * 64 / s.threads));
  void* args[] = {&p};
  if (s.most == 64 && a->y_amax && blocks > 128)
    e = hipLaunchKernel(reinterpret_cast<const void*>(&rms_norm_kernel<64, 1, kWaveRows>),
                        dim3((unsigned)((blocks + kWaveRows - 1) / kWaveRows)), dim3(64 * kWaveRows), args, 0, stream);
  else
    e = hipLaunchKernel(norm_kernel_for(s, kForward), dim3((unsigned)blocks), dim3(s.threads), args, 0, stream);
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

int64_t coat_fp8_rms_norm_bwd_workspace(int64_t rows, int64_t cols) {
  if (!norm_sizes_ok(rows, cols) || cols % 16 != 0) return -1;
  return cols == 0 ? 0 : norm_parts(rows, cols) * cols * (int64_t)sizeof(float);
}

coat_status_t coat_fp8_rms_norm_bwd(const coat_rms_norm_bwd_args_t* a, hipStream_t stream) {
  if (!a) return COAT_ERR_NULL_POINTER;
  const coat_status_t st = check_norm_shape(a->rows, a->cols, a->group_size);
  if (st != COAT_OK) return st;
  if (a->cols == 0 || (a->rows == 0 && (!a->dw || a->accumulate))) return COAT_OK;
  if (a->dw && !a->workspace && a->rows > 0) return COAT_ERR_NULL_POINTER;
  if (a->rows > 0 && (!a->dy || !a->codes || !a->scales || !a->rstd || !a->weight || !a->dx))
    return COAT_ERR_NULL_POINTER;
  if (!aligned(a->dy, 16) || !aligned(a->codes, 16) || !aligned(a->scales, 4) || !aligned(a->rstd, 4) ||
      !aligned(a->weight, 16) || !aligned(a->d_residual, 16) || !aligned(a->dx, 16) || !aligned(a->dw, 4) ||
      !aligned(a->workspace, 16))
    return COAT_ERR_MISALIGNED;
  if (a->dw && a->rows > 0 && a->workspace_bytes < coat_fp8_rms_norm_bwd_workspace(a->rows, a->cols))
    return COAT_ERR_INVALID_VALUE;
  if (a->rows > 0 && (const void*)a->dx == (const void*)a->dy) return COAT_ERR_INVALID_VALUE;   // (see the kernel of few rows)
  const bool few = a->dw && a->rows > 0 && few_rows(a->rows, norm_shape(a->cols, true).threads);
  const int64_t blocks = norm_parts(a->rows, a->cols);
  hipError_t e = hipSuccess;
  if (a->rows > 0) {
    NormBwdParams p;
    memset(&p, 0, sizeof(p));
    p.dy = a->dy;
    p.codes = a->codes;
    p.scales = a->scales;
    p.rstd = a->rstd;
    p.weight = a->weight;
    p.d_residual = a->d_residual;
    p.dx = a->dx;
    p.partials = a->dw && !few ? (float*)a->workspace : nullptr;
    p.dw = a->dw;
    p.accumulate = a->accumulate != 0;
    p.rows = a->rows;
    p.cols = (int32_t)a->cols;
    p.group_shift = __builtin_ctz((unsigned)a->group_size);
    p.inv_cols = (float)(1.0 / (double)a->cols);
    const NormShape s = norm_shape(a->cols, true);
    void* args[] = {&p};
    const int64_t grid = few ? a->rows + (a->cols + kFewCols - 1) / kFewCols : blocks;
    e = hipLaunchKernel(norm_kernel_for(s, few ? kBackwardFew : kBackward), dim3((unsigned)grid), dim3(s.threads), args,
                        0, stream);
  }
  // no rows: the sum of no partial sums, zero
  if (e == hipSuccess && a->dw && !few)
    e = launch_sum_partials((const float*)a->workspace, (int)blocks, a->cols, a->dw, a->cols, nullptr,
                            a->accumulate != 0, stream);
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

}  // extern "C"
