// coat_tile.h -- the matrix-core tile that the cross entropy's products share
// (not part of the C ABI).
//
// A block computes a kBM x kBN tile of C[m][n] = sum over k of A(m, k) B(n, k).
// Each operand lies in memory either with k fastest ("minor": rows of k, BF16
// or E4M3) or with k slowest ("slow": k rows of m or n values, BF16).  A step
// of the pipeline is 128 bytes of k for minor operands, 64 BF16 values or 128
// codes, so a stage's panel of R rows takes 128 R bytes either way.  Panels go
// from global memory straight into the LDS as they lie; the MFMA's operands
// are read from minor panels as 16-byte chunks and from slow ones by the LDS's
// transposing reads, which hand each lane eight consecutive k of its column.
//
// Two stages.  A step is two phases, one for each half of its k.  Phase 0 runs
// on fragment set 0 while set 1 is read; then every wave waits for its reads
// and for its loads into the other stage, and the block meets; phase 1 runs on
// set 1 while set 0 of the next step is read from the other stage and the
// loads of the step after next go into this one.
//
// Not taken (loss of 8192 x 32000 x 4096): the neighbours' common panels fetched
// into the L2 some steps ahead (2.79e6 cycles, 2.87e6 with it), waves that take
// turns with their loads (2.76e6, 2.97e6).
//
// The MFMA takes B as its first operand, so each result is a tile of C^T.  With
// results of kMf x kMf (32 or 16), L = 64 / kMf lanes share a row, and lane l
// holds of the wave's row tile i
//   row = kMf i + l % kMf,  columns 4 L u + 4 (l / kMf) + 0..3 for u < kRuns,
// in runs of four (quad()).
//
// BF16 products use the 16 x 16 x 32 instruction, codes 32 x 32 x 64.  Large
// products are bound by the card's power, and 32 x 32 x 16 takes more of it: it
// reads and writes twice the accumulators for a product, for half the
// operands.  The same tile with it needs fewer cycles (matrix cores busy for
// 77% of them, not 72%), at 1.66 GHz instead of 1.89: loss of
// 8192 x 32000 x 4096 1593 us, with 16 x 16 x 32 1519; gradients 4897 and 4765.
#ifndef COAT_TILE_H
#define COAT_TILE_H

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "coat_elem.h"

namespace coat {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// kWM x kWN waves of kI x kJ tiles of 32 x 32.  kArrA: bytes of an LDS array
// of A, for tiles that share a kernel's arrays with a larger one.  kStages: of
// mma_stream; 2 for mma_run.  kMf: of the MFMA's results.
template <int kMf_, int kWM_, int kWN_, int kI_, int kJ_, int kArrA_ = 0, int kStages_ = 2>
struct MmaTile {
  static constexpr int kWM = kWM_, kWN = kWN_, kI = kI_, kJ = kJ_, kStages = kStages_, kMf = kMf_;
  static constexpr int kRT = 32 * kI / kMf, kCT = 32 * kJ / kMf;     // results of a wave
  static constexpr int kL = 64 / kMf, kRuns = 8 * kJ / kL;           // lanes of a row, and their runs of columns
  using Acc = std::conditional_t<kMf == 32, v16f, v4f>[kRT][kCT];
  static constexpr int kWaves = kWM * kWN, kThreads = 64 * kWaves;
  static constexpr int kBM = 32 * kWM * kI, kBN = 32 * kWN * kJ;
  static constexpr int kA = 128 * kBM, kB = 128 * kBN;               // bytes of a stage's panels
  static constexpr int kLA = kA / 1024 / kWaves, kLB = kB / 1024 / kWaves;   // loads of a wave
  static constexpr int kArrA = kArrA_ ? kArrA_ : kA;
};

// The LDS arrays of a kernel: A and B of two stages (arrays 0 to 3), or with
// more stages an array for each, A's panel and B's behind it.  Being distinct
// objects, the compiler can tell the loads into one stage from the reads of
// the other, and does not wait for loads in flight before it reads (it keeps
// apart seven such objects at most).
template <int kBytes, int kWhich>
__device__ __forceinline__ uint8_t* mma_array() {
  __shared__ __attribute__((aligned(1024))) uint8_t bytes[kBytes];
  return bytes;
}

template <class T>
constexpr int mma_part_bytes(int which) {
  return T::kStages > 2 ? T::kA + T::kB : which % 2 == 0 ? T::kArrA : T::kB;
}

template <class T, int kWhich>
__device__ __forceinline__ uint8_t* mma_part() {
  return mma_array<mma_part_bytes<T>(kWhich), kWhich>();
}

// Minor panels: the 16-byte chunk of a 128-byte row is XORed with (row / 2) % 8,
// slow ones: the 32-byte chunk of a row with 2 (k % 4) + k / 8 % 2; then no read
// meets a bank twice (slow rows are multiples of 256 bytes).
__device__ __forceinline__ int minor_swz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int slow_chunk(int k, int c32) { return c32 ^ (2 * (k & 3) + ((k >> 3) & 1)); }

// Byte offsets of a lane's loads into a minor panel of kBlock rows: row(r)
// gives the byte offset of the panel's row r.
template <int kLoads, class Row>
__device__ __forceinline__ void minor_offsets(int wave, int lane, Row row, uint32_t (&off)[kLoads]) {
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = 8 * (kLoads * wave + i) + (lane >> 3);
    off[i] = row(r) + 16u * (uint32_t)((lane & 7) ^ minor_swz(r));
  }
}

// Those of a slow panel of kCols columns: k rows of `stride` bytes; columns
// from `valid` on (a multiple of 8) re-load the last chunk.  Loads whose rows
// have their chunks alike share an offset: load i takes
// off[i % kSlowDistinct], and 4 rows more for each time round.
template <int kLoads, int kCols>
constexpr int kSlowDistinct = kCols == 256 && kLoads == 4 ? 2 : kLoads;   // (two rows a load, alike four rows apart)

template <int kLoads, int kCols>
__device__ __forceinline__ void slow_offsets(int wave, int lane, uint32_t stride, int64_t valid,
                                             uint32_t (&off)[kSlowDistinct<kLoads, kCols>]) {
#pragma unroll
  for (int i = 0; i < kSlowDistinct<kLoads, kCols>; ++i) {
    const int byte = 1024 * (kLoads * wave + i) + 16 * lane, k = byte / (2 * kCols), c16 = byte % (2 * kCols) / 16;
    const int col = 8 * (2 * slow_chunk(k, c16 >> 1) + (c16 & 1));
    off[i] = (uint32_t)k * stride + 2u * (uint32_t)(col < valid ? col : (int)valid - 8);
  }
}

template <class T>
__device__ __forceinline__ void mma_zero(typename T::Acc& acc) {
#pragma unroll
  for (int i = 0; i < T::kRT; ++i)
#pragma unroll
    for (int j = 0; j < T::kCT; ++j)
#pragma unroll
      for (int r = 0; r < T::kMf * T::kMf / 64; ++r) acc[i][j][r] = 0.0f;
}

// Value s of the lane's run u of row tile i.
template <class T>
__device__ __forceinline__ float quad(const typename T::Acc& acc, int i, int u, int s) {
  if constexpr (T::kMf == 32) return acc[i][u / 4][4 * (u % 4) + s];
  else return acc[i][u][s];
}

template <class T>
__device__ __forceinline__ void set_quad(typename T::Acc& acc, int i, int u, int s, float v) {
  if constexpr (T::kMf == 32) acc[i][u / 4][4 * (u % 4) + s] = v;
  else acc[i][u][s] = v;
}

// Adds the products of `steps` steps.  a(step), b(step): the panels' base
// addresses (uniform); aoff, boff: the lane's offsets, where slow those of rows
// of a_stride, b_stride bytes; b_bytes(step): bytes behind b(step) that may be
// read (what lies behind them is taken as zero).  The block has met at the end,
// and no load is in flight.
template <class T, bool kFP8, bool kASlow, bool kBSlow, class A, int kDA, class B, int kDB, class Bytes>
__device__ __forceinline__ void mma_run(typename T::Acc& acc, int steps, A a, const uint32_t (&aoff)[kDA], uint32_t a_stride,
                                        B b, const uint32_t (&boff)[kDB], uint32_t b_stride, Bytes b_bytes) {
#if __HIP_DEVICE_COMPILE__   // (the host has no type for a buffer's description)
  constexpr int kI = T::kI, kJ = T::kJ, kLA = T::kLA, kLB = T::kLB, kL = kLA + kLB;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % T::kWM, wn = wave / T::kWM;
  static_assert(kFP8 == (T::kMf == 32), "the instructions used");
  if (steps <= 0) {
    __syncthreads();
    return;
  }
  static_assert(kDA == (kASlow ? kSlowDistinct<kLA, T::kBM> : kLA) && kDB == (kBSlow ? kSlowDistinct<kLB, T::kBN> : kLB), "");
  auto rsrc = [](const void* p, uint32_t bytes) __attribute__((always_inline)) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
  };
  struct From {
    __amdgpu_buffer_rsrc_t a, b;
  };
  // (past the last step the last one is fetched again, into a stage that is not read)
  auto from = [&](int step) __attribute__((always_inline)) {
    const int s = step < steps ? step : steps - 1;
    return From{rsrc(a(s), 0xFFFFFFFFu), rsrc(b(s), kBSlow ? (uint32_t)b_bytes(s) : 0xFFFFFFFFu)};
  };
  auto load1 = [&](const From& f, auto S, int q) __attribute__((always_inline)) {
    constexpr int st = decltype(S)::value;
    if (q < kLA) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(f.a, mma_part<T, 2 * st>() + 1024 * (kLA * wave + q), 16,
                                               (int)aoff[q % kDA], (int)(4 * (q / kDA) * a_stride), 0, 0);
    } else {
      const int i = q - kLA;
      // (a load whose two offsets reach the description's bytes puts zeros into
      // the LDS, also where the scalar one alone does)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(f.b, mma_part<T, 2 * st + 1>() + 1024 * (kLB * wave + i), 16,
                                               (int)boff[i % kDB], (int)(4 * (i / kDB) * b_stride), 0, 0);
    }
  };

  // Fragments, 16 rows of 16 bytes a lane.  A phase takes 64 bytes of each row,
  // chunks 4 kk + 0..3.  16 x 16 x 32 (BF16): row 16 i + lane % 16, chunk
  // 4 kk + lane / 16, so k = 32 kk + 8 (lane / 16) + 0..7, which slow panels are
  // read at too.  32 x 32 x 64 (codes): two for row 32 i + lane % 32, chunks
  // 4 kk + 2 (lane / 32) + {0, 1}.
  // (Offsets are single opaque values: the compiler follows an address back
  // over a few additions only.)
  constexpr int kFA = 2 * kI, kFB = 2 * kJ;
  uint4 fa[2][kFA], fb[2][kFB];
  // minor: the first rows' chunks of phase 0 (of codes, the two; phase 1 flips
  // bit 6), other rows whole tiles further; slow: the first tile's (tile i flips
  // the bits of 32 i), phases and the second half whole rows further
  constexpr int kChunks = T::kMf == 32 ? 2 : 1;
  int a_at[kASlow ? 1 : kChunks], b_at[kBSlow ? 1 : kChunks];
  auto slow_at = [&](int first, int cols) __attribute__((always_inline)) {
    const int c = first + 4 * (lane & 3), k = 8 * (lane >> 4) + ((lane & 15) >> 2);
    return k * 2 * cols + 32 * slow_chunk(k, c >> 4) + 2 * (c & 15);
  };
  auto minor_at = [&](int first, int e) __attribute__((always_inline)) {
    const int row = lane % T::kMf;
    return 128 * (first + row) + 16 * ((kChunks * (lane / T::kMf) + e) ^ minor_swz(row));
  };
#pragma unroll
  for (int i = 0; i < (kASlow ? 1 : kChunks); ++i) {
    a_at[i] = kASlow ? slow_at(32 * kI * wm, T::kBM) : minor_at(32 * kI * wm, i);
    asm volatile("" : "+v"(a_at[i]));
  }
#pragma unroll
  for (int j = 0; j < (kBSlow ? 1 : kChunks); ++j) {
    b_at[j] = kBSlow ? slow_at(32 * kJ * wn, T::kBN) : minor_at(32 * kJ * wn, j);
    asm volatile("" : "+v"(b_at[j]));
  }
  auto slow4 = [&](const uint8_t* panel, int at) __attribute__((always_inline)) {
    const v4s v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(panel + at));
    return __builtin_bit_cast(uint2, v);
  };
  // Reads of a phase: A before B; a fragment of a slow panel is two reads.  (The
  // MFMAs go column by column: of the set at hand all A fragments stay to the
  // end and B's, which are more, are done with one after the other.)
  constexpr int kNA = kASlow ? 2 : 1, kNB = kBSlow ? 2 : 1, kR = kFB * kNB + kFA * kNA;
  int tile = 0;
  auto read_to = [&](uint4& to, const uint8_t* panel, const int* at, auto Slow, int cols, int kk, int t) __attribute__((always_inline)) {
    if constexpr (decltype(Slow)::value) {
      static_assert((kFA & (kFA - 1)) == 0 && (kFB & (kFB - 1)) == 0 && kFA <= 8 && kFB <= 8, "flipped bits of a tile's chunk");
      // (formed for its two reads: kept, they would not fit the registers)
      if (t == 0) tile = at[0];
      else if (t % 2 == 0) asm volatile("v_xor_b32 %0, %1, %2" : "=v"(tile) : "s"(32 * (t / 2)), "v"(at[0]));
      const uint2 v = slow4(panel, tile + (32 * kk + 4 * (t % 2)) * 2 * cols);
      if (t % 2 == 0) to.x = v.x, to.y = v.y;
      else to.z = v.x, to.w = v.y;
    } else {
      to = *reinterpret_cast<const uint4*>(panel + (at[t % kChunks] ^ (64 * kk)) + 128 * T::kMf * (t / kChunks));
    }
  };
  auto read1 = [&](int f, const uint8_t* As, const uint8_t* Bs, int kk, int r) __attribute__((always_inline)) {
    if (r < kFA * kNA) read_to(fa[f][r / kNA], As, a_at, std::bool_constant<kASlow>{}, T::kBM, kk, r);
    else read_to(fb[f][(r - kFA * kNA) / kNB], Bs, b_at, std::bool_constant<kBSlow>{}, T::kBN, kk, r - kFA * kNA);
  };
  auto as_v8 = [](const uint4* v) __attribute__((always_inline)) {
    return v8i{(int)v[0].x, (int)v[0].y, (int)v[0].z, (int)v[0].w,
               (int)v[1].x, (int)v[1].y, (int)v[1].z, (int)v[1].w};
  };
  constexpr int kMF = T::kRT * T::kCT;
  // MFMAs that reads go out behind, the rest give them time to arrive (loss of
  // 8192 x 32000 x 4096: 1531 us behind 7/8, 1524 behind 3/4, 1514, 1534 behind 1/2)
  constexpr int kRF = kMF * 5 / 8;
  // Loads go out kPer at a time behind every kGap-th MFMA.  All waves begin with
  // theirs after the same barrier, and a wave whose load has to queue issues
  // nothing else.  Of codes, with 8 MFMAs a phase, two behind each (loss of
  // 8192 x 32000 x 4096: 795 us, 802 with one); of BF16, with 32, one behind
  // every second (1519 us, 1528 behind every fourth, 1531 behind each), and one
  // behind every fourth where slow panels' reads, twice as many, go out too
  // (gradients of that loss: 4765, 4804 behind every third).
  constexpr int kMost = kBSlow ? 4 : 2;
  constexpr int kPer = kFP8 ? 2 : 1, kGap = kFP8 ? 1 : kMF / kL < kMost ? kMF / kL : kMost;
  static_assert(kPer * kMF >= kGap * kL, "a phase issues a stage's loads");
  auto mma1 = [&](int f, int n) __attribute__((always_inline)) {
    const int i = n % T::kRT, j = n / T::kRT;
    if constexpr (kFP8)
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(as_v8(&fb[f][2 * j]), as_v8(&fa[f][2 * i]), acc[i][j], 0, 0,
                                                                  0, 0, 0, 0);
    else
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, fb[f][j]),
                                                          __builtin_bit_cast(v8bf, fa[f][i]), acc[i][j], 0, 0, 0);
  };
  auto kstep = [&](int step, auto S) __attribute__((always_inline)) {
    constexpr int st = decltype(S)::value;
    const uint8_t *As = mma_part<T, 2 * st>(), *Bs = mma_part<T, 2 * st + 1>();
    const uint8_t *An = mma_part<T, 2 * (1 - st)>(), *Bn = mma_part<T, 2 * (1 - st) + 1>();
#pragma unroll
    for (int n = 0; n < kMF; ++n) {
      mma1(0, n);
#pragma unroll
      for (int r = n * kR / kRF; r < (n + 1) * kR / kRF; ++r)
        if (r < kR) read1(1, As, Bs, 1, r);
      __builtin_amdgcn_sched_barrier(0);
    }
    const From next = from(step + 2);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kMF; ++n) {
      mma1(1, n);
#pragma unroll
      for (int r = n * kR / kRF; r < (n + 1) * kR / kRF; ++r)
        if (r < kR) read1(0, An, Bn, 0, r);
#pragma unroll
      for (int q = 0; q < kL; ++q)
        if (q / kPer * kGap == n) load1(next, S, q);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  // vmcnt(kL): the loads of stage 1 may stay in flight (vmcnt in bits 3:0 and
  // 15:14, expcnt in 6:4, lgkmcnt in 11:8)
  static_assert(kL < 64, "vmcnt holds at most 63");
  constexpr int kStage1InFlight = (kL & 15) | ((kL >> 4) << 14) | (7 << 4) | (15 << 8);
  {
    const From f0 = from(0), f1 = from(1);
#pragma unroll
    for (int q = 0; q < kL; ++q) load1(f0, S0{}, q);
    if (steps == 1) __builtin_amdgcn_s_waitcnt(7 << 4 | 15 << 8);   // vmcnt(0)
    else {
#pragma unroll
      for (int q = 0; q < kL; ++q) load1(f1, S1{}, q);
    }
  }
  __builtin_amdgcn_s_waitcnt(kStage1InFlight);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
#pragma unroll
  for (int r = 0; r < kR; ++r) read1(0, mma_part<T, 0>(), mma_part<T, 1>(), 0, r);
  int step = 0;
  for (; step + 1 < steps; step += 2) {
    kstep(step, S0{});
    kstep(step + 1, S1{});
  }
  if (step < steps) kstep(step, S0{});
  __builtin_amdgcn_s_waitcnt(0);   // no load into the LDS outlives the loop
  __syncthreads();
#endif
}

// The same for minor operands in a thin tile, which waits for memory and not
// for the MFMAs: kStages stages in a ring, kStages - 1 steps of loads in
// flight, one barrier a step.
template <class T, bool kFP8>
__device__ __forceinline__ void mma_stream(typename T::Acc& acc, int steps, const uint8_t* a,
                                           const uint32_t (&aoff)[T::kLA], const uint8_t* b,
                                           const uint32_t (&boff)[T::kLB]) {
#if __HIP_DEVICE_COMPILE__
  constexpr int kI = T::kI, kJ = T::kJ, kLA = T::kLA, kLB = T::kLB, kL = kLA + kLB, kS = T::kStages;
  static_assert(T::kMf == 32, "the instructions used");
  static_assert(kS > 2 && kS <= 7 && kL * (kS - 1) < 64, "stages and loads in flight");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % T::kWM, wn = wave / T::kWM, half = lane >> 5, l32 = lane & 31;
  int a_at[2], b_at[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int chunk = 16 * ((2 * half + e) ^ minor_swz(l32));
    a_at[e] = 128 * (32 * kI * wm + l32) + chunk;
    b_at[e] = T::kA + 128 * (32 * kJ * wn + l32) + chunk;
    asm volatile("" : "+v"(a_at[e]), "+v"(b_at[e]));
  }
  auto load = [&](int step, auto S) __attribute__((always_inline)) {
    constexpr int st = decltype(S)::value;
    const int64_t at = 128 * (int64_t)(step < steps ? step : steps - 1);
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)(a + at), (short)0, (int)0xFFFFFFFF, 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void*)(b + at), (short)0, (int)0xFFFFFFFF, 0x00020000);
#pragma unroll
    for (int q = 0; q < kLB; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, mma_part<T, st>() + T::kA + 1024 * (kLB * wave + q), 16, (int)boff[q], 0, 0, 0);
#pragma unroll
    for (int q = 0; q < kLA; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, mma_part<T, st>() + 1024 * (kLA * wave + q), 16, (int)aoff[q], 0, 0, 0);
  };
  // vmcnt(kL (kS - 2)), and lgkmcnt(0): the wave has read the stage before
  constexpr int kFlight = kL * (kS - 2), kWait = (kFlight & 15) | ((kFlight >> 4) << 14) | (7 << 4);
  auto kstep = [&](int step, auto S) __attribute__((always_inline)) {
    constexpr int st = decltype(S)::value;
    __builtin_amdgcn_s_waitcnt(kWait);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    load(step + kS - 1, std::integral_constant<int, (st + kS - 1) % kS>{});
    const uint8_t* p = mma_part<T, st>();
    auto as_v8 = [](const uint4& lo, const uint4& hi) __attribute__((always_inline)) {
      return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      uint4 fa[kI][2], fb[kJ][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int j = 0; j < kJ; ++j) fb[j][e] = *reinterpret_cast<const uint4*>(p + (b_at[e] ^ (64 * kk)) + 4096 * j);
#pragma unroll
        for (int i = 0; i < kI; ++i) fa[i][e] = *reinterpret_cast<const uint4*>(p + (a_at[e] ^ (64 * kk)) + 4096 * i);
      }
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          if constexpr (kFP8) {
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(as_v8(fb[j][0], fb[j][1]), as_v8(fa[i][0], fa[i][1]),
                                                                        acc[i][j], 0, 0, 0, 0, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, fb[j][e]),
                                                                  __builtin_bit_cast(v8bf, fa[i][e]), acc[i][j], 0, 0, 0);
          }
        }
    }
  };
  auto each = [&](auto self, int step, auto S, auto fn) __attribute__((always_inline)) -> void {
    constexpr int st = decltype(S)::value;
    if constexpr (st < kS) {
      if (!fn(step + st, S)) return;
      self(self, step, std::integral_constant<int, st + 1>{}, fn);
    }
  };
  using S0 = std::integral_constant<int, 0>;
  each(each, 0, S0{}, [&](int step, auto S) __attribute__((always_inline)) {
    if constexpr (decltype(S)::value < kS - 1) load(step, S);
    return true;
  });
  int step = 0;
  for (; step + kS <= steps; step += kS)
    each(each, step, S0{}, [&](int t, auto S) __attribute__((always_inline)) {
      kstep(t, S);
      return true;
    });
  each(each, step, S0{}, [&](int t, auto S) __attribute__((always_inline)) {
    if (t >= steps) return false;
    kstep(t, S);
    return true;
  });
  __builtin_amdgcn_s_waitcnt(0);   // no load into the LDS outlives the loop
  __syncthreads();
#endif
}

// A BF16 tile through the LDS, so that it leaves in whole 16-byte chunks of
// rows.  word(i, u) gives the four values of a run, packed; out(row, chunk,
// bytes) takes chunk `chunk` (8 columns) of row `row` of the tile.  The block
// must have met before and meets inside; patch(i, set) may replace single
// values of the lane's row of tile i before it does, by set(column, bits).
// Chunks are XORed with row % 16 (or
// the chunks of a shorter row): 8-byte writes of 32 rows and 16-byte reads
// meet no bank conflicts.
template <class T, class Word, class Out, class Patch>
__device__ __forceinline__ void tile_out_bf16(Word word, Out out, Patch patch) {
  constexpr int kRowBytes = 2 * T::kBN, kChunks = kRowBytes / 16, kMask = (kChunks < 16 ? kChunks : 16) - 1;
  constexpr int kPart = mma_part_bytes<T>(0), kRows = kPart / kRowBytes / 32 * 32;   // rows of an LDS array
  static_assert(kRows >= 32 && kRows * 4 >= T::kBM && mma_part_bytes<T>(1) >= kPart, "the tile fits the arrays");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % T::kWM, wn = wave / T::kWM, share = lane / T::kMf;
  auto part = [](int q) __attribute__((always_inline)) {
    return q == 0 ? mma_part<T, 0>() : q == 1 ? mma_part<T, 1>() : q == 2 ? mma_part<T, 2>() : mma_part<T, 3>();
  };
  auto at = [](int row, int c) __attribute__((always_inline)) { return row % kRows * kRowBytes + 16 * (c ^ (row & kMask)); };
#pragma unroll
  for (int i = 0; i < T::kRT; ++i) {
    const int first = 32 * T::kI * wm + T::kMf * i, row = first + lane % T::kMf;
    uint8_t* tile = part(first / kRows);
#pragma unroll
    for (int u = 0; u < T::kRuns; ++u) {
      *reinterpret_cast<uint2*>(tile + at(row, 4 * T::kJ * wn + T::kL / 2 * u + share / 2) + 8 * (share & 1)) = word(i, u);
      if (u % 2) __builtin_amdgcn_sched_barrier(0);   // (or every word is begun before one is stored)
    }
    patch(i, [&](int col, uint32_t bits) __attribute__((always_inline)) {
      *reinterpret_cast<uint16_t*>(tile + at(row, col >> 3) + 2 * (col & 7)) = (uint16_t)bits;
    });
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < T::kBM * kChunks / T::kThreads; ++k) {
    const int task = k * T::kThreads + threadIdx.x, row = task / kChunks, c = task % kChunks;
    out(row, c, *reinterpret_cast<const uint4*>(part(row / kRows) + at(row, c)));
  }
}

// The value at column `col` (of the wave's 32 kJ, in one of the lane's runs) of
// the lane's row of tile i: a tree of selections by the column's bits, each a
// mask.  (Of conditions the compiler makes searches through whole vectors.)
template <class T>
__device__ __forceinline__ float value_at(const typename T::Acc& acc, int i, int col) {
  constexpr int kRuns = T::kRuns;
  static_assert((kRuns & (kRuns - 1)) == 0 && kRuns <= 16, "a power of two");
  auto mask_of = [&](int bit) __attribute__((always_inline)) {
    uint32_t m = 0u - (uint32_t)((col >> bit) & 1);
    asm volatile("" : "+v"(m));
    return m;
  };
  auto pick = [](uint32_t m, uint32_t zero, uint32_t one) __attribute__((always_inline)) { return (one & m) | (zero & ~m); };
  const uint32_t m0 = mask_of(0), m1 = mask_of(1);
  uint32_t v[kRuns];
#pragma unroll
  for (int u = 0; u < kRuns; ++u) {
    auto bits = [&](int s) __attribute__((always_inline)) { return __float_as_uint(quad<T>(acc, i, u, s)); };
    v[u] = pick(m1, pick(m0, bits(0), bits(1)), pick(m0, bits(2), bits(3)));
  }
  constexpr int kFirst = T::kL == 2 ? 3 : 4;   // the column's bits: 2 of the run, those of the lane, those of u
#pragma unroll
  for (int b = 0; (1 << b) < kRuns; ++b) {
    const uint32_t m = mask_of(kFirst + b);
#pragma unroll
    for (int u = 0; u < kRuns; u += 2 << b) v[u] = pick(m, v[u], v[u + (1 << b)]);
  }
  return __uint_as_float(v[0]);
}

template <class T, class Word, class Out>
__device__ __forceinline__ void tile_out_bf16(Word word, Out out) {
  tile_out_bf16<T>(word, out, [](int, auto) {});
}

// xcd_contiguous for 32-bit indexes.
__device__ __forceinline__ uint32_t xcd_contiguous32(uint32_t b, uint32_t nb) {
  const uint32_t q = nb / 8, r = nb % 8, xcd = b % 8, local = b / 8;
  return xcd < r ? xcd * (q + 1) + local : r * (q + 1) + (xcd - r) * q + local;
}

}  // namespace coat

#endif  // COAT_TILE_H
