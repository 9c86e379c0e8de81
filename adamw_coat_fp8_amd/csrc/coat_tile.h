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
// The MFMA takes B as its first operand, so each 32 x 32 result is a tile of
// C^T: register 4 q + s of acc[i][j] is C[row][col] with
//   row = 32 kI wm + 32 i + lane % 32,  col = 32 kJ wn + 32 j + 8 q + 4 (lane / 32) + s,
// runs of four columns a lane, and lanes l and l ^ 32 hold all the wave's
// columns of a row.
#ifndef COAT_TILE_H
#define COAT_TILE_H

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "coat_elem.h"

namespace coat {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// kWM x kWN waves of kI x kJ tiles of 32 x 32.  kArrA: bytes of an LDS array
// of A, for tiles that share a kernel's arrays with a larger one.  kStages: of
// mma_stream; 2 for mma_run.
template <int kWM_, int kWN_, int kI_, int kJ_, int kArrA_ = 0, int kStages_ = 2>
struct MmaTile {
  static constexpr int kWM = kWM_, kWN = kWN_, kI = kI_, kJ = kJ_, kStages = kStages_;
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
// slow ones: the 64-byte chunk of a row with k % 4; then no read meets a bank
// twice (slow rows are multiples of 256 bytes).
__device__ __forceinline__ int minor_swz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int slow_chunk(int k, int c64) { return c64 ^ (k & 3); }

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
// from `valid` on (a multiple of 8) re-load the last chunk, and rows from
// `k_rows` on the last row.
template <int kLoads, int kCols>
__device__ __forceinline__ void slow_offsets(int wave, int lane, uint32_t stride, int64_t valid, int k_rows,
                                             uint32_t (&off)[kLoads]) {
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int byte = 1024 * (kLoads * wave + i) + 16 * lane, k = byte / (2 * kCols), c16 = byte % (2 * kCols) / 16;
    const int col = 8 * (4 * slow_chunk(k, c16 >> 2) + (c16 & 3));
    off[i] = (uint32_t)(k < k_rows ? k : k_rows - 1) * stride + 2u * (uint32_t)(col < valid ? col : (int)valid - 8);
  }
}

template <class T>
__device__ __forceinline__ void mma_zero(v16f (&acc)[T::kI][T::kJ]) {
#pragma unroll
  for (int i = 0; i < T::kI; ++i)
#pragma unroll
    for (int j = 0; j < T::kJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
}

// Adds the products of `steps` steps.  a(step), b(step): the panels' base
// addresses (uniform); aoff, boff: the lane's offsets; blast: those of B in
// steps for which b_last(step) holds.  The block has met at the end, and no
// load is in flight.
template <class T, bool kFP8, bool kASlow, bool kBSlow, class A, class B, class Last>
__device__ __forceinline__ void mma_run(v16f (&acc)[T::kI][T::kJ], int steps, A a, const uint32_t (&aoff)[T::kLA], B b,
                                        const uint32_t (&boff)[T::kLB], const uint32_t (&blast)[T::kLB], Last b_last) {
#if __HIP_DEVICE_COMPILE__   // (the host has no type for a buffer's description)
  constexpr int kI = T::kI, kJ = T::kJ, kLA = T::kLA, kLB = T::kLB, kL = kLA + kLB;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % T::kWM, wn = wave / T::kWM;
  const int half = lane >> 5, l32 = lane & 31;
  if (steps <= 0) {
    __syncthreads();
    return;
  }
  auto rsrc = [](const void* p) __attribute__((always_inline)) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)0xFFFFFFFF, 0x00020000);
  };
  struct From {
    __amdgpu_buffer_rsrc_t a, b;
    bool last;
  };
  // (past the last step the last one is fetched again, into a stage that is not read)
  auto from = [&](int step) __attribute__((always_inline)) {
    const int s = step < steps ? step : steps - 1;
    return From{rsrc(a(s)), rsrc(b(s)), kBSlow ? (bool)b_last(s) : false};
  };
  auto load1 = [&](const From& f, auto S, int q) __attribute__((always_inline)) {
    constexpr int st = decltype(S)::value;
    if (q < kLA) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(f.a, mma_part<T, 2 * st>() + 1024 * (kLA * wave + q), 16, (int)aoff[q],
                                               0, 0, 0);
    } else {
      const int i = q - kLA;
      const uint32_t off = kBSlow && f.last ? blast[i] : boff[i];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(f.b, mma_part<T, 2 * st + 1>() + 1024 * (kLB * wave + i), 16, (int)off,
                                               0, 0, 0);
    }
  };

  // Fragments: [set][tile][chunk].  Phase kk of a step takes 32 bytes a lane
  // and tile, the chunks 4 kk + 2 half + {0, 1} of a minor row: for BF16 the
  // k 32 kk + 16 half + 8 {0, 1} + 0..7, which slow panels are read at too.
  // (Offsets are single opaque values: the compiler follows an address back
  // over a few additions only.)
  uint4 fa[2][kI][2], fb[2][kJ][2];
  const int t16 = lane & 15, col16 = (lane >> 4) & 1;
  // minor: the first tile's chunks of phase 0 ([e]; phase 1 flips bit 6), other
  // tiles 4096 bytes further; slow: the tiles ([i], [j]), phases and chunks
  // whole rows further
  int a_at[kASlow ? kI : 2], b_at[kBSlow ? kJ : 2];
  auto slow_at = [&](int first, int cols) __attribute__((always_inline)) {
    const int c = first + 16 * col16 + 4 * (t16 & 3), k = 16 * half + (t16 >> 2);
    return k * 2 * cols + 64 * slow_chunk(k, c >> 5) + 2 * (c & 31);
  };
  auto minor_at = [&](int first, int e) __attribute__((always_inline)) {
    return 128 * (first + l32) + 16 * ((2 * half + e) ^ minor_swz(l32));
  };
#pragma unroll
  for (int i = 0; i < (kASlow ? kI : 2); ++i) {
    a_at[i] = kASlow ? slow_at(32 * (kI * wm + i), T::kBM) : minor_at(32 * kI * wm, i);
    asm volatile("" : "+v"(a_at[i]));
  }
#pragma unroll
  for (int j = 0; j < (kBSlow ? kJ : 2); ++j) {
    b_at[j] = kBSlow ? slow_at(32 * (kJ * wn + j), T::kBN) : minor_at(32 * kJ * wn, j);
    asm volatile("" : "+v"(b_at[j]));
  }
  auto slow4 = [&](const uint8_t* panel, int at) __attribute__((always_inline)) {
    const v4s v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(panel + at));
    return __builtin_bit_cast(uint2, v);
  };
  // Reads of a phase: first the chunks 0 of every tile, B before A, then the
  // chunks 1; a chunk of a slow panel is two reads.
  constexpr int kNA = kASlow ? 2 : 1, kNB = kBSlow ? 2 : 1, kSet = kJ * kNB + kI * kNA, kR = 2 * kSet;
  auto read1 = [&](int f, const uint8_t* As, const uint8_t* Bs, int kk, int r) __attribute__((always_inline)) {
    const int e = r / kSet, t = r % kSet;
    if (t < kJ * kNB) {
      const int j = t / kNB;
      if constexpr (kBSlow) {
        const uint2 v = slow4(Bs, b_at[j] + (32 * kk + 8 * e + 4 * (t % 2)) * 2 * T::kBN);
        if (t % 2 == 0) fb[f][j][e].x = v.x, fb[f][j][e].y = v.y;
        else fb[f][j][e].z = v.x, fb[f][j][e].w = v.y;
      } else {
        fb[f][j][e] = *reinterpret_cast<const uint4*>(Bs + (b_at[e] ^ (64 * kk)) + 4096 * j);
      }
    } else {
      const int u = t - kJ * kNB, i = u / kNA;
      if constexpr (kASlow) {
        const uint2 v = slow4(As, a_at[i] + (32 * kk + 8 * e + 4 * (u % 2)) * 2 * T::kBM);
        if (u % 2 == 0) fa[f][i][e].x = v.x, fa[f][i][e].y = v.y;
        else fa[f][i][e].z = v.x, fa[f][i][e].w = v.y;
      } else {
        fa[f][i][e] = *reinterpret_cast<const uint4*>(As + (a_at[e] ^ (64 * kk)) + 4096 * i);
      }
    }
  };
  auto as_v8 = [](const uint4* v) __attribute__((always_inline)) {
    return v8i{(int)v[0].x, (int)v[0].y, (int)v[0].z, (int)v[0].w,
               (int)v[1].x, (int)v[1].y, (int)v[1].z, (int)v[1].w};
  };
  constexpr int kTiles = kI * kJ, kMF = kFP8 ? kTiles : 2 * kTiles;
  constexpr int kRF = kMF - kMF / 8;   // MFMAs that reads go out behind
  // Loads behind an MFMA.  All waves' loads go out after the same barrier, and
  // a wave whose load has to queue issues nothing else: one behind each of a
  // phase's 16 MFMAs of BF16 rather than two takes 4% fewer cycles (loss of
  // 8192 x 32000 x 4096: 1581 -> 1561 us at a lower clock, with the gradients
  // 4925 -> 4851; behind every second 1572 and 4906).  Of codes, with half the
  // MFMAs, two (795 us, one 802).
  constexpr int kPer = kFP8 ? 2 : 1;
  static_assert(kPer * kMF >= kL, "a phase issues a stage's loads");
  auto mma1 = [&](int f, int n) __attribute__((always_inline)) {
    const int i = n % kTiles / kJ, j = n % kJ, e = n / kTiles;
    if constexpr (kFP8)
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(as_v8(fb[f][j]), as_v8(fa[f][i]), acc[i][j], 0, 0, 0,
                                                                  0, 0, 0);
    else
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, fb[f][j][e]),
                                                          __builtin_bit_cast(v8bf, fa[f][i][e]), acc[i][j], 0, 0, 0);
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
      for (int q = kPer * n; q < kPer * n + kPer; ++q)
        if (q < kL) load1(next, S, q);
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
__device__ __forceinline__ void mma_stream(v16f (&acc)[T::kI][T::kJ], int steps, const uint8_t* a,
                                           const uint32_t (&aoff)[T::kLA], const uint8_t* b,
                                           const uint32_t (&boff)[T::kLB]) {
#if __HIP_DEVICE_COMPILE__
  constexpr int kI = T::kI, kJ = T::kJ, kLA = T::kLA, kLB = T::kLB, kL = kLA + kLB, kS = T::kStages;
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
// rows.  word(i, j, q) gives the four values of a run, packed; out(row, chunk,
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
  const int wm = wave % T::kWM, wn = wave / T::kWM, half = lane >> 5, l32 = lane & 31;
  auto part = [](int q) __attribute__((always_inline)) {
    return q == 0 ? mma_part<T, 0>() : q == 1 ? mma_part<T, 1>() : q == 2 ? mma_part<T, 2>() : mma_part<T, 3>();
  };
  auto at = [](int row, int c) __attribute__((always_inline)) { return row % kRows * kRowBytes + 16 * (c ^ (row & kMask)); };
#pragma unroll
  for (int i = 0; i < T::kI; ++i) {
    const int first = 32 * (T::kI * wm + i), row = first + l32;
    uint8_t* tile = part(first / kRows);
#pragma unroll
    for (int j = 0; j < T::kJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        *reinterpret_cast<uint2*>(tile + at(row, 4 * (T::kJ * wn + j) + q) + 8 * half) = word(i, j, q);
        if (q % 2) __builtin_amdgcn_sched_barrier(0);   // (or every word is begun before one is stored)
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

// The value at column `col` (of the wave's 32 kJ, in the lane's half) of the
// lane's row of tile i: a tree of selections by the column's bits, each a
// mask.  (Of conditions the compiler makes searches through whole vectors.)
template <class T>
__device__ __forceinline__ float value_at(const v16f (&acc)[T::kI][T::kJ], int i, int col) {
  static_assert(T::kJ == 1 || T::kJ == 2 || T::kJ == 4, "a power of two");
  uint32_t mask[6];
  constexpr int kBit[6] = {0, 1, 3, 4, 5, 6};
#pragma unroll
  for (int b = 0; b < 6; ++b) {
    mask[b] = 0u - (uint32_t)((col >> kBit[b]) & 1);
    asm volatile("" : "+v"(mask[b]));
  }
  auto pick = [&](int b, uint32_t zero, uint32_t one) __attribute__((always_inline)) {
    return (one & mask[b]) | (zero & ~mask[b]);
  };
  uint32_t of_j[T::kJ];
#pragma unroll
  for (int j = 0; j < T::kJ; ++j) {
    uint32_t of_q[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      auto bits = [&](int e) __attribute__((always_inline)) { return __float_as_uint(acc[i][j][4 * q + e]); };
      of_q[q] = pick(1, pick(0, bits(0), bits(1)), pick(0, bits(2), bits(3)));
    }
    of_j[j] = pick(3, pick(2, of_q[0], of_q[1]), pick(2, of_q[2], of_q[3]));
  }
  if constexpr (T::kJ == 4) return __uint_as_float(pick(5, pick(4, of_j[0], of_j[1]), pick(4, of_j[2], of_j[3])));
  if constexpr (T::kJ == 2) return __uint_as_float(pick(4, of_j[0], of_j[1]));
  return __uint_as_float(of_j[0]);
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
