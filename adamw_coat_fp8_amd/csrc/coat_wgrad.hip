// coat_wgrad.hip -- gfx950 weight gradient of a linear layer whose input was
// kept in E4M3, and its C ABI.
//
// Sources (see include/coat_fp8.h for the full citations):
//   [P1] COAT paper review (xllm-io.github.io), section 三: linear layers keep
//        their input in E4M3 (混合粒度激活量化) and the backward pass computes
//        the weight gradient from it.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "coat_elem.h"

using namespace coat;

namespace {

// dW[n][k] = sum over rows m of dy[m][n] x[m][k],  x[m][k] = code[m][k] S
//
// A product whose contracted axis is the slow one of both operands: the MFMA
// wants eight consecutive m of one column in a lane.  Both panels go from
// global memory straight into the LDS as they lie (dy in BF16, x as codes),
// and the LDS's transposing reads (16-bit for dy, 8-bit for the codes) hand
// each lane its column.  The codes become BF16 in registers, on the way into
// the MFMA: under one scale their values are exact in BF16 and the scale
// multiplies the FP32 result; with group scales, which change along m, the
// product code * S is rounded to BF16 (by up to 2^-8 of a value that E4M3 had
// already rounded by up to 2^-4).  That rounding alone leaves a relative error
// of 1.7e-3 (norms, random scales): as much as rounding the result to BF16
// does, 2.3e-3 together, and all the error of an FP32 result.  So an FP32
// result takes code * S in two BF16 parts (the second what the first left) and
// two MFMAs: 2.6e-6, at 1.78 times the time (8192 x 4096 x 4096, G = 128: 403 us
// against 226); a BF16 result takes one.  Sums are FP32 in the matrix cores.
//
// A block computes a kBN x kBK tile of dW; kWN x kWK waves own kJ x kI tiles
// of 32 x 32.  64 rows a step, three LDS stages.  A step is four substeps of
// 16 rows; while the MFMAs of one run, the fragments of the next are read and
// its codes expanded.  Before the last substep every wave waits for its reads
// of the step's stage and for its loads into the next one, and the block
// meets at the step's one barrier: the last substep then reads ahead from the
// next stage, and the loads of step t + 3 go into the one just read, so each
// load has two steps and more to arrive.
//
// Bound by the matrix cores and the power they may draw: 8192 x 22016 x 4096
// under one scale takes 1021 us (1.446 PFLOP/s; timed in turn with it, a
// library product of the same sizes in BF16 takes 1048 us with both operands
// contraction-minor and 1402 as they lie here; 1015 to 1078 us from one run and
// card to the next, up to 1257 in single calls after a pause), the MFMAs busy
// 81% of the cycles at about 1.7 GHz.  With group scales the expansion is 16
// vector instructions a fragment and not 4, and takes 1252 us (1.18 PFLOP/s),
// with an FP32 result 2185.  A 128 x 128 tile by eight waves of
// 64 x 32 is bound by LDS reads (2048 cubed: 21.2 us against 19.9).

constexpr int kStep = 64;   // rows per pipeline step

typedef short v4s __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));

enum Out { kBF16 = 0, kF32 = 1, kF32Add = 2, kPartial = 3 };

struct WgradParams {
  const uint16_t* dy;
  const uint8_t* codes;
  const float* scales;   // rows x K/G, or NULL: `scale` for all
  void* dw;              // N x K, or the partial sums (splits x N x K)
  int64_t M, N, K;
  int64_t groups;        // K / G
  int32_t n_tiles, k_tiles;
  int32_t steps;         // steps of all rows, ceil(M / 64)
  int32_t splits;
  int32_t whole;         // tiles of the order computed whole; each later one as two halves
  int32_t out;
  float scale;
};

// kLds: bytes of a stage's dy panel in the LDS, or 0 for what the tile needs.
template <int kWN_, int kWK_, int kJ_, int kI_, int kLds = 0>
struct Tile {
  static constexpr int kWN = kWN_, kWK = kWK_, kJ = kJ_, kI = kI_;
  static constexpr int kWaves = kWN * kWK, kThreads = 64 * kWaves;
  static constexpr int kBN = 32 * kWN * kJ, kBK = 32 * kWK * kI;
  static constexpr int kA = kStep * kBN * 2, kB = kStep * kBK;   // bytes of a stage's panels
  static constexpr int kLA = kA / 1024 / kWaves, kLB = kB / 1024 / kWaves;
  static constexpr int kLdsA = kLds ? kLds : kA;
};

// A dy row holds kBN values; its 64-byte chunks are XORed with m % 4, so that
// a transposing read's 4 rows x 64 bytes (32 lanes) meet all 64 banks once.
// (Rows are a multiple of 256 bytes.)
__device__ __forceinline__ int dy_chunk(int m, int c64) { return c64 ^ (m & 3); }

// A code row holds kBK bytes, 256 or 128; an 8-bit read's 8 rows x 32 bytes
// meet all banks once when the 32-byte chunks are XORed with m % 8, or for
// 128-byte rows, two to a sweep of the banks, with (m / 2) % 4.
template <int kBK>
__device__ __forceinline__ int code_chunk(int m, int c32) {
  return kBK == 256 ? c32 ^ (m & 7) : c32 ^ ((m >> 1) & 3);
}

template <class T, int G>
struct Stage {
  static constexpr int kGroups = G ? T::kBK / G : 0;                             // of a tile's row
  static constexpr int kLS = G ? (kGroups + T::kWaves - 1) / T::kWaves : 0;      // scale loads of a wave
  static constexpr int kSlots = kLS * T::kWaves;
};

// LDS arrays of the three stages: the dy panel, and the code panel with the
// scales behind it.  They are distinct objects: the compiler can tell the
// loads into one stage from the reads of another and does not wait for loads
// in flight.  (It follows a read's address back over a few additions only, so
// the lane's offsets below are single opaque values, and it keeps apart seven
// such objects at most.)
template <int kBytes, int kWhich>
__device__ __forceinline__ uint8_t* lds_array() {
  __shared__ __attribute__((aligned(1024))) uint8_t bytes[kBytes];
  return bytes;
}

template <class T, int kSt>
__device__ __forceinline__ uint8_t* dy_stage() { return lds_array<T::kLdsA, kSt>(); }

template <class T, int G, int kSt>
__device__ __forceinline__ uint8_t* code_stage() { return lds_array<T::kB + 256 * Stage<T, G>::kSlots, 3 + kSt>(); }

// Load q of a wave's loads of a step, into stage kSt: dy, codes, scales.  `off`
// are the lane's byte offsets from the step's first row.  kLast: the step may
// end past row M - 1, and those rows re-load it; or lie at or past step1, and
// then every lane loads the first bytes of the last step, which nothing reads:
// the number of loads in flight does not depend on the step.
template <class T, int G, int kSt, bool kLast>
__device__ __forceinline__ void load_one(const WgradParams& p, int step, int step1, int wave, int lane, int q,
                                         const uint32_t (&off)[T::kLA + T::kLB + Stage<T, G>::kLS]) {
#if __HIP_DEVICE_COMPILE__   // (the host has no type for a buffer's description)
  const int64_t m0 = (int64_t)(kLast && step >= step1 ? step1 - 1 : step) * kStep;
  const int last = (int)(p.M - m0 < kStep ? p.M - m0 : kStep) - 1;
  auto at = [&](int row, uint32_t stride) __attribute__((always_inline)) {
    if constexpr (!kLast) return (int)off[q];
    const uint32_t back = row > last ? (uint32_t)(row - last) * stride : 0u;
    return (int)(off[q] - back) & ((step - step1) >> 31);   // 0 where step >= step1
  };
  if (q < T::kLA) {
    const int row = (1024 * (T::kLA * wave + q) + 16 * lane) / (2 * T::kBN);
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)(p.dy + m0 * p.N), (short)0, (int)0xFFFFFFFF, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dy_stage<T, kSt>() + 1024 * (T::kLA * wave + q), 16,
                                             at(row, 2u * (uint32_t)p.N), 0, 0, 0);
  } else if (q < T::kLA + T::kLB) {
    const int i = q - T::kLA, row = (1024 * (T::kLB * wave + i) + 16 * lane) / T::kBK;
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)(p.codes + m0 * p.K), (short)0, (int)0xFFFFFFFF, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, code_stage<T, G, kSt>() + 1024 * (T::kLB * wave + i), 16,
                                             at(row, (uint32_t)p.K), 0, 0, 0);
  } else {
    const int i = q - T::kLA - T::kLB;
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)(p.scales + m0 * p.groups), (short)0, (int)0xFFFFFFFF, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, code_stage<T, G, kSt>() + T::kB + 256 * (Stage<T, G>::kLS * wave + i), 4,
                                             at(lane, 4u * (uint32_t)p.groups), 0, 0, 0);
  }
#endif
}

// Between a wave's writes to its part of the LDS and its reads of what other
// lanes wrote there (and back): nothing for the hardware, which keeps a wave's
// accesses in order, but the compiler may otherwise exchange them.
__device__ __forceinline__ void wave_meet() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// xcd_contiguous for 32-bit indexes.
__device__ __forceinline__ uint32_t xcd_contiguous32(uint32_t b, uint32_t nb) {
  const uint32_t q = nb / 8, r = nb % 8, xcd = b % 8, local = b / 8;
  return xcd < r ? xcd * (q + 1) + local : r * (q + 1) + (xcd - r) * q + local;
}

// Computes the tile of dW at (n0, k0), over the steps of `part`.  G = 0: one
// scale.  kFine: X in two BF16 parts.
template <class T, int G, bool kFine>
__device__ __forceinline__ void wgrad_tile(const WgradParams& p, const int64_t n0, const int64_t k0, const uint32_t part) {
  using S = Stage<T, G>;
  constexpr int kBN = T::kBN, kBK = T::kBK, kWK = T::kWK, kJ = T::kJ, kI = T::kI;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / kWK, wk = wave % kWK;
  const int step0 = p.splits == 1 ? 0 : (int)((int64_t)p.steps * part / p.splits);
  const int step1 = p.splits == 1 ? p.steps : (int)((int64_t)p.steps * (part + 1) / p.splits);

  // Loads.  A wave-wide 16-byte load fills 1 KB of a panel, lane L at byte
  // 16 L; the swizzles act on the global side.  Rows past M re-load row M - 1
  // (their dy is cleared below), columns past N or K the last whole chunk
  // (they reach only results that are not stored): no address is out of
  // range.  Slot g of the scales holds those of group g for the step's 64
  // rows; slots past the tile's groups repeat them, so that every wave issues
  // as many loads.
  const int64_t N = p.N, K = p.K, M = p.M;
  constexpr int kL = T::kLA + T::kLB + S::kLS;
  uint32_t off[kL];
#pragma unroll
  for (int i = 0; i < T::kLA; ++i) {
    const int byte = 1024 * (T::kLA * wave + i) + 16 * lane, m = byte / (2 * kBN), c16 = byte % (2 * kBN) / 16;
    const int64_t n = n0 + 8 * (4 * dy_chunk(m, c16 >> 2) + (c16 & 3));
    off[i] = 2u * ((uint32_t)m * (uint32_t)N + (uint32_t)(n < N ? n : N - 8));
  }
#pragma unroll
  for (int i = 0; i < T::kLB; ++i) {
    const int byte = 1024 * (T::kLB * wave + i) + 16 * lane, m = byte / kBK, c16 = byte % kBK / 16;
    const int64_t k = k0 + 16 * (2 * code_chunk<kBK>(m, c16 >> 1) + (c16 & 1));
    off[T::kLA + i] = (uint32_t)m * (uint32_t)K + (uint32_t)(k < K ? k : K - 16);
  }
  if constexpr (G != 0) {
#pragma unroll
    for (int i = 0; i < S::kLS; ++i) {
      const int64_t g = (uint32_t)k0 / G + (S::kLS * wave + i) % S::kGroups;
      off[T::kLA + T::kLB + i] =
          4u * ((uint32_t)lane * (uint32_t)p.groups + (uint32_t)(g < p.groups ? g : p.groups - 1));
    }
  }
  // s_waitcnt immediates that leave the loads of two or one steps in flight,
  // and lgkmcnt(0): the wave's reads of the stage that is loaded next are done
  // (vmcnt in bits 3:0 and 15:14, expcnt in 6:4, lgkmcnt in 11:8)
  static_assert(2 * kL < 64, "vmcnt holds at most 63");
  constexpr int kTwoStepsInFlight = (2 * kL & 15) | ((2 * kL >> 4) << 14) | (7 << 4);
  constexpr int kOneStepInFlight = (kL & 15) | ((kL >> 4) << 14) | (7 << 4);

  v16f acc[kI][kJ];
#pragma unroll
  for (int i = 0; i < kI; ++i)
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // Fragment reads.  16 lanes of a transposing read share a block: for 16-bit
  // values 4 rows x 16 columns (lane t points at row t / 4, values 4 (t % 4)),
  // for codes 8 rows x 16 columns (row t / 2, bytes 8 (t % 2)); lane t
  // receives column t.  Lanes 0-31 cover 32 columns of rows 0-7 of a 16-row
  // substep, lanes 32-63 rows 8-15.
  const int t16 = lane & 15, col16 = (lane >> 4) & 1, half = lane >> 5;
  v4s dlo[2][kJ], dhi[2][kJ];   // dy fragments of two substeps
  v2i xw[kI];                   // codes of the substep being read
  float4 slo[kI], shi[kI];      // and their scales
  u32x4v x[2][kI];
  u32x4v rest[kFine ? 2 : 1][kI];   // what BF16 left of x
  int dy_off[kJ], x_off[kI], s_off[kI];
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int c = 32 * (wn * kJ + j) + 16 * col16 + 4 * (t16 & 3), m = 8 * half + (t16 >> 2);
    dy_off[j] = m * 2 * kBN + 64 * dy_chunk(m, c >> 5) + 2 * (c & 31);
    asm volatile("" : "+v"(dy_off[j]));
  }
#pragma unroll
  for (int i = 0; i < kI; ++i) {
    const int c = 32 * (wk * kI + i) + 16 * col16 + 8 * (t16 & 1), m = 8 * half + (t16 >> 1);
    x_off[i] = m * kBK + 32 * code_chunk<kBK>(m, c >> 5) + (c & 31);
    asm volatile("" : "+v"(x_off[i]));
    s_off[i] = G ? T::kB + 4 * (64 * ((32 * (wk * kI + i) + (lane & 31)) / (G ? G : 1)) + 8 * half) : 0;
    if constexpr (G != 0) asm volatile("" : "+v"(s_off[i]));
  }
  // (the swizzles repeat every 4 and 8 rows: a substep is 16 further, the
  // second half of a dy fragment 4)
  auto read_dy = [&](const uint8_t* panel, int f, int s, int j, int high) __attribute__((always_inline)) {
    (high ? dhi : dlo)[f][j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4s*)(panel + (dy_off[j] + (16 * s + 4 * high) * 2 * kBN)));
  };
  auto read_x = [&](const uint8_t* panel, int s, int i) __attribute__((always_inline)) {
    xw[i] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
        (__attribute__((address_space(3))) v2i*)(panel + (x_off[i] + 16 * s * kBK)));
    if (G != 0 && (i == 0 || G < 32 * kI)) {   // (a wave's columns may share their group)
      slo[i] = *reinterpret_cast<const float4*>(panel + (s_off[i] + 64 * s));
      shi[i] = *reinterpret_cast<const float4*>(panel + (s_off[i] + 64 * s + 16));
    }
  };
  // Dword q of fragment i: two values.
  auto expand = [&](int f, int i, int q) __attribute__((always_inline)) {
    if constexpr (G == 0) {
      x[f][i][q] = __builtin_bit_cast(uint32_t, q & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(xw[i][q / 2], 1.0f, true)
                                                      : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(xw[i][q / 2], 1.0f, false));
    } else {
      const int g = G >= 32 * kI ? 0 : i;
      const auto v = q & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(xw[i][q / 2], true) : __builtin_amdgcn_cvt_pk_f32_fp8(xw[i][q / 2], false);
      const float4 sc = q < 2 ? slo[g] : shi[g];
      const float v0 = v[0] * (q & 1 ? sc.z : sc.x), v1 = v[1] * (q & 1 ? sc.w : sc.y);
      const uint32_t w = bf16_pack2(v0, v1);
      x[f][i][q] = w;
      if constexpr (kFine) rest[f][i][q] = bf16_pack2(v0 - bf16_lo(w), v1 - bf16_hi(w));
    }
  };
  auto mma = [&](int f, int n) __attribute__((always_inline)) {
    const int i = n / kJ, j = n % kJ;
    const v8bf d = __builtin_bit_cast(v8bf, __builtin_shufflevector(dlo[f][j], dhi[f][j], 0, 1, 2, 3, 4, 5, 6, 7));
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, x[f][i]), d, acc[i][j], 0, 0, 0);
    if constexpr (kFine)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, rest[f][i]), d, acc[i][j], 0, 0, 0);
  };
  // The MFMAs of fragment set f, with substep s of a stage read into the other
  // set between them: the codes first, expanded dword by dword behind the
  // later MFMAs.
  constexpr int kMF = kI * kJ, kR = 2 * kJ, kE = 4 * kI, kFirst = kMF > 4 ? 3 : 1;
  auto substep = [&](int f, const uint8_t* a, const uint8_t* b, int s, auto also) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < kMF; ++n) {
      mma(f, n);
      if (n == 0) {
#pragma unroll
        for (int i = 0; i < kI; ++i) read_x(b, s, i);
      }
#pragma unroll
      for (int r = n * kR / kMF; r < (n + 1) * kR / kMF; ++r) read_dy(a, 1 - f, s, r / 2, r % 2);
      if (n >= kFirst) {
#pragma unroll
        for (int e = (n - kFirst) * kE / (kMF - kFirst); e < (n - kFirst + 1) * kE / (kMF - kFirst); ++e)
          expand(1 - f, e / 4, e % 4);
      }
      also(n);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto nothing = [](int) __attribute__((always_inline)) {};
  // Clears dy past row M - 1 in the stage of a step, behind its barrier.
  auto clear_tail = [&](int step, uint8_t* a) __attribute__((always_inline)) {
    if (M - (int64_t)step * kStep < kStep) {
      const int valid = (int)(M - (int64_t)step * kStep);
      for (int o = valid * 2 * kBN + 16 * (int)threadIdx.x; o < T::kA; o += 16 * T::kThreads)
        *reinterpret_cast<uint4*>(a + o) = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
  };
  auto meet = [&](auto wait) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(decltype(wait)::value);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
  };
  // last: the step's successors may be the last step or none
  auto run = [&](int step, auto st, auto next, auto last) __attribute__((always_inline)) {
    constexpr bool kLast = decltype(last)::value;
    constexpr int kSt = decltype(st)::value, kNext = decltype(next)::value;
    const uint8_t* a = dy_stage<T, kSt>();
    const uint8_t* b = code_stage<T, G, kSt>();
    substep(0, a, b, 1, nothing);
    substep(1, a, b, 2, nothing);
    substep(0, a, b, 3, nothing);
    uint8_t* an = dy_stage<T, kNext>();
    meet(std::integral_constant<int, kOneStepInFlight>{});
    if constexpr (kLast) {
      if (step + 1 < step1) clear_tail(step + 1, an);
    }
    // (behind the last step this reads a stage that nothing uses)
    substep(1, an, code_stage<T, G, kNext>(), 0, [&](int n) __attribute__((always_inline)) {
#pragma unroll
      for (int q = n * kL / kMF; q < (n + 1) * kL / kMF; ++q)
        load_one<T, G, kSt, kLast>(p, step + 3, step1, wave, lane, q, off);
    });
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
#pragma unroll
  for (int q = 0; q < kL; ++q) load_one<T, G, 0, true>(p, step0, step1, wave, lane, q, off);
#pragma unroll
  for (int q = 0; q < kL; ++q) load_one<T, G, 1, true>(p, step0 + 1, step1, wave, lane, q, off);
#pragma unroll
  for (int q = 0; q < kL; ++q) load_one<T, G, 2, true>(p, step0 + 2, step1, wave, lane, q, off);
  meet(std::integral_constant<int, kTwoStepsInFlight>{});
  clear_tail(step0, dy_stage<T, 0>());
#pragma unroll
  for (int i = 0; i < kI; ++i) read_x(code_stage<T, G, 0>(), 0, i);
#pragma unroll
  for (int r = 0; r < kR; ++r) read_dy(dy_stage<T, 0>(), 0, 0, r / 2, r % 2);
#pragma unroll
  for (int e = 0; e < kE; ++e) expand(0, e / 4, e % 4);
  int step = step0;
  for (; step + 6 < step1; step += 3) {
    run(step, C0{}, C1{}, std::false_type{});
    run(step + 1, C1{}, C2{}, std::false_type{});
    run(step + 2, C2{}, C0{}, std::false_type{});
  }
  // the last one to six steps, without a loop (where paths of different
  // lengths meet, the compiler waits for every load)
  auto last_steps = [&](auto self, int s, auto st, auto left) __attribute__((always_inline)) -> void {
    constexpr int kSt = decltype(st)::value, kLeft = decltype(left)::value;
    using Next = std::integral_constant<int, (kSt + 1) % 3>;
    if (s >= step1) return;
    run(s, st, Next{}, std::true_type{});
    if constexpr (kLeft > 1) self(self, s + 1, Next{}, std::integral_constant<int, kLeft - 1>{});
  };
  last_steps(last_steps, step, C0{}, std::integral_constant<int, 6>{});
  __builtin_amdgcn_s_waitcnt(7 << 4 | 15 << 8);   // no load into the LDS outlives the block

  // Epilogue.  Register 4 q + e of acc[i][j] is dW[n][k] with
  //   n = n0 + 32 (wn kJ + j) + lane % 32,  k = k0 + 32 (wk kI + i) + 8 q + 4 half + e,
  // runs of four k a lane.  Each wave passes its tile through a part of the
  // LDS of its own, in rows of 128 bytes (64 values in BF16, in one pass; 32 in
  // FP32, a pass for each i), and stores whole 128-byte lines.  (Stores of the
  // runs as they are took 3.7 us of a 7.8 us call of one step.)  The 16-byte
  // chunks are XORed with row % 8, and on rows with bit 3 set the 8-byte halves
  // of a chunk swapped: 8-byte writes go 16 rows at a time, 16-byte writes and
  // reads 8 chunks, each time all of 128 different bytes of the banks (counted:
  // no conflicts; XORed with row / 2 % 8, two rows met, 4 cycles a write).
  __syncthreads();   // every wave is done with the stages
  constexpr int kRows = 32 * kJ, kBytes = 128 * kRows, kPer = T::kLdsA / kBytes;
  uint8_t* own = wave < kPer       ? dy_stage<T, 0>() + kBytes * wave
                 : wave < 2 * kPer ? dy_stage<T, 1>() + kBytes * (wave - kPer)
                                   : dy_stage<T, 2>() + kBytes * (wave - 2 * kPer);
  if constexpr (T::kWaves > 3 * kPer) {
    static_assert(T::kWaves <= 3 * kPer + 2 && T::kB >= kBytes, "a code panel holds one wave's tile");
    if (wave == 3 * kPer) own = code_stage<T, G, 0>();
    if (wave == 3 * kPer + 1) own = code_stage<T, G, 1>();
  }
  const float scale = p.out == kPartial ? 1.0f : p.scale;
  const int64_t wave_n = n0 + kRows * wn, wave_k = k0 + 32 * kI * wk;
  auto chunk_at = [&](int row, int c) __attribute__((always_inline)) { return 128 * row + 16 * (c ^ (row & 7)); };
  // each 16-byte chunk of the staged rows: fn(row, chunk of the row, its bytes)
  auto rows_out = [&](auto fn) __attribute__((always_inline)) {
    wave_meet();
#pragma unroll
    for (int r = 0; r < kRows / 8; ++r) {
      const int row = 8 * r + (lane >> 3), c = lane & 7;
      uint4 v = *reinterpret_cast<const uint4*>(own + chunk_at(row, c));
      fn(row, c, v);
    }
  };
  if (p.out == kBF16) {
    static_assert(kI == 2, "64 values of k a wave");
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = 32 * j + (lane & 31);
          *reinterpret_cast<uint2*>(own + chunk_at(row, 4 * i + q) + 8 * (half ^ ((row >> 3) & 1))) =
              make_uint2(bf16_pack2(acc[i][j][4 * q] * scale, acc[i][j][4 * q + 1] * scale),
                         bf16_pack2(acc[i][j][4 * q + 2] * scale, acc[i][j][4 * q + 3] * scale));
        }
    rows_out([&](int row, int c, uint4 v) __attribute__((always_inline)) {
      if ((row >> 3) & 1) v = make_uint4(v.z, v.w, v.x, v.y);
      const int64_t n = wave_n + row, k = wave_k + 8 * c;
      if (n < N && k < K) store_stream16((uint16_t*)p.dw + n * K + k, v);
    });
  } else {
    float* dw = (float*)p.dw + (p.out == kPartial ? part * N * K : 0);
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      if (i > 0) wave_meet();   // the rows of the last pass are read
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float4*>(own + chunk_at(32 * j + (lane & 31), 2 * q + half)) =
              make_float4(acc[i][j][4 * q] * scale, acc[i][j][4 * q + 1] * scale, acc[i][j][4 * q + 2] * scale,
                          acc[i][j][4 * q + 3] * scale);
      rows_out([&](int row, int c, uint4 v) __attribute__((always_inline)) {
        const int64_t n = wave_n + row, k = wave_k + 32 * i + 4 * c;
        if (n >= N || k >= K) return;
        float4* dst = reinterpret_cast<float4*>(dw + n * K + k);
        float4 f = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
        if (p.out == kF32Add) {
          const float4 old = *dst;
          f = make_float4(old.x + f.x, old.y + f.y, old.z + f.z, old.w + f.w);
        }
        *dst = f;
      });
    }
  }
}

// Tile order: an XCD takes a contiguous run; inside it eight k tiles are
// walked for each n tile, so the 32 tiles an XCD works on at once share about
// 4 dy panels and 8 code panels (half as wide) in its L2.  (32-bit numbers: a
// block's share of them is scalar work of a few cycles.)
template <class T>
__device__ __forceinline__ void tile_at(const WgradParams& p, uint32_t local, int64_t& n0, int64_t& k0) {
  const uint32_t n_tiles = (uint32_t)p.n_tiles, k_tiles = (uint32_t)p.k_tiles;
  const uint32_t band = local / (8 * n_tiles), first_k = 8 * band;
  const uint32_t wide = k_tiles - first_k < 8 ? k_tiles - first_k : 8;
  const uint32_t in_band = local - band * 8 * n_tiles, row = in_band / wide;
  n0 = (int64_t)row * T::kBN;
  k0 = (int64_t)(first_k + in_band - row * wide) * T::kBK;
}

using Large = Tile<2, 4, 4, 2>;             // 256 x 256, eight waves of 128 x 64
using Half = Tile<2, 4, 2, 2, Large::kA>;   // 128 x 256, eight waves of 64 x 64
using Small = Tile<2, 2, 2, 2>;             // 128 x 128, four waves of 64 x 64

// Blocks 0 .. whole - 1 compute whole tiles, the blocks behind them halves of
// the remaining ones: a last round that would be at most half full takes half
// a round's time (1376 tiles on 256 compute units: 1067 us against 1105; 320
// tiles: 146 against 176).
template <int G, bool kFine>
__global__ __launch_bounds__(Large::kThreads) void wgrad_large_kernel(const WgradParams p) {
  int64_t n0, k0;
  const uint32_t b = blockIdx.x, whole = (uint32_t)p.whole;
  if (b < whole) {
    tile_at<Large>(p, xcd_contiguous32(b, whole), n0, k0);
    wgrad_tile<Large, G, kFine>(p, n0, k0, 0);
  } else {
    const uint32_t order = xcd_contiguous32(b - whole, gridDim.x - whole);
    tile_at<Large>(p, whole + (order >> 1), n0, k0);
    n0 += Half::kBN * (order & 1);
    if (n0 < p.N) wgrad_tile<Half, G, kFine>(p, n0, k0, 0);
  }
}

template <int G, bool kFine>
__global__ __launch_bounds__(Small::kThreads) void wgrad_small_kernel(const WgradParams p) {
  int64_t n0, k0;
  const uint32_t tiles = (uint32_t)p.n_tiles * (uint32_t)p.k_tiles;
  const uint32_t order = xcd_contiguous32(blockIdx.x, gridDim.x), part = order / tiles;
  tile_at<Small>(p, order - part * tiles, n0, k0);
  wgrad_tile<Small, G, kFine>(p, n0, k0, part);
}

// Adds the partial sums of the splits in order, scales and stores.
__global__ __launch_bounds__(256) void wgrad_join_kernel(const float* partials, int splits, int64_t size, void* dw,
                                                         int out, float scale) {
  const int64_t at = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (at >= size) return;
  float4 v = *reinterpret_cast<const float4*>(partials + at);
  for (int s = 1; s < splits; s += 8) {   // eight loads in flight at a time
    float4 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = s + i < splits ? *reinterpret_cast<const float4*>(partials + (s + i) * size + at) : make_float4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) v.x += o[i].x, v.y += o[i].y, v.z += o[i].z, v.w += o[i].w;
  }
  v.x *= scale, v.y *= scale, v.z *= scale, v.w *= scale;
  if (out == kBF16) {
    *reinterpret_cast<uint2*>((uint16_t*)dw + at) = make_uint2(bf16_pack2(v.x, v.y), bf16_pack2(v.z, v.w));
  } else {
    float4* dst = reinterpret_cast<float4*>((float*)dw + at);
    if (out == kF32Add) {
      const float4 old = *dst;
      v.x += old.x, v.y += old.y, v.z += old.z, v.w += old.w;
    }
    *dst = v;
  }
}

// No rows: the empty sum.
__global__ __launch_bounds__(256) void wgrad_zero_kernel(void* dw, int64_t bytes) {
  for (int64_t at = 16 * ((int64_t)blockIdx.x * 256 + threadIdx.x); at < bytes; at += 4096 * (int64_t)gridDim.x)
    *reinterpret_cast<uint4*>((uint8_t*)dw + at) = make_uint4(0, 0, 0, 0);
}

template <int G, bool kFine>
const void* wgrad_fn(bool large) {
  return large ? reinterpret_cast<const void*>(&wgrad_large_kernel<G, kFine>)
               : reinterpret_cast<const void*>(&wgrad_small_kernel<G, kFine>);
}

// g: the group size, 0 for one scale.
const void* wgrad_kernel_for(bool large, int32_t g, bool fine) {
  switch (g) {
    case 0: return wgrad_fn<0, false>(large);
    case 16: return fine ? wgrad_fn<16, true>(large) : wgrad_fn<16, false>(large);
    case 32: return fine ? wgrad_fn<32, true>(large) : wgrad_fn<32, false>(large);
    case 64: return fine ? wgrad_fn<64, true>(large) : wgrad_fn<64, false>(large);
    default: return fine ? wgrad_fn<128, true>(large) : wgrad_fn<128, false>(large);
  }
}

constexpr int64_t kMaxDim = 1 << 24;     // 64 rows of dy stay below 2^32 bytes
constexpr int64_t kMaxTiles = 1 << 23;   // of 128 x 128: a launch's threads stay below 2^32
constexpr int64_t kUnits = 256;          // compute units of the device the split is made for

struct Plan {
  bool large;
  int32_t n_tiles, k_tiles, splits;
};

// Small tiles as long as each has a compute unit to itself (2048 x 2048 over
// 8192 rows: 60 us, 69 as large ones).  Beyond that two share a unit, and large
// tiles, which read half as much a product and run as halves where there are
// few, are faster: 72 of them (2304 x 2048) 76 us against 88 as small ones, 121
// (2816 x 2816) 99 against 108, 240 (3840 x 4096) 181 against 211.  Not where
// they would multiply over a quarter more padding: 272 x 16640 takes 128 us in
// large tiles and 107 in small, 128 x 65536 198 and 152.  Where even small ones
// leave units empty and there are rows for it, the rows are split, 256 rows to
// a part at least, and the parts joined from the workspace.  A function of the
// sizes alone, so that the workspace and the order of the sums are.
Plan plan(int64_t M, int64_t N, int64_t K) {
  Plan p;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const int64_t small = up(N, Small::kBN) * up(K, Small::kBK);
  p.large = small > kUnits && 16 * up(N, Large::kBN) * up(K, Large::kBK) <= 5 * small;
  p.n_tiles = (int32_t)up(N, p.large ? Large::kBN : Small::kBN);
  p.k_tiles = (int32_t)up(K, p.large ? Large::kBK : Small::kBK);
  const int64_t tiles = (int64_t)p.n_tiles * p.k_tiles;
  int64_t splits = 1;
  if (!p.large && tiles < kUnits) {
    splits = kUnits / tiles;
    const int64_t most = M / 256;
    splits = splits < most ? splits : most;
    splits = splits < 1 ? 1 : splits;
  }
  p.splits = (int32_t)splits;
  return p;
}

bool wgrad_sizes_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && K >= 0 && N % 16 == 0 && K % 16 == 0 && N <= kMaxDim && K <= kMaxDim &&
         M <= (int64_t)kStep * 0x7FFFFFF0 && (N == 0 || K <= INT64_MAX / 8 / N) &&
         (N + 127) / 128 * ((K + 127) / 128) <= kMaxTiles;
}

}  // namespace

extern "C" {

int64_t coat_fp8_weight_grad_workspace(int64_t M, int64_t N, int64_t K) {
  if (!wgrad_sizes_ok(M, N, K)) return -1;
  if (M == 0 || N == 0 || K == 0) return 0;
  const Plan p = plan(M, N, K);
  return p.splits > 1 ? p.splits * N * K * (int64_t)sizeof(float) : 0;
}

coat_status_t coat_fp8_weight_grad(const coat_weight_grad_args_t* a, hipStream_t stream) {
  if (!a) return COAT_ERR_NULL_POINTER;
  const int64_t M = a->M, N = a->N, K = a->K;
  if (!wgrad_sizes_ok(M, N, K)) return COAT_ERR_INVALID_VALUE;
  if (a->x_scales && !valid_group_size(a->group_size)) return COAT_ERR_GROUP_SIZE;
  if (a->x_scales && K % a->group_size != 0) return COAT_ERR_INVALID_VALUE;
  if (!a->x_scales && !isfinite(a->x_scale)) return COAT_ERR_INVALID_VALUE;
  if (a->dw_bf16 && (a->dw_f32 || a->accumulate)) return COAT_ERR_INVALID_VALUE;
  if (N == 0 || K == 0) return COAT_OK;
  if (!a->dw_bf16 && !a->dw_f32) return COAT_ERR_NULL_POINTER;
  if (M > 0 && (!a->dy || !a->x_codes)) return COAT_ERR_NULL_POINTER;
  if (!aligned(a->dy, 16) || !aligned(a->x_codes, 16) || !aligned(a->x_scales, 4) || !aligned(a->dw_bf16, 16) ||
      !aligned(a->dw_f32, 16) || !aligned(a->workspace, 16))
    return COAT_ERR_MISALIGNED;
  void* dw = a->dw_bf16 ? (void*)a->dw_bf16 : (void*)a->dw_f32;
  const int out = a->dw_bf16 ? kBF16 : a->accumulate ? kF32Add : kF32;
  hipError_t e = hipSuccess;
  if (M == 0) {
    if (out == kF32Add) return COAT_OK;
    int64_t bytes = N * K * (a->dw_bf16 ? 2 : 4);
    const int64_t blocks = (bytes + 4095) / 4096;
    void* args[] = {&dw, &bytes};
    e = hipLaunchKernel(reinterpret_cast<const void*>(&wgrad_zero_kernel),
                        dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), args, 0, stream);
    return e == hipSuccess ? COAT_OK : hip_fail(e);
  }
  const Plan pl = plan(M, N, K);
  if (pl.splits > 1) {
    if (!a->workspace) return COAT_ERR_NULL_POINTER;
    if (a->workspace_bytes < coat_fp8_weight_grad_workspace(M, N, K)) return COAT_ERR_INVALID_VALUE;
  }
  WgradParams p;
  memset(&p, 0, sizeof(p));
  p.dy = a->dy;
  p.codes = a->x_codes;
  p.scales = a->x_scales;
  p.dw = pl.splits > 1 ? a->workspace : dw;
  p.M = M;
  p.N = N;
  p.K = K;
  p.groups = a->x_scales ? K / a->group_size : 0;
  p.n_tiles = pl.n_tiles;
  p.k_tiles = pl.k_tiles;
  p.steps = (int32_t)((M + kStep - 1) / kStep);
  p.splits = pl.splits;
  p.out = pl.splits > 1 ? (int)kPartial : out;
  p.scale = a->x_scales ? 1.0f : a->x_scale;
  void* args[] = {&p};
  // the last round of large tiles in halves where that fills it
  const int64_t tiles = (int64_t)pl.n_tiles * pl.k_tiles, rest = pl.large ? tiles % kUnits : 0;
  const int64_t halves = 2 * rest <= kUnits ? rest : 0;
  p.whole = (int32_t)(tiles - halves);
  e = hipLaunchKernel(wgrad_kernel_for(pl.large, a->x_scales ? a->group_size : 0, out != kBF16),
                      dim3((unsigned)((tiles + halves) * pl.splits)),
                      dim3(pl.large ? Large::kThreads : Small::kThreads), args, 0, stream);
  if (e == hipSuccess && pl.splits > 1) {
    const float* partials = (const float*)a->workspace;
    int splits = pl.splits, o = out;
    int64_t size = N * K;
    float scale = p.scale;
    void* join[] = {&partials, &splits, &size, &dw, &o, &scale};
    e = hipLaunchKernel(reinterpret_cast<const void*>(&wgrad_join_kernel), dim3((unsigned)((size + 1023) / 1024)),
                        dim3(256), join, 0, stream);
  }
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

}  // extern "C"
