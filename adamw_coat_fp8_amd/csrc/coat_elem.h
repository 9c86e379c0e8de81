// coat_elem.h -- device helpers of the activation kernels: eight-value chunks
// of a row, their E4M3 codes, and sums over lanes (not part of the C ABI).
#ifndef COAT_ELEM_H
#define COAT_ELEM_H

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "coat_common.h"

namespace coat {

typedef unsigned u32x2v __attribute__((ext_vector_type(2)));
typedef unsigned u32x4v __attribute__((ext_vector_type(4)));

// Streaming accesses: every byte is read or written once, so the loads and
// stores are nontemporal, as in the activation quantizer (whose own file has
// the measurement).
__device__ __forceinline__ uint4 load_stream16(const void* p) {
  const u32x4v v = __builtin_nontemporal_load(reinterpret_cast<const u32x4v*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}

__device__ __forceinline__ uint2 load_stream8(const void* p) {
  const u32x2v v = __builtin_nontemporal_load(reinterpret_cast<const u32x2v*>(p));
  return make_uint2(v.x, v.y);
}

__device__ __forceinline__ void store_stream8(void* p, uint2 v) {
  const u32x2v w = {v.x, v.y};
  __builtin_nontemporal_store(w, reinterpret_cast<u32x2v*>(p));
}

__device__ __forceinline__ void store_stream16(void* p, uint4 v) {
  const u32x4v w = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(w, reinterpret_cast<u32x4v*>(p));
}

// Largest BF16 magnitude (as its 15 bits) among the 8 values of a chunk:
// sign-cleared BF16 patterns order like the magnitudes they encode, two to a
// packed 16-bit maximum.
__device__ __forceinline__ uint32_t bf16x8_max_mag(uint4 r) {
  typedef uint16_t u16x2v __attribute__((ext_vector_type(2)));
  auto mag = [](uint32_t w) __attribute__((always_inline)) { return __builtin_bit_cast(u16x2v, w & 0x7FFF7FFFu); };
  const u16x2v m = __builtin_elementwise_max(__builtin_elementwise_max(mag(r.x), mag(r.y)),
                                             __builtin_elementwise_max(mag(r.z), mag(r.w)));
  return max((uint32_t)m[0], (uint32_t)m[1]);
}

// E4M3 codes of the group quotients of four BF16 values.
__device__ __forceinline__ uint32_t act_pack4(uint32_t w0, uint32_t w1, const GroupQuot& d) {
  const float q0 = group_quot(bf16_lo(w0), d), q1 = group_quot(bf16_hi(w0), d);
  const float q2 = group_quot(bf16_lo(w1), d), q3 = group_quot(bf16_hi(w1), d);
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(q0, q1, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(q2, q3, v, true);
  return (uint32_t)v;
}

// lanes_max_u32 for a group size known at run time only (uniform branches):
// `lanes` = group_size / 8, one of 2, 4, 8, 16.
__device__ __forceinline__ uint32_t group_max_u32(uint32_t v, int lanes) {
  v = lanes_max_u32<2>(v);
  if (lanes >= 4) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  if (lanes >= 8) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  if (lanes >= 16) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  return v;
}

// amax / 448 rounded as the IEEE division rounds it, for BF16 amax: one
// residual correction with the rounded reciprocal, which is exact for every
// BF16 value from 2^-100 up (checked value by value in the tests); the
// division below.
__device__ __forceinline__ float scale_of(float amax) {
  constexpr float kInv = 1.0f / 448.0f;
  if (amax < 0x1p-100f) return amax / 448.0f;
  const float q = amax * kInv;
  const float v = __builtin_fmaf(__builtin_fmaf(-q, 448.0f, amax), kInv, q);
  return v == v ? v : amax;   // infinity
}

// The checkpoint of one 8-value BF16 chunk whose group lies on `lanes`
// neighbouring lanes: its codes, and the group's scale max / 448.  The
// reciprocal in the quotients is the hardware's, one ulp off at most: ties
// stay exact under the correction in group_quot, and for BF16 values no other
// quotient lies close enough to a midpoint for it to matter.
__device__ __forceinline__ uint2 checkpoint8(uint4 raw, int lanes, float& scale) {
  const float amax = __uint_as_float(group_max_u32(bf16x8_max_mag(raw), lanes) << 16);
  const float pre = amax < 0x1p-100f ? 0x1p64f : 1.0f;
  GroupQuot d;
  d.c = 0.875f * pre;
  d.b = amax * pre * 0x1p-9f;
  d.r = __builtin_amdgcn_rcpf(d.b);
  scale = scale_of(amax);
  if (amax == 0.0f) return make_uint2(0, 0);
  return make_uint2(act_pack4(raw.x, raw.y, d), act_pack4(raw.z, raw.w, d));
}

__device__ __forceinline__ void unpack8(uint4 r, float (&f)[8]) {
  f[0] = bf16_lo(r.x), f[1] = bf16_hi(r.x), f[2] = bf16_lo(r.y), f[3] = bf16_hi(r.y);
  f[4] = bf16_lo(r.z), f[5] = bf16_hi(r.z), f[6] = bf16_lo(r.w), f[7] = bf16_hi(r.w);
}

// Two FP32 values rounded to BF16 (nearest even), the first in the low half.
__device__ __forceinline__ uint32_t bf16_pack2(float lo, float hi) {
  typedef float f32x2v __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
  const f32x2v f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2v));
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(bf16_pack2(f[0], f[1]), bf16_pack2(f[2], f[3]), bf16_pack2(f[4], f[5]),
                    bf16_pack2(f[6], f[7]));
}

// Values of four E4M3 codes.
__device__ __forceinline__ void e4m3_values4(uint32_t w, float* f) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  f[0] = lo[0], f[1] = lo[1], f[2] = hi[0], f[3] = hi[1];
}

__device__ __forceinline__ void e4m3_values8(uint2 c, float (&f)[8]) {
  e4m3_values4(c.x, f);
  e4m3_values4(c.y, f + 4);
}

// Largest magnitude of kN values (kN even); NaNs are not counted.
template <int kN>
__device__ __forceinline__ float max_mag(const float (&f)[kN]) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < kN; e += 2) m = fmaxf(fmaxf(m, fabsf(f[e])), fabsf(f[e + 1]));   // one v_max3
  return m;
}

// E4M3 codes of kN values already divided by their scale, saturating at
// +-448; a NaN stays one.  `top` is their largest magnitude: values inside
// the format's range skip the clamp.
template <int kN>
__device__ __forceinline__ void e4m3_pack(float (&f)[kN], float top, uint32_t (&w)[kN / 4]) {
  if (top > 448.0f) {
#pragma unroll
    for (int e = 0; e < kN; ++e) f[e] = f[e] != f[e] ? f[e] : __builtin_amdgcn_fmed3f(f[e], -448.0f, 448.0f);
  }
#pragma unroll
  for (int q = 0; q < kN / 4; ++q) {
    const int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * q], f[4 * q + 1], 0, false);
    w[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * q + 2], f[4 * q + 3], v, true);
  }
}

template <int kCtrl>
__device__ __forceinline__ float dpp_f32(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), kCtrl, 0xF, 0xF, false));
}

// Sum over kLanes neighbouring lanes (a power of two up to 64, aligned):
// quad swaps, the half-row and row mirrors, then the row and half-wave swaps.
// Every lane ends with the same sum, always formed in the same order.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (kLanes >= 2) v += dpp_f32<0xB1>(v);
  if constexpr (kLanes >= 4) v += dpp_f32<0x4E>(v);
  if constexpr (kLanes >= 8) v += dpp_f32<0x141>(v);
  if constexpr (kLanes >= 16) v += dpp_f32<0x140>(v);
  if constexpr (kLanes >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (kLanes >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// v^-1/2 for normal v: the hardware's (one ulp off) and one Newton step, which
// leaves little more than the last rounding.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = __builtin_amdgcn_rsqf(v);
  const float s = __builtin_fmaf(0.5f * r, __builtin_fmaf(-v * r, r, 1.0f), r);
  return v > 0x1.fffffep127f ? 0.0f : s;   // infinity
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = lanes_max_u32<16>(v);
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(r[0], r[1]);
  const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(s[0], s[1]);
}

// Raises *amax (a non-negative float) to the block's largest `top` >= 0; all
// threads of the block (whole waves) call it, once.  The maximum does not
// depend on the order of the atomics; a stale value read only costs one more.
//
// Atomics on one address go one after the other, 5 to 10 ns each, and the
// blocks of a call end together: with one from every wave, each having read
// the 0 that a new maximum starts with, 8192 waves took 90 us in a kernel of
// 4.6.  So a block joins its waves first, and where there are many blocks
// every 61st goes ahead (61: not in step with the rows, whose columns differ);
// the others wait 1.5 us and look again: about as many as the first are still
// higher.  Same call 9.0 us; gated activation 8192 x 11008 from E4M3 73.9 ->
// 53.0 us (50.4 without a maximum), 1024 x 11008 65 -> 12.4 (8.2), norm
// 2048 x 2048 50.6 -> 8.1 (4.4).  A wait of 1 us is 0.3 us better at few hundred
// blocks and 1 worse at the large sizes, 2 us the other way round.  Up to 128
// blocks take no wait.
__device__ __forceinline__ void raise_amax(float* amax, float top) {
  uint32_t bits = wave_max_u32(__float_as_uint(top));
  if (blockDim.x > 64) {
    __shared__ uint32_t best[16];
    if ((threadIdx.x & 63) == 0) best[threadIdx.x >> 6] = bits;
    __syncthreads();
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) bits = max(bits, best[w]);
  }
  if (threadIdx.x != 0) return;
  uint32_t* a = reinterpret_cast<uint32_t*>(amax);
  auto higher = [&] { return bits > __hip_atomic_load(a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  if (!higher()) return;
  if (gridDim.x > 128 && blockIdx.x % 61 != 0) {
    __builtin_amdgcn_s_sleep(48);   // of 64 cycles
    if (!higher()) return;
  }
  atomicMax(a, bits);
}

// Column sums of `parts` rows of partial sums (row stride `cols`), written or
// added to dst0 (columns below `split`) and dst1 (the others).  Enqueued by
// the backward passes behind the kernel that writes the partial sums.
__attribute__((visibility("hidden"))) hipError_t launch_sum_partials(const float* partials, int parts, int64_t cols,
                                                                     float* dst0, int64_t split, float* dst1,
                                                                     bool accumulate, hipStream_t stream);

}  // namespace coat

#endif  // COAT_ELEM_H
