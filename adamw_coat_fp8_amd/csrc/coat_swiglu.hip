// coat_swiglu.hip -- gfx950 kernels and C ABI of the gated activation
// silu(gate) * up from E4M3 or BF16, and of its backward pass from the E4M3
// checkpoint.
//
// Sources (see include/coat_fp8.h for the full citations):
//   [P1] COAT paper review (xllm-io.github.io), section 三: the activation of
//        the FFN (MLPResidual) reads and keeps its input in E4M3 per 1xG
//        group; the linear layer behind it takes one scale per tensor.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "coat_elem.h"

using namespace coat;

namespace {

// Rows of 2 `cols` values, the gates first.  Element-wise but for the scales:
// a thread takes kE neighbouring columns of the gates and the same of the
// ups; units (row, kE columns) are numbered through the matrix, a block takes
// 256 in a row at a time.  kE is 16 where input and output are both E4M3
// (16-byte accesses), else 8 (16 bytes of BF16).
//
// Bound by HBM (8192 x 11008, G = 128): E4M3 to E4M3 49.4 us, 5.6 TB/s, with
// vector instructions in 85% of the cycles, 52.7 us where it raises a maximum
// from zero; E4M3 to BF16 61.9 us, 5.92; BF16 to E4M3 with checkpoint 113 us,
// 5.65, with a maximum 117; backward 123 us, 5.93 TB/s.

struct ActParams {
  const uint16_t* gate_up;
  uint8_t* codes;   // read without gate_up, else written if not NULL
  float* scales;
  uint16_t* h;
  uint8_t* h_codes;
  float* h_amax;
  const uint16_t* dh;
  uint16_t* d_gate_up;
  uint32_t units;          // of this launch, < 2^31
  uint32_t units_per_row;
  uint32_t magic;          // unit / units_per_row = umulhi(unit, magic) >> shift (units_per_row > 1)
  int32_t shift;
  int32_t cols;
  int32_t group_shift;
  float inv_h_scale;
};

// Row of a unit: with d = units_per_row >= 2, s = ceil(log2 d) and
// magic = floor(2^(31+s) / d) + 1, the product overshoots unit / d by at most
// unit / 2^(31+s) < 1 / 2^s <= 1 / d, so its floor is exact below 2^31.
__device__ __forceinline__ uint32_t unit_row(const ActParams& p, uint32_t u) {
  return p.units_per_row == 1 ? u : __umulhi(u, p.magic) >> p.shift;
}

// s = sigmoid(g) and 1 - s from z = exp(-|g|) <= 1: nothing overflows, and
// neither value cancels.  The reciprocal is the hardware's (one ulp); z's
// relative error grows to 5e-6 at |g| = 80, where it no longer counts, and
// below 2^-126 (|g| > 87.33) z is 0.
__device__ __forceinline__ void sigmoid(float g, float& s, float& rest) {
  const float z = __expf(-fabsf(g)), r = __builtin_amdgcn_rcpf(1.0f + z), zr = z * r;
  s = g >= 0.0f ? r : zr;
  rest = g >= 0.0f ? zr : r;
}

template <bool kBF16In, bool kFP8Out>
__global__ __launch_bounds__(kBlockThreads) void swiglu_kernel(const ActParams p) {
  constexpr int kE = !kBF16In && kFP8Out ? 16 : 8;
  float top = 0.0f;
  for (uint32_t base = blockIdx.x * kBlockThreads; base < p.units; base += gridDim.x * kBlockThreads) {
    const uint32_t u = base + threadIdx.x;
    const bool ok = u < p.units;   // whole groups: units_per_row is a multiple of a group's lanes
    const uint32_t row = unit_row(p, ok ? u : 0);
    const int col = kE * (int)((ok ? u : 0) - row * p.units_per_row);
    const int64_t gate_at = (int64_t)row * 2 * p.cols + col, up_at = gate_at + p.cols;
    float g[kE], v[kE];
    if constexpr (kBF16In) {
      uint4 rg = make_uint4(0, 0, 0, 0), ru = rg;
      if (ok) {
        rg = load_stream16(p.gate_up + gate_at);
        ru = load_stream16(p.gate_up + up_at);
      }
      if (p.codes) {   // all lanes: groups exchange their maxima
        const int lanes = 1 << (p.group_shift - 3);
        float sg, su;
        const uint2 cg = checkpoint8(rg, lanes, sg), cu = checkpoint8(ru, lanes, su);
        if (ok) {
          store_stream8(p.codes + gate_at, cg);
          store_stream8(p.codes + up_at, cu);
          if ((threadIdx.x & (lanes - 1)) == 0) {
            p.scales[gate_at >> p.group_shift] = sg;
            p.scales[up_at >> p.group_shift] = su;
          }
        }
      }
      unpack8(rg, g);
      unpack8(ru, v);
    } else if (ok) {
      const float sg = p.scales[gate_at >> p.group_shift], su = p.scales[up_at >> p.group_shift];
      if constexpr (kE == 16) {
        const uint4 cg = load_stream16(p.codes + gate_at), cu = load_stream16(p.codes + up_at);
        e4m3_values4(cg.x, g), e4m3_values4(cg.y, g + 4), e4m3_values4(cg.z, g + 8), e4m3_values4(cg.w, g + 12);
        e4m3_values4(cu.x, v), e4m3_values4(cu.y, v + 4), e4m3_values4(cu.z, v + 8), e4m3_values4(cu.w, v + 12);
      } else {
        const uint2 cg = load_stream8(p.codes + gate_at), cu = load_stream8(p.codes + up_at);
        e4m3_values4(cg.x, g), e4m3_values4(cg.y, g + 4);
        e4m3_values4(cu.x, v), e4m3_values4(cu.y, v + 4);
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        g[e] *= sg;
        v[e] *= su;
      }
    }
    if (!ok) continue;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      float s, rest;
      sigmoid(g[e], s, rest);
      v[e] *= g[e] * s;
    }
    const int64_t at = (int64_t)row * p.cols + col;
    if constexpr (kFP8Out) {
      const float m = max_mag(v);
      top = fmaxf(top, m);
      uint32_t w[kE / 4];
#pragma unroll
      for (int e = 0; e < kE; ++e) v[e] *= p.inv_h_scale;
      e4m3_pack(v, m * p.inv_h_scale, w);
      if constexpr (kE == 16)
        store_stream16(p.h_codes + at, make_uint4(w[0], w[1], w[2], w[3]));
      else
        store_stream8(p.h_codes + at, make_uint2(w[0], w[1]));
    } else {
      store_stream16(p.h + at, pack8(v));
    }
  }
  if (kFP8Out && p.h_amax) raise_amax(p.h_amax, top);
}

// With s = sigmoid(gate):  d_up = dh gate s,  d_gate = dh up s (1 + gate (1 - s)).
__global__ __launch_bounds__(kBlockThreads) void swiglu_bwd_kernel(const ActParams p) {
  for (uint32_t base = blockIdx.x * kBlockThreads; base < p.units; base += gridDim.x * kBlockThreads) {
    const uint32_t u = base + threadIdx.x;
    if (u >= p.units) continue;
    const uint32_t row = unit_row(p, u);
    const int col = 8 * (int)(u - row * p.units_per_row);
    const int64_t gate_at = (int64_t)row * 2 * p.cols + col, up_at = gate_at + p.cols;
    const uint4 rd = load_stream16(p.dh + (int64_t)row * p.cols + col);
    const uint2 cg = load_stream8(p.codes + gate_at), cu = load_stream8(p.codes + up_at);
    const float sg = p.scales[gate_at >> p.group_shift], su = p.scales[up_at >> p.group_shift];
    float g[8], v[8], d[8];
    unpack8(rd, d);
    e4m3_values8(cg, g);
    e4m3_values8(cu, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float gate = g[e] * sg, up = v[e] * su;
      float s, rest;
      sigmoid(gate, s, rest);
      const float ds = d[e] * s;
      g[e] = ds * up * __builtin_fmaf(gate, rest, 1.0f);
      v[e] = ds * gate;
    }
    store_stream16(p.d_gate_up + gate_at, pack8(g));
    store_stream16(p.d_gate_up + up_at, pack8(v));
  }
}

coat_status_t check_act_shape(int64_t rows, int64_t cols, int32_t group_size) {
  if (rows < 0 || cols < 0) return COAT_ERR_INVALID_VALUE;
  if (!valid_group_size(group_size)) return COAT_ERR_GROUP_SIZE;
  if (cols % group_size != 0 || cols > (1 << 30)) return COAT_ERR_INVALID_VALUE;
  if (cols > 0 && rows > INT64_MAX / 16 / cols) return COAT_ERR_INVALID_VALUE;
  return COAT_OK;
}

// Launches fn over all rows, in slabs of fewer than 2^31 units (one slab for
// any matrix below 2^34 values).
hipError_t launch_act(const void* fn, ActParams p, int64_t rows, int elems, hipStream_t stream) {
  int cus = 0;
  hipError_t e = current_cu_count(&cus);
  if (e != hipSuccess) return e;
  p.units_per_row = (uint32_t)(p.cols / elems);
  int s = 0;
  while ((1u << s) < p.units_per_row) ++s;
  p.shift = s - 1;
  p.magic = s == 0 ? 0 : (uint32_t)((1ull << (31 + s)) / p.units_per_row + 1);
  const int64_t most = 0x7FFFFFFF / p.units_per_row;
  while (rows > 0) {
    const int64_t now = rows < most ? rows : most;
    p.units = (uint32_t)(now * p.units_per_row);
    const int64_t blocks = ((int64_t)p.units + kBlockThreads - 1) / kBlockThreads;
    const int64_t fill = (int64_t)cus * 32;
    void* args[] = {&p};
    e = hipLaunchKernel(fn, dim3((unsigned)(blocks < fill ? blocks : fill)), dim3(kBlockThreads), args, 0, stream);
    if (e != hipSuccess) return e;
    rows -= now;
    const int64_t in = 2 * now * p.cols, out = now * p.cols;
    if (p.gate_up) p.gate_up += in;
    if (p.codes) p.codes += in, p.scales += in >> p.group_shift;
    if (p.h) p.h += out;
    if (p.h_codes) p.h_codes += out;
    if (p.dh) p.dh += out;
    if (p.d_gate_up) p.d_gate_up += in;
  }
  return hipSuccess;
}

}  // namespace

extern "C" {

coat_status_t coat_fp8_swiglu(const coat_swiglu_args_t* a, hipStream_t stream) {
  if (!a) return COAT_ERR_NULL_POINTER;
  const coat_status_t st = check_act_shape(a->rows, a->cols, a->group_size);
  if (st != COAT_OK) return st;
  if (a->h && a->h_codes) return COAT_ERR_INVALID_VALUE;
  if (a->h_codes && !(a->h_scale > 0.0f && isfinite(a->h_scale) && isfinite(1.0f / a->h_scale)))
    return COAT_ERR_INVALID_VALUE;
  if (a->h_amax && !a->h_codes) return COAT_ERR_INVALID_VALUE;
  if (a->rows == 0 || a->cols == 0) return COAT_OK;
  if (!a->h && !a->h_codes) return COAT_ERR_NULL_POINTER;
  if (!a->codes != !a->scales || (!a->gate_up && !a->codes)) return COAT_ERR_NULL_POINTER;
  if (!aligned(a->gate_up, 16) || !aligned(a->codes, 16) || !aligned(a->scales, 4) || !aligned(a->h, 16) ||
      !aligned(a->h_codes, 16) || !aligned(a->h_amax, 4))
    return COAT_ERR_MISALIGNED;
  ActParams p;
  memset(&p, 0, sizeof(p));
  p.gate_up = a->gate_up;
  p.codes = a->codes;
  p.scales = a->scales;
  p.h = a->h;
  p.h_codes = a->h_codes;
  p.h_amax = a->h_amax;
  p.cols = (int32_t)a->cols;
  p.group_shift = __builtin_ctz((unsigned)a->group_size);
  p.inv_h_scale = a->h_codes ? 1.0f / a->h_scale : 0.0f;
  const void* fn = a->gate_up ? (a->h ? reinterpret_cast<const void*>(&swiglu_kernel<true, false>)
                                      : reinterpret_cast<const void*>(&swiglu_kernel<true, true>))
                              : (a->h ? reinterpret_cast<const void*>(&swiglu_kernel<false, false>)
                                      : reinterpret_cast<const void*>(&swiglu_kernel<false, true>));
  const hipError_t e = launch_act(fn, p, a->rows, !a->gate_up && a->h_codes ? 16 : 8, stream);
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

coat_status_t coat_fp8_swiglu_bwd(const uint16_t* dh, const uint8_t* codes, const float* scales, int64_t rows,
                                  int64_t cols, int32_t group_size, uint16_t* d_gate_up, hipStream_t stream) {
  const coat_status_t st = check_act_shape(rows, cols, group_size);
  if (st != COAT_OK) return st;
  if (rows == 0 || cols == 0) return COAT_OK;
  if (!dh || !codes || !scales || !d_gate_up) return COAT_ERR_NULL_POINTER;
  if (!aligned(dh, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(d_gate_up, 16))
    return COAT_ERR_MISALIGNED;
  ActParams p;
  memset(&p, 0, sizeof(p));
  p.dh = dh;
  p.codes = const_cast<uint8_t*>(codes);
  p.scales = const_cast<float*>(scales);
  p.d_gate_up = d_gate_up;
  p.cols = (int32_t)cols;
  p.group_shift = __builtin_ctz((unsigned)group_size);
  const hipError_t e = launch_act(reinterpret_cast<const void*>(&swiglu_bwd_kernel), p, rows, 8, stream);
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

}  // extern "C"
