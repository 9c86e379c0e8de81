// coat_qk.hip -- gfx950 kernels and C ABI of the RMS norm of query and key
// heads with the position rotation in the same pass and an E4M3 checkpoint
// of the heads, and of its backward pass.
//
// Sources (see include/coat_fp8.h for the full citations):
//   [P1] COAT paper review (xllm-io.github.io), section 三: the inputs of
//        non-linear layers are kept in E4M3 per 1xG group (混合粒度激活量化).

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "coat_elem.h"

using namespace coat;

namespace {

// A head of D values lies on kLanes lanes of a wave, eight values a lane
// (kLanes the power of two >= D/8, at least 8; lanes past D/8 idle), so a
// wave works on a set of 64 / kLanes neighbouring heads at once.  A wave takes
// one token and kH sets of its query heads or of its key heads (a slab): it
// loads them all before it works on the first, and the token's cosines and
// sines and the weight once.
//
// Rotation.  Pair j of a head, (a, b), becomes (a cos_j - b sin_j,
// b cos_j + a sin_j).  Interleaved: (a, b) = values (2j, 2j + 1), inside a
// lane.  Otherwise values (j, j + rot/2): rot is a multiple of 16, so a whole
// chunk's partner is the chunk rot/16 lanes away, which sends its BF16 words
// over (ds_bpermute).  The forward pass multiplies the weights into the
// token's cosines and sines once, so a value costs x A + partner B and rstd:
// 31 -> 17 vector instructions a value with that and the cheaper checkpoint
// arithmetic, which had bound the kernel.
// A token whose position is outside the table is padding: everything written
// for it is zero.
//
// 8192 tokens, 64 heads of 128 values, with checkpoint: 59.9 us, 5.71 TB/s, at
// 69% vector issue (67 us before the weights were folded in).

struct QkParams {
  const uint16_t* q;        // forward: heads; backward: their output gradients
  const uint16_t* k;
  int64_t q_stride, k_stride;   // values between tokens
  uint16_t* q_out;
  uint16_t* k_out;
  int64_t q_out_stride, k_out_stride;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  const float* cos;
  const float* sin;
  const int64_t* positions;
  uint8_t* codes;
  float* scales;
  float* rstd;
  float* partials;          // backward: gridDim.x rows of 2 D, or NULL
  int64_t table_rows;
  int32_t units;            // (token, slab) pairs, < 2^31
  int32_t slabs, q_slabs;   // slabs of heads of a token, and those of queries
  int32_t q_heads, k_heads;
  int32_t dim, rot;
  int32_t interleaved;
  int32_t group_shift;
  float eps, inv_dim;
};

// Index of the wave in the launch, the same for all its lanes (so what
// follows from it is scalar work).
__device__ __forceinline__ uint32_t wave_index(uint32_t block) {
  return block * kWavesPerBlock + (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

// What a lane keeps of a token: the rotation of its chunk.  `sin` is signed
// for what the partner's value is multiplied with.
struct Turn {
  float cos[8], sin[8];
  bool live;
};

__device__ __forceinline__ void load4(const float* p, float* f) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}

// dir = 1 forward, -1 for the transposed rotation of the backward pass.
__device__ __forceinline__ Turn load_turn(const QkParams& p, int64_t pos, int chunk, float dir) {
  Turn r;
  r.live = pos >= 0 && pos < p.table_rows;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    r.cos[e] = 1.0f;
    r.sin[e] = 0.0f;
  }
  if (r.live && 8 * chunk < p.rot) {
    const int64_t row = pos * (p.rot / 2);
    if (p.interleaved) {
      float c[4], s[4];
      load4(p.cos + row + 4 * chunk, c);
      load4(p.sin + row + 4 * chunk, s);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r.cos[2 * j] = r.cos[2 * j + 1] = c[j];
        r.sin[2 * j] = -dir * s[j];
        r.sin[2 * j + 1] = dir * s[j];
      }
    } else {
      const int half = p.rot / 16;   // chunks of half the rotated values
      const bool second = chunk >= half;
      const int64_t at = row + 8 * (second ? chunk - half : chunk);
      load4(p.cos + at, r.cos);
      load4(p.cos + at + 4, r.cos + 4);
      load4(p.sin + at, r.sin);
      load4(p.sin + at + 4, r.sin + 4);
      const float sign = second ? dir : -dir;
#pragma unroll
      for (int e = 0; e < 8; ++e) r.sin[e] *= sign;
    }
  }
  return r;
}

// Byte address for ds_bpermute of the lane that holds a chunk's partner.
__device__ __forceinline__ int partner_lane(const QkParams& p, int lane, int chunk) {
  const int half = p.rot / 16;
  if (p.interleaved || chunk >= 2 * half) return 4 * lane;
  return 4 * (chunk < half ? lane + half : lane - half);
}

__device__ __forceinline__ uint4 from_lane(uint4 v, int addr) {
  return make_uint4((uint32_t)__builtin_amdgcn_ds_bpermute(addr, (int)v.x), (uint32_t)__builtin_amdgcn_ds_bpermute(addr, (int)v.y),
                    (uint32_t)__builtin_amdgcn_ds_bpermute(addr, (int)v.z), (uint32_t)__builtin_amdgcn_ds_bpermute(addr, (int)v.w));
}

// The partner of each value of an interleaved chunk.
__device__ __forceinline__ void swap_pairs(const float (&f)[8], float (&g)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) g[e] = f[e ^ 1];
}

// What a wave works on: a token and heads first .. first + count - 1 (this
// lane's head `sub` of a set further on) of its queries or keys.
struct Slab {
  int64_t token;
  bool key;
  int heads, first;      // of the queries or keys
  int64_t row;           // index of the token's head 0 in the checkpoint
  const uint16_t* in;    // the token's heads
  uint16_t* out;
  const uint16_t* weight;
};

template <int kSet, int kH>
__device__ __forceinline__ Slab slab_of(const QkParams& p, uint32_t unit) {
  Slab s;
  const uint32_t token = unit / (uint32_t)p.slabs;
  int slab = (int)(unit - token * (uint32_t)p.slabs);
  s.token = token;
  s.key = slab >= p.q_slabs;
  if (s.key) slab -= p.q_slabs;
  s.heads = s.key ? p.k_heads : p.q_heads;
  s.first = slab * (kSet * kH);
  s.row = s.token * (p.q_heads + p.k_heads) + (s.key ? p.q_heads : 0);
  s.in = s.key ? p.k + s.token * p.k_stride : p.q + s.token * p.q_stride;
  s.out = s.key ? p.k_out + s.token * p.k_out_stride : p.q_out + s.token * p.q_out_stride;
  s.weight = s.key ? p.k_weight : p.q_weight;
  return s;
}

// Element `i` past a uniform address: a scalar base and a 32-bit offset.
template <class V>
__device__ __forceinline__ V* at(V* base, int i) {
  return reinterpret_cast<V*>(reinterpret_cast<uintptr_t>(base) + (uint32_t)i * (uint32_t)sizeof(V));
}

template <int kLanes, int kH>
__global__ __launch_bounds__(kBlockThreads) void qk_norm_rope_kernel(const QkParams p) {
  constexpr int kSet = 64 / kLanes;   // heads a wave works on at once
  const int lane = threadIdx.x & 63, chunk = lane & (kLanes - 1), sub = lane / kLanes;
  const bool on = 8 * chunk < p.dim;
  const uint32_t unit = wave_index(blockIdx.x);
  if (unit >= (uint32_t)p.units) return;
  const Slab s = slab_of<kSet, kH>(p, unit);
  uint4 raw[kH];
#pragma unroll
  for (int i = 0; i < kH; ++i) {
    const int head = s.first + kSet * i + sub;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (on && head < s.heads) raw[i] = load_stream16(at(s.in, head * p.dim + 8 * chunk));
  }
  const Turn turn = load_turn(p, p.positions[s.token], chunk, 1.0f);
  const int addr = partner_lane(p, lane, chunk), lanes = 1 << (p.group_shift - 3);
  float own[8], other[8];   // what a value and its partner are multiplied with, but for rstd
  {
    uint4 w = on ? *reinterpret_cast<const uint4*>(at(s.weight, 8 * chunk)) : make_uint4(0, 0, 0, 0);
    if (!turn.live) w = make_uint4(0, 0, 0, 0);   // padding stays zero whatever the weight holds
    float f[8], g[8];
    unpack8(w, f);
    if (p.interleaved)
      swap_pairs(f, g);
    else
      unpack8(from_lane(w, addr), g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      own[e] = f[e] * turn.cos[e];
      other[e] = g[e] * turn.sin[e];
    }
  }
#pragma unroll
  for (int i = 0; i < kH; ++i) {
    const int head = s.first + kSet * i + sub;
    const bool ok = on && head < s.heads;
    if (!turn.live) raw[i] = make_uint4(0, 0, 0, 0);
    float x[8], far[8];
    unpack8(raw[i], x);
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(x[e], x[e], ss);
    float rstd = inv_sqrt(__builtin_fmaf(lanes_sum<kLanes>(ss), p.inv_dim, p.eps));
    if (!turn.live) rstd = 0.0f;
    if (p.codes) {
      float scale;
      const uint2 c = checkpoint8(raw[i], lanes, scale);
      if (ok) {
        const int from = head * p.dim + 8 * chunk;
        store_stream8(at(p.codes + s.row * p.dim, from), c);
        if ((chunk & (lanes - 1)) == 0)
          *at(p.scales + ((s.row * p.dim) >> p.group_shift), from >> p.group_shift) = scale;
      }
    }
    if (p.rstd && ok && chunk == 0) *at(p.rstd + s.row, head) = rstd;
    if (p.interleaved)
      swap_pairs(x, far);
    else
      unpack8(from_lane(raw[i], addr), far);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = rstd * __builtin_fmaf(far[e], other[e], x[e] * own[e]);
    if (ok) store_stream16(at(s.out, head * p.dim + 8 * chunk), pack8(x));
  }
}

// Backward.  dy is the output gradient turned back by the same angle; then
// the norm's gradient with n = code scale rstd:
//   dn = dy w,  dx = rstd (dn - n mean(dn n)),  dw = sum over tokens and heads of dy n
// Waves walk (token, slab) units with a stride and keep dy n of their chunk
// in FP32 registers, queries and keys apart; a block joins its lanes' sums in
// the LDS in a fixed order and writes one row of partial sums.  64 heads of 128
// values over 8192 tokens: 64.7 us, 5.3 TB/s, 4 of them the second launch.
template <int kLanes, int kH>
__global__ __launch_bounds__(kBlockThreads) void qk_norm_rope_bwd_kernel(const QkParams p) {
  constexpr int kSet = 64 / kLanes;
  const int lane = threadIdx.x & 63, chunk = lane & (kLanes - 1), sub = lane / kLanes;
  const bool on = 8 * chunk < p.dim;
  const int addr = partner_lane(p, lane, chunk);
  float dwq[8], dwk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.0f;
  const uint32_t step = gridDim.x * kWavesPerBlock;
  // The next unit's heads and position are loaded before the current one's
  // are worked on.
  uint4 raw_n[kH];
  uint2 code_n[kH];
  float scale_n[kH], rs_n[kH];
  int64_t pos_n = 0;
  auto load = [&](uint32_t unit) __attribute__((always_inline)) {
    const Slab s = slab_of<kSet, kH>(p, unit);
    pos_n = p.positions[s.token];
#pragma unroll
    for (int i = 0; i < kH; ++i) {
      const int head = s.first + kSet * i + sub;
      raw_n[i] = make_uint4(0, 0, 0, 0);
      code_n[i] = make_uint2(0, 0);
      scale_n[i] = rs_n[i] = 0.0f;
      if (on && head < s.heads) {
        const int from = head * p.dim + 8 * chunk;
        raw_n[i] = load_stream16(at(s.in, from));
        code_n[i] = load_stream8(at(p.codes + s.row * p.dim, from));
        scale_n[i] = *at(p.scales + ((s.row * p.dim) >> p.group_shift), from >> p.group_shift);
        rs_n[i] = *at(p.rstd + s.row, head);
      }
    }
  };
  uint32_t unit = wave_index(blockIdx.x);
  if (unit < (uint32_t)p.units) load(unit);
  for (; unit < (uint32_t)p.units; unit += step) {
    const Slab s = slab_of<kSet, kH>(p, unit);
    const Turn turn = load_turn(p, pos_n, chunk, -1.0f);
    uint4 raw[kH];
    uint2 code[kH];
    float scale[kH], rs[kH];
#pragma unroll
    for (int i = 0; i < kH; ++i) raw[i] = raw_n[i], code[i] = code_n[i], scale[i] = scale_n[i], rs[i] = rs_n[i];
    if (unit + step < (uint32_t)p.units) load(unit + step);
    float w[8], g[8];
    uint4 rw = on ? *reinterpret_cast<const uint4*>(at(s.weight, 8 * chunk)) : make_uint4(0, 0, 0, 0);
    if (!turn.live) rw = make_uint4(0, 0, 0, 0);
    unpack8(rw, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < kH; ++i) {
      const int head = s.first + kSet * i + sub;
      float d[8], far[8], n[8];
      if (!turn.live) {   // padding: nothing of it counts, whatever its buffers and the weight hold
        raw[i] = make_uint4(0, 0, 0, 0);
        code[i] = make_uint2(0, 0);
        scale[i] = rs[i] = 0.0f;
      }
      unpack8(raw[i], d);
      if (p.interleaved)
        swap_pairs(d, far);
      else
        unpack8(from_lane(raw[i], addr), far);
      e4m3_values8(code[i], n);
      const float sr = scale[i] * rs[i];
      float dot = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] = __builtin_fmaf(far[e], turn.sin[e], d[e] * turn.cos[e]);
        n[e] *= sr;
        g[e] = __builtin_fmaf(d[e], n[e], g[e]);
        d[e] *= w[e];
        dot = __builtin_fmaf(d[e], n[e], dot);
      }
      const float mean = lanes_sum<kLanes>(dot) * p.inv_dim;
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = rs[i] * __builtin_fmaf(-n[e], mean, d[e]);
      if (on && head < s.heads) store_stream16(at(s.out, head * p.dim + 8 * chunk), pack8(d));
    }
    if (s.key) {
#pragma unroll
      for (int e = 0; e < 8; ++e) dwk[e] += g[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) dwq[e] += g[e];
    }
  }
  if (p.partials) {
    // [wave and set of heads][2 D]: the block's rows, added column by column
    constexpr int kRows = kWavesPerBlock * kSet;
    __shared__ float sums[kRows][2 * 8 * kLanes + 4];
    const int r = (threadIdx.x >> 6) * kSet + sub;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sums[r][8 * chunk + e] = dwq[e];
      sums[r][8 * kLanes + 8 * chunk + e] = dwk[e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.dim; c += kBlockThreads) {
      const int from = c < p.dim ? c : 8 * kLanes + c - p.dim;
      float v = sums[0][from];
#pragma unroll
      for (int i = 1; i < kRows; ++i) v += sums[i][from];
      p.partials[(int64_t)blockIdx.x * 2 * p.dim + c] = v;
    }
  }
}

constexpr int64_t kMaxHeads = 1 << 16;
constexpr int64_t kMaxDim = 256;

// Most rows of partial sums of the backward pass, and blocks: what the
// registers hold at one or two sets a slab; three quarters of it at more (a
// second round of few blocks otherwise: 64 heads of 128 values over 8192
// tokens take 75.8 us with 1024 blocks, 64.7 with 768).  Constants for the
// reasons of the norm's.
constexpr int64_t kQkParts = 1024;

int lanes_for(int64_t dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

// Sets of heads a wave takes (a slab): up to 4, the number that leaves the
// fewest sets over; 1 where that would give fewer waves than the chip holds at
// four per SIMD.
struct QkSplit {
  int sets;
  int32_t slabs, q_slabs;
  int64_t units;   // at most kMaxUnits
};

constexpr int64_t kMaxUnits = 0x7FFFFFFF - kWavesPerBlock * 65536;   // unit + step stays below 2^32

QkSplit split_heads(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim, int most = 4) {
  const int64_t set = 64 / lanes_for(dim);
  auto slabs = [&](int64_t heads, int64_t h) { return (heads + set * h - 1) / (set * h); };
  // a slab costs about one set more than its own (tables and weight); counted as
  // half a set, 24 and 8 heads of 64 values took 17.7 us and not 14.9
  int best = 1;
  int64_t cost = INT64_MAX;
  for (int h = most; h >= 1; --h) {
    const int64_t c = (slabs(q_heads, h) + slabs(k_heads, h)) * (h + 1);
    if (c < cost) cost = c, best = h;
  }
  if (tokens * (slabs(q_heads, best) + slabs(k_heads, best)) < 4096) best = 1;
  const int64_t q = slabs(q_heads, best), all = q + slabs(k_heads, best);
  return {best, (int32_t)all, (int32_t)q, tokens * all};
}

bool units_ok(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim) {
  return tokens <= kMaxUnits && split_heads(tokens, q_heads, k_heads, dim, 1).units <= kMaxUnits;
}

int64_t qk_parts(int64_t units, int sets) {
  const int64_t blocks = (units + kWavesPerBlock - 1) / kWavesPerBlock, most = sets > 2 ? kQkParts * 3 / 4 : kQkParts;
  return blocks < most ? blocks : most;
}

const void* qk_kernel_for(int lanes, int sets, bool backward) {
#define COAT_QK(L, H)                                                                 \
  if (lanes == L && sets == H)                                                        \
    return backward ? reinterpret_cast<const void*>(&qk_norm_rope_bwd_kernel<L, H>)   \
                    : reinterpret_cast<const void*>(&qk_norm_rope_kernel<L, H>);
  COAT_QK(8, 1)
  COAT_QK(8, 2)
  COAT_QK(8, 3)
  COAT_QK(8, 4)
  COAT_QK(16, 1)
  COAT_QK(16, 2)
  COAT_QK(16, 3)
  COAT_QK(16, 4)
  COAT_QK(32, 1)
  COAT_QK(32, 2)
  COAT_QK(32, 3)
  COAT_QK(32, 4)
#undef COAT_QK
  return nullptr;
}

bool bad_stride(int64_t stride, int64_t heads, int64_t dim, int64_t tokens) {
  return stride % 8 != 0 || (tokens > 1 && stride < heads * dim) || stride > (INT64_MAX / 4) / (tokens > 0 ? tokens : 1);
}

coat_status_t check_qk(const coat_qk_shape_t& s) {
  if (s.tokens < 0 || s.q_heads < 0 || s.k_heads < 0 || s.q_heads > kMaxHeads || s.k_heads > kMaxHeads ||
      s.table_rows < 0)
    return COAT_ERR_INVALID_VALUE;
  if (!valid_group_size(s.group_size)) return COAT_ERR_GROUP_SIZE;
  if (s.head_dim < 16 || s.head_dim > kMaxDim || s.head_dim % 16 != 0 || s.head_dim % s.group_size != 0)
    return COAT_ERR_INVALID_VALUE;
  if (s.rot_dim < 16 || s.rot_dim > s.head_dim || s.rot_dim % 16 != 0) return COAT_ERR_INVALID_VALUE;
  if (s.table_rows > INT64_MAX / 4 / s.head_dim) return COAT_ERR_INVALID_VALUE;
  if (!units_ok(s.tokens, s.q_heads, s.k_heads, s.head_dim)) return COAT_ERR_INVALID_VALUE;
  return COAT_OK;
}

void fill(QkParams& p, const coat_qk_shape_t& s, const QkSplit& split) {
  memset(&p, 0, sizeof(p));
  p.table_rows = s.table_rows;
  p.units = (int32_t)split.units;
  p.slabs = split.slabs;
  p.q_slabs = split.q_slabs;
  p.q_heads = s.q_heads;
  p.k_heads = s.k_heads;
  p.dim = s.head_dim;
  p.rot = s.rot_dim;
  p.interleaved = s.interleaved != 0;
  p.group_shift = __builtin_ctz((unsigned)s.group_size);
  p.inv_dim = (float)(1.0 / (double)s.head_dim);
}

}  // namespace

extern "C" {

coat_status_t coat_fp8_qk_norm_rope(const coat_qk_norm_rope_args_t* a, hipStream_t stream) {
  if (!a) return COAT_ERR_NULL_POINTER;
  const coat_qk_shape_t& s = a->shape;
  const coat_status_t st = check_qk(s);
  if (st != COAT_OK) return st;
  if (!isfinite(a->eps) || a->eps < 0x1p-126f) return COAT_ERR_INVALID_VALUE;
  if (bad_stride(a->q_stride, s.q_heads, s.head_dim, s.tokens) ||
      bad_stride(a->k_stride, s.k_heads, s.head_dim, s.tokens) ||
      bad_stride(a->q_out_stride, s.q_heads, s.head_dim, s.tokens) ||
      bad_stride(a->k_out_stride, s.k_heads, s.head_dim, s.tokens))
    return COAT_ERR_INVALID_VALUE;
  if (s.tokens == 0 || s.q_heads + s.k_heads == 0) return COAT_OK;
  if ((s.q_heads && (!a->q || !a->q_out)) || (s.k_heads && (!a->k || !a->k_out)) || !a->q_weight || !a->k_weight ||
      !a->positions || (s.table_rows && (!a->cos || !a->sin)) || !a->codes != !a->scales)
    return COAT_ERR_NULL_POINTER;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->q_out, 16) || !aligned(a->k_out, 16) ||
      !aligned(a->q_weight, 16) || !aligned(a->k_weight, 16) || !aligned(a->cos, 16) || !aligned(a->sin, 16) ||
      !aligned(a->positions, 8) || !aligned(a->codes, 16) || !aligned(a->scales, 4) || !aligned(a->rstd, 4))
    return COAT_ERR_MISALIGNED;
  const QkSplit split = split_heads(s.tokens, s.q_heads, s.k_heads, s.head_dim);
  const int64_t blocks = (split.units + kWavesPerBlock - 1) / kWavesPerBlock;
  QkParams p;
  fill(p, s, split);
  p.q = a->q;
  p.k = a->k;
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.q_out = a->q_out;
  p.k_out = a->k_out;
  p.q_out_stride = a->q_out_stride;
  p.k_out_stride = a->k_out_stride;
  p.q_weight = a->q_weight;
  p.k_weight = a->k_weight;
  p.cos = a->cos;
  p.sin = a->sin;
  p.positions = a->positions;
  p.codes = a->codes;
  p.scales = a->scales;
  p.rstd = a->rstd;
  p.eps = a->eps;
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(qk_kernel_for(lanes_for(s.head_dim), split.sets, false), dim3((unsigned)blocks),
                                       dim3(kBlockThreads), args, 0, stream);
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

int64_t coat_fp8_qk_norm_rope_bwd_workspace(int64_t tokens, int64_t heads, int64_t head_dim) {
  if (tokens < 0 || heads < 0 || heads > 2 * kMaxHeads || head_dim < 16 || head_dim > kMaxDim || head_dim % 16 != 0 ||
      tokens > kMaxUnits)
    return -1;
  if (tokens == 0 || heads == 0) return 0;
  // the fewest and the most units that a division of the heads into queries and keys gives
  const int64_t set = 64 / lanes_for(head_dim), least = tokens * ((heads + set - 1) / set), units = least + tokens;
  if (least > kMaxUnits) return -1;
  return qk_parts(units, 1) * 2 * head_dim * (int64_t)sizeof(float);
}

coat_status_t coat_fp8_qk_norm_rope_bwd(const coat_qk_norm_rope_bwd_args_t* a, hipStream_t stream) {
  if (!a) return COAT_ERR_NULL_POINTER;
  const coat_qk_shape_t& s = a->shape;
  const coat_status_t st = check_qk(s);
  if (st != COAT_OK) return st;
  if (bad_stride(a->dq_out_stride, s.q_heads, s.head_dim, s.tokens) ||
      bad_stride(a->dk_out_stride, s.k_heads, s.head_dim, s.tokens) ||
      bad_stride(a->dq_stride, s.q_heads, s.head_dim, s.tokens) ||
      bad_stride(a->dk_stride, s.k_heads, s.head_dim, s.tokens))
    return COAT_ERR_INVALID_VALUE;
  if (!a->dq_weight != !a->dk_weight) return COAT_ERR_NULL_POINTER;
  const bool dw = a->dq_weight != nullptr, work = s.tokens > 0 && s.q_heads + s.k_heads > 0;
  if (!work && (!dw || a->accumulate)) return COAT_OK;
  if (work && ((s.q_heads && (!a->dq_out || !a->dq)) || (s.k_heads && (!a->dk_out || !a->dk)) || !a->codes ||
               !a->scales || !a->rstd || !a->q_weight || !a->k_weight || !a->positions ||
               (s.table_rows && (!a->cos || !a->sin)) || (dw && !a->workspace)))
    return COAT_ERR_NULL_POINTER;
  if (!aligned(a->dq_out, 16) || !aligned(a->dk_out, 16) || !aligned(a->codes, 16) || !aligned(a->scales, 4) ||
      !aligned(a->rstd, 4) || !aligned(a->q_weight, 16) || !aligned(a->k_weight, 16) || !aligned(a->cos, 16) ||
      !aligned(a->sin, 16) || !aligned(a->positions, 8) || !aligned(a->dq, 16) || !aligned(a->dk, 16) ||
      !aligned(a->dq_weight, 4) || !aligned(a->dk_weight, 4) || !aligned(a->workspace, 16))
    return COAT_ERR_MISALIGNED;
  if (work && dw &&
      a->workspace_bytes < coat_fp8_qk_norm_rope_bwd_workspace(s.tokens, s.q_heads + s.k_heads, s.head_dim))
    return COAT_ERR_INVALID_VALUE;
  const QkSplit split = split_heads(s.tokens, s.q_heads, s.k_heads, s.head_dim);
  const int64_t blocks = work ? qk_parts(split.units, split.sets) : 0;
  hipError_t e = hipSuccess;
  if (work) {
    QkParams p;
    fill(p, s, split);
    p.q = a->dq_out;
    p.k = a->dk_out;
    p.q_stride = a->dq_out_stride;
    p.k_stride = a->dk_out_stride;
    p.q_out = a->dq;
    p.k_out = a->dk;
    p.q_out_stride = a->dq_stride;
    p.k_out_stride = a->dk_stride;
    p.q_weight = a->q_weight;
    p.k_weight = a->k_weight;
    p.cos = a->cos;
    p.sin = a->sin;
    p.positions = a->positions;
    p.codes = const_cast<uint8_t*>(a->codes);
    p.scales = const_cast<float*>(a->scales);
    p.rstd = const_cast<float*>(a->rstd);
    p.partials = dw ? (float*)a->workspace : nullptr;
    void* args[] = {&p};
    e = hipLaunchKernel(qk_kernel_for(lanes_for(s.head_dim), split.sets, true), dim3((unsigned)blocks),
                        dim3(kBlockThreads), args, 0, stream);
  }
  if (e == hipSuccess && dw)
    e = launch_sum_partials((const float*)a->workspace, (int)blocks, 2 * s.head_dim, a->dq_weight, s.head_dim,
                            a->dk_weight, a->accumulate != 0, stream);
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

}  // extern "C"
