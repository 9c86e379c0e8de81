// coat_embed.hip -- gfx950 embedding lookup and its gradient, and their C ABI.

#include <hip/hip_runtime.h>

#include <float.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "coat_elem.h"

using namespace coat;

namespace {

// ------------------------------------------------------------------ lookup

struct LookupParams {
  const uint8_t* table;     // BF16, or codes
  const int64_t* tokens;
  uint16_t* out;
  int64_t vocab;
  uint32_t chunks, total;   // of 8 values: of a row, of all rows
  float scale;
};

// out[r] = bf16(scale * table[token of r]), zeros for a token outside the
// table.  A thread copies two chunks of eight values.
template <bool kFP8>
__global__ __launch_bounds__(256) void embedding_kernel(const LookupParams p) {
  uint32_t at[2];
  uint4 v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    at[i] = blockIdx.x * 512 + 256 * i + threadIdx.x;
    if (at[i] >= p.total) continue;
    const uint32_t row = at[i] / p.chunks, c = at[i] - row * p.chunks;
    const int64_t token = p.tokens[row];
    float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (token >= 0 && token < p.vocab) {
      const int64_t from = token * p.chunks + c;
      if constexpr (kFP8) e4m3_values8(*reinterpret_cast<const uint2*>(p.table + 8 * from), f);
      else unpack8(*reinterpret_cast<const uint4*>(p.table + 16 * from), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= p.scale;
    }
    v[i] = pack8(f);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (at[i] < p.total) store_stream16(p.out + 8 * (int64_t)at[i], v[i]);
}

// ---------------------------------------------------------------- gradient
//
// dW[v] = scale * sum of dy over the rows whose token is v, in the rows'
// order: the rows are sorted by (token, row), runs of one token are summed in
// FP32 from that order, 32 rows to a part, and runs that span parts are joined
// from partial sums.  No atomics: the result does not depend on timing.

enum Out { kBF16 = 0, kF32 = 1, kF32Add = 2 };

constexpr int kSortRows = 16384;   // rows that one block's keys cover
constexpr int kPart = 32;          // sorted rows of a part

struct SortParams {
  const int64_t* tokens;
  int32_t* key;             // sorted tokens of each run of kSortRows rows
  int32_t* order;           // and their rows
  int32_t* count;           // of each run: rows whose token is in the table
  uint8_t* dw;              // zeroed by the blocks behind the sort's, or NULL
  int64_t rows, vocab, dw_bytes;
  int32_t sort_blocks;
};

// A row's place in its run: how many keys are smaller, or equal and earlier.
// A block of 16 waves places 64 rows, one a lane; each wave counts a
// sixteenth of the keys, which lie in the LDS and are read by all lanes at
// once.
__global__ __launch_bounds__(1024) void sort_kernel(const SortParams p) {
  __shared__ __attribute__((aligned(16))) int32_t keys[kSortRows];
  __shared__ int32_t below[16][64];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  if ((int)blockIdx.x >= p.sort_blocks) {
    const int64_t stride = 16384 * (int64_t)(gridDim.x - p.sort_blocks);
    for (int64_t at = 16384 * (int64_t)(blockIdx.x - p.sort_blocks) + 16 * t; at < p.dw_bytes; at += stride)
      store_stream16(p.dw + at, make_uint4(0, 0, 0, 0));
    return;
  }
  const int64_t row0 = 64 * (int64_t)blockIdx.x, run0 = row0 / kSortRows * kSortRows;
  const int n = (int)(p.rows - run0 < kSortRows ? p.rows - run0 : kSortRows);
  const int padded = (n + 63) / 64 * 64;
  const int32_t none = (int32_t)p.vocab;   // behind every token
  for (int i = t; i < padded; i += 1024) {
    const int64_t token = i < n ? p.tokens[run0 + i] : -1;
    keys[i] = token >= 0 && token < p.vocab ? (int32_t)token : none;
  }
  __syncthreads();
  const int first = (int)(row0 - run0);     // of the block's rows in the run
  const int32_t mine = first + lane < n ? keys[first + lane] : none;
  int32_t less = 0;
  const int groups = padded / 64, g0 = groups * wave / 16, g1 = groups * (wave + 1) / 16;
  for (int g = g0; g < g1; ++g) {
    // keys before the row count if equal too
    const int32_t limit = 64 * g < first ? mine + 1 : mine;
#pragma unroll
    for (int i = 0; i < 64; i += 4) {
      const int4 k = *reinterpret_cast<const int4*>(&keys[64 * g + i]);
      less += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
    }
    if (64 * g == first) {
      for (int i = 0; i < 64; ++i) less += i < lane && keys[first + i] == mine;
    }
  }
  below[wave][lane] = less;
  __syncthreads();
  if (wave == 0) {
    int32_t place = 0;
    for (int w = 0; w < 16; ++w) place += below[w][lane];
    if (mine < none) {
      p.key[run0 + place] = mine;
      p.order[run0 + place] = (int32_t)(row0 + lane);
    }
  }
  // the run's first block counts its rows
  if (first == 0) {
    __syncthreads();
    int32_t live = 0;
    for (int i = t; i < n; i += 1024) live += keys[i] < none;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) live += __shfl_xor(live, s);
    if (lane == 0) below[0][wave] = live;
    __syncthreads();
    if (t == 0) {
      for (int w = 1; w < 16; ++w) live += below[0][w];
      p.count[run0 / kSortRows] = live;
    }
  }
}

struct MergeParams {
  const int32_t *key, *order, *count;   // sorted runs
  int32_t *key_out, *order_out, *total;
  int32_t runs;
};

// Merges the runs: a row's place among all is its place in its run and, for
// every other run, the number of its keys that go before.
__global__ __launch_bounds__(256) void merge_kernel(const MergeParams p) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int run = (int)(at / kSortRows), i = (int)(at % kSortRows);
  if (at == 0) {
    int32_t n = 0;
    for (int r = 0; r < p.runs; ++r) n += p.count[r];
    *p.total = n;
  }
  if (run >= p.runs || i >= p.count[run]) return;
  const int32_t mine = p.key[at];
  int64_t place = i;
  for (int r = 0; r < p.runs; ++r) {
    if (r == run) continue;
    const int32_t* key = p.key + (int64_t)r * kSortRows;
    const int32_t limit = r < run ? mine + 1 : mine;
    int lo = 0, hi = p.count[r];
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (key[mid] < limit) lo = mid + 1;
      else hi = mid;
    }
    place += lo;
  }
  p.key_out[place] = mine;
  p.order_out[place] = p.order[at];
}

struct SumParams {
  const uint16_t* dy;
  const int32_t *key, *order, *total;
  float* partial;           // [part][2][cols]: of the run that a part begins in, of the one it ends in
  void* dw;
  int64_t cols;
  int32_t parts, width;     // width: threads along the columns
  int32_t mode;
  float scale;
};

__device__ __forceinline__ void store_row(const SumParams& p, int64_t v, int64_t col, float (&s)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] *= p.scale;
  if (p.mode == kBF16) {
    store_stream16((uint16_t*)p.dw + v * p.cols + col, pack8(s));
    return;
  }
  float4* dst = reinterpret_cast<float4*>((float*)p.dw + v * p.cols + col);
  if (p.mode == kF32Add) {
    const float4 a = dst[0], b = dst[1];
    s[0] += a.x, s[1] += a.y, s[2] += a.z, s[3] += a.w;
    s[4] += b.x, s[5] += b.y, s[6] += b.z, s[7] += b.w;
  }
  dst[0] = make_float4(s[0], s[1], s[2], s[3]);
  dst[1] = make_float4(s[4], s[5], s[6], s[7]);
}

__device__ __forceinline__ void store_partial(float* to, const float (&s)[8]) {
  reinterpret_cast<float4*>(to)[0] = make_float4(s[0], s[1], s[2], s[3]);
  reinterpret_cast<float4*>(to)[1] = make_float4(s[4], s[5], s[6], s[7]);
}

// One part of the sorted rows, eight columns a thread.
__global__ __launch_bounds__(256) void sum_kernel(const SumParams p) {
  const int per = 256 / p.width, lane = threadIdx.x % p.width;
  const int part = blockIdx.x * per + threadIdx.x / p.width;
  const int64_t col = 8 * ((int64_t)blockIdx.y * p.width + lane);
  const int total = *p.total, first = part * kPart;
  if (part >= p.parts || first >= total || col >= p.cols) return;
  const int last = first + kPart < total ? first + kPart : total;
  const bool from_before = first > 0 && p.key[first - 1] == p.key[first];
  const bool goes_on = last < total && p.key[last] == p.key[last - 1];
  float* partial = p.partial + 2 * (int64_t)part * p.cols + col;
  uint4 raw[kPart];
#pragma unroll
  for (int i = 0; i < kPart; ++i) {
    const int at = first + i < last ? first + i : last - 1;
    raw[i] = load_stream16(p.dy + (int64_t)p.order[at] * p.cols + col);
  }
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  bool head = from_before;   // the run at hand began in an earlier part
#pragma unroll
  for (int i = 0; i < kPart; ++i) {
    if (first + i >= last) break;
    float f[8];
    unpack8(raw[i], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += f[e];
    const bool end = first + i + 1 == last;
    const int32_t key = p.key[first + i];
    if (!end && p.key[first + i + 1] == key) continue;
    if (head) store_partial(partial, s);
    else if (end && goes_on) store_partial(partial + p.cols, s);
    else store_row(p, key, col, s);
    head = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.0f;
  }
}

// Joins the runs that begin in a part and go on behind it.
__global__ __launch_bounds__(256) void join_kernel(const SumParams p) {
  const int per = 256 / p.width, lane = threadIdx.x % p.width;
  const int part = blockIdx.x * per + threadIdx.x / p.width;
  const int64_t col = 8 * ((int64_t)blockIdx.y * p.width + lane);
  const int total = *p.total, first = part * kPart, next = first + kPart;
  if (part >= p.parts || next >= total || col >= p.cols) return;
  const int32_t key = p.key[next - 1];
  if (p.key[next] != key) return;
  if (p.key[first] == key && first > 0 && p.key[first - 1] == key) return;   // it began before
  const float* partial = p.partial + 2 * (int64_t)part * p.cols + col;
  float s[8];
  auto load = [&](const float* from, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4*>(from)[0], b = reinterpret_cast<const float4*>(from)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  };
  load(partial + p.cols, s);
  int q = part + 1;   // parts that the run reaches into
  for (;; ++q) {
    float f[8];
    load(p.partial + 2 * (int64_t)q * p.cols + col, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += f[e];
    const int end = (q + 1) * kPart;
    if (end >= total || p.key[end] != key) break;
  }
  store_row(p, key, col, s);
}

// ------------------------------------------------------------------ host

constexpr int64_t kMaxRows = 1 << 23, kMaxVocab = 1 << 22, kMaxCols = 1 << 16;

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool embed_sizes_ok(int64_t rows, int64_t vocab, int64_t cols) {
  return rows >= 0 && rows <= kMaxRows && vocab >= 0 && vocab <= kMaxVocab && cols >= 0 && cols <= kMaxCols &&
         cols % 16 == 0 && rows * cols <= (int64_t)1 << 33 && vocab * cols <= (int64_t)1 << 34;
}

struct Space {
  int32_t *key, *order, *count, *run_key, *run_order, *total;
  float* partial;
  int64_t bytes;
  int32_t runs, parts;
};

Space space_of(void* base, int64_t rows, int64_t cols) {
  int64_t used = 0;
  auto take = [&](int64_t bytes) {
    void* p = base ? (uint8_t*)base + used : nullptr;
    used += up(bytes, 256) * 256;
    return p;
  };
  Space s;
  memset(&s, 0, sizeof(s));
  s.runs = (int32_t)up(rows, kSortRows);
  s.parts = (int32_t)up(rows, kPart);
  s.key = (int32_t*)take(4 * rows);
  s.order = (int32_t*)take(4 * rows);
  s.count = (int32_t*)take(4 * s.runs);
  s.total = s.count;
  s.run_key = s.key;
  s.run_order = s.order;
  if (s.runs > 1) {
    s.total = (int32_t*)take(4);
    s.run_key = (int32_t*)take(4 * rows);
    s.run_order = (int32_t*)take(4 * rows);
  }
  s.partial = (float*)take(8 * s.parts * cols);
  s.bytes = used;
  return s;
}

}  // namespace

extern "C" {

coat_status_t coat_fp8_embedding(const coat_embedding_args_t* a, hipStream_t stream) {
  if (!a) return COAT_ERR_NULL_POINTER;
  if (!embed_sizes_ok(a->rows, a->vocab, a->cols)) return COAT_ERR_INVALID_VALUE;
  if (a->table && a->table_codes) return COAT_ERR_INVALID_VALUE;
  const float scale = a->table_scale * a->scale;
  if (!isfinite(a->table_scale) || !isfinite(a->scale) || !isfinite(scale)) return COAT_ERR_INVALID_VALUE;
  if (a->rows == 0 || a->cols == 0) return COAT_OK;
  if (!a->tokens || !a->out || (a->vocab > 0 && !a->table && !a->table_codes)) return COAT_ERR_NULL_POINTER;
  if (!aligned(a->table, 16) || !aligned(a->table_codes, 16) || !aligned(a->tokens, 8) || !aligned(a->out, 16))
    return COAT_ERR_MISALIGNED;
  LookupParams p;
  memset(&p, 0, sizeof(p));
  p.table = a->table_codes ? a->table_codes : (const uint8_t*)a->table;
  p.tokens = a->tokens;
  p.out = a->out;
  p.vocab = a->vocab;
  p.chunks = (uint32_t)(a->cols / 8);
  p.total = (uint32_t)(a->rows * (a->cols / 8));
  p.scale = scale;
  void* args[] = {&p};
  const void* fn = a->table_codes ? reinterpret_cast<const void*>(&embedding_kernel<true>)
                                  : reinterpret_cast<const void*>(&embedding_kernel<false>);
  const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)up(p.total, 512)), dim3(256), args, 0, stream);
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

int64_t coat_fp8_embedding_bwd_workspace(int64_t rows, int64_t vocab, int64_t cols) {
  if (!embed_sizes_ok(rows, vocab, cols)) return -1;
  return rows == 0 || vocab == 0 || cols == 0 ? 0 : space_of(nullptr, rows, cols).bytes;
}

coat_status_t coat_fp8_embedding_bwd(const coat_embedding_bwd_args_t* a, hipStream_t stream) {
  if (!a) return COAT_ERR_NULL_POINTER;
  const int64_t rows = a->rows, vocab = a->vocab, cols = a->cols;
  if (!embed_sizes_ok(rows, vocab, cols) || !isfinite(a->scale)) return COAT_ERR_INVALID_VALUE;
  if (a->dw_bf16 && (a->dw_f32 || a->accumulate)) return COAT_ERR_INVALID_VALUE;
  if (vocab == 0 || cols == 0) return COAT_OK;
  if (!a->dw_bf16 && !a->dw_f32) return COAT_ERR_NULL_POINTER;
  if (rows > 0 && (!a->dy || !a->tokens || !a->workspace)) return COAT_ERR_NULL_POINTER;
  if (!aligned(a->dy, 16) || !aligned(a->tokens, 8) || !aligned(a->dw_bf16, 16) || !aligned(a->dw_f32, 16) ||
      !aligned(a->workspace, 16))
    return COAT_ERR_MISALIGNED;
  const Space s = space_of(a->workspace, rows, cols);
  if (rows > 0 && a->workspace_bytes < s.bytes) return COAT_ERR_INVALID_VALUE;
  const int mode = a->dw_bf16 ? kBF16 : a->accumulate ? kF32Add : kF32;
  void* dw = a->dw_bf16 ? (void*)a->dw_bf16 : (void*)a->dw_f32;
  if (rows == 0 && mode == kF32Add) return COAT_OK;

  SortParams q;
  memset(&q, 0, sizeof(q));
  q.tokens = a->tokens;
  q.key = s.run_key;
  q.order = s.run_order;
  q.count = s.count;
  q.rows = rows;
  q.vocab = vocab;
  q.sort_blocks = (int32_t)up(rows, 64);
  if (mode != kF32Add) {
    q.dw = (uint8_t*)dw;
    q.dw_bytes = vocab * cols * (mode == kBF16 ? 2 : 4);
  }
  const int64_t fill = up(q.dw_bytes, 16384);
  void* sort_args[] = {&q};
  hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&sort_kernel),
                                 dim3((unsigned)(q.sort_blocks + (fill < 2048 ? fill : 2048))), dim3(1024), sort_args, 0, stream);
  if (e == hipSuccess && s.runs > 1) {
    MergeParams m = {s.run_key, s.run_order, s.count, s.key, s.order, s.total, s.runs};
    void* args[] = {&m};
    e = hipLaunchKernel(reinterpret_cast<const void*>(&merge_kernel), dim3((unsigned)up(rows, 256)), dim3(256), args, 0,
                        stream);
  }
  if (e == hipSuccess && rows > 0) {
    SumParams p;
    memset(&p, 0, sizeof(p));
    p.dy = a->dy;
    p.key = s.key;
    p.order = s.order;
    p.total = s.total;
    p.partial = s.partial;
    p.dw = dw;
    p.cols = cols;
    p.parts = s.parts;
    p.width = 1;
    while (p.width < 256 && 8 * p.width < cols) p.width *= 2;
    p.mode = mode;
    p.scale = a->scale;
    void* args[] = {&p};
    const dim3 grid((unsigned)up(s.parts, 256 / p.width), (unsigned)up(cols, 8 * p.width));
    e = hipLaunchKernel(reinterpret_cast<const void*>(&sum_kernel), grid, dim3(256), args, 0, stream);
    if (e == hipSuccess)
      e = hipLaunchKernel(reinterpret_cast<const void*>(&join_kernel), grid, dim3(256), args, 0, stream);
  }
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

}  // extern "C"
