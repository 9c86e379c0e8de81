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
// table.  The one rounding is the result's; codes and BF16 are exact in FP32.
// A thread copies two chunks of eight values, 4 KB apart in the output, so that
// two chains of loads (token, row) are in flight.  Bound by the writes and by
// the table's rows that are not in a cache: 8191 rows of 4096 columns from an
// 8-bit table 13.6 us (5.9 TB/s of 80 MB, of which counters see 20 MB read),
// from BF16 17.5 (5.4); one row 1.8 us, in 5.2 from call to call.
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
//
// It cannot do without reading dy and writing dW once, 329 MB for 8192 rows of
// 4096 columns over 32000 rows of BF16: 70 us at a copy's rate.  Measured 74.4
// (under the profiler sort 23, sums 40, join 15), a part of dW's zeros written
// in each of the three.  What is left is the sort's and the join's latency,
// where the memory is not busy all the time.  2048 columns and 4099 rows over
// 50001 rows of FP32: 85.6 (sort 16, sums 55, join 15), 90 at a copy's rate.

enum Out { kBF16 = 0, kF32 = 1, kF32Add = 2 };

constexpr int kSortRows = 16384;   // rows whose keys a block's registers hold
constexpr int kPart = 32;          // sorted rows of a part
constexpr int64_t kFill = 64 << 20;   // bytes of dw zeroed beside the sort, and beside the join, at most

struct SortParams {
  const int64_t* tokens;
  int32_t* key;             // sorted tokens of each run of kSortRows rows
  int32_t* order;           // and their rows
  int32_t* count;           // of each run: rows whose token is in the table
  int64_t rows, vocab;
  uint8_t* dw;              // its first fill_bytes are zeroed by the blocks behind the sort's
  int64_t fill_bytes;
  int32_t sort_blocks;
};

constexpr int kSortBlock = 32;     // rows that a block places

// A row's place in its run: how many keys are smaller, or equal and earlier:
// rows^2 comparisons, but 64 of them an instruction and all rows at once, where
// a sort in passes is a chain of launches or barriers.
// A block of 16 waves places 32 rows: a wave holds a sixteenth of the run's
// keys in its lanes' registers (kEach each), and for each row compares 64 at a
// time and counts the bits of the result.  key_of(i): the key of the run's row
// i.  Returns, in lane r, the wave's count for row r; live: its keys that are
// tokens.
template <int kEach, class Key>
__device__ __forceinline__ int32_t count_below(int wave, int lane, int first, int32_t mine, int32_t none, Key key_of,
                                               int& live) {
  const int own = first / 64 - wave * kEach;   // the 64 keys that hold the block's rows, if the wave has them
  int32_t key[kEach], own_key = none;
  live = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    int32_t k = key_of(64 * (wave * kEach + j) + lane);
    live += __popcll(__ballot(k < none));
    if (j == own) own_key = k, k = none;
    key[j] = j < own ? k - 1 : k;              // earlier keys count if equal: k - 1 < mine
  }
  int32_t counts = 0;
  const bool has_own = own >= 0 && own < kEach;
#pragma unroll 4
  for (int r = 0; r < kSortBlock; ++r) {
    const int32_t m = __builtin_amdgcn_readlane(mine, r);
    int c = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) c += __popcll(__ballot(key[j] < m));
    counts = lane == r ? c : counts;
  }
  if (has_own) {
    for (int r = 0; r < kSortBlock; ++r) {
      const int32_t m = __builtin_amdgcn_readlane(mine, r);
      const int c = __popcll(__ballot(own_key < m)) +
                    __popcll(__ballot(own_key == m) & (((uint64_t)1 << ((first + r) & 63)) - 1));
      counts += lane == r ? c : 0;
    }
  }
  return counts;
}

__global__ __launch_bounds__(1024) void sort_kernel(const SortParams p) {
  __shared__ int32_t below[16][kSortBlock], live_of[16];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  if ((int)blockIdx.x >= p.sort_blocks) {
    const int64_t stride = 16384 * (int64_t)(gridDim.x - p.sort_blocks);
    for (int64_t at = 16384 * (int64_t)(blockIdx.x - p.sort_blocks) + 16 * t; at < p.fill_bytes; at += stride)
      *reinterpret_cast<uint4*>(p.dw + at) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int64_t row0 = (int64_t)kSortBlock * blockIdx.x, run0 = row0 / kSortRows * kSortRows;
  const int n = (int)(p.rows - run0 < kSortRows ? p.rows - run0 : kSortRows);
  const int first = (int)(row0 - run0);    // of the block's rows in the run
  const int32_t none = (int32_t)p.vocab;   // behind every token
  auto key_of = [&](int i) {
    const int64_t token = i < n ? p.tokens[run0 + i] : -1;
    return token >= 0 && token < p.vocab ? (int32_t)token : none;
  };
  const int32_t mine = key_of(first + (lane & 31));
  int live;
  int32_t counts;
  if (n <= 1024) counts = count_below<1>(wave, lane, first, mine, none, key_of, live);
  else if (n <= 2048) counts = count_below<2>(wave, lane, first, mine, none, key_of, live);
  else if (n <= 4096) counts = count_below<4>(wave, lane, first, mine, none, key_of, live);
  else if (n <= 8192) counts = count_below<8>(wave, lane, first, mine, none, key_of, live);
  else counts = count_below<16>(wave, lane, first, mine, none, key_of, live);
  if (lane < kSortBlock) below[wave][lane] = counts;
  if (lane == 0) live_of[wave] = live;
  __syncthreads();
  if (t < kSortBlock && mine < none) {
    int32_t place = 0;
    for (int w = 0; w < 16; ++w) place += below[w][t];
    p.key[run0 + place] = mine;
    p.order[run0 + place] = (int32_t)(row0 + t);
  }
  if (first == 0 && t == 0) {
    int32_t all = 0;
    for (int w = 0; w < 16; ++w) all += live_of[w];
    p.count[run0 / kSortRows] = all;
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
  int64_t cols, vocab;
  int32_t parts, width;     // width: threads along the columns
  int32_t slabs;            // of the columns, for the blocks that sum
  int32_t sum_blocks;
  int64_t fill_from, fill_to;   // rows of dw that the launch's other blocks fill
  float scale;
};

// Eight of dw's values from before, for kF32Add.
struct Old {
  float4 a, b;
};

__device__ __forceinline__ Old load_old(const SumParams& p, int64_t v, int64_t col) {
  const float4* src = reinterpret_cast<const float4*>((const float*)p.dw + v * p.cols + col);
  return Old{src[0], src[1]};
}

template <int kMode>
__device__ __forceinline__ void store_row(const SumParams& p, int64_t v, int64_t col, float (&s)[8], const Old& old) {
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] *= p.scale;
  if constexpr (kMode == kBF16) {
    *reinterpret_cast<uint4*>((uint16_t*)p.dw + v * p.cols + col) = pack8(s);
  } else {
    float4 a = make_float4(s[0], s[1], s[2], s[3]), b = make_float4(s[4], s[5], s[6], s[7]);
    if constexpr (kMode == kF32Add) {
      a.x += old.a.x, a.y += old.a.y, a.z += old.a.z, a.w += old.a.w;
      b.x += old.b.x, b.y += old.b.y, b.z += old.b.z, b.w += old.b.w;
    }
    float4* dst = reinterpret_cast<float4*>((float*)p.dw + v * p.cols + col);
    dst[0] = a;
    dst[1] = b;
  }
}

__device__ __forceinline__ void store_partial(float* to, const float (&s)[8]) {
  reinterpret_cast<float4*>(to)[0] = make_float4(s[0], s[1], s[2], s[3]);
  reinterpret_cast<float4*>(to)[1] = make_float4(s[4], s[5], s[6], s[7]);
}

// Value `i` of a part's 32 lanes: those of the thread's half of the wave, or
// with kWide, where a wave's threads share their part, the first 32.
template <bool kWide>
__device__ __forceinline__ int32_t of_row(int32_t v, int i) {
  if constexpr (kWide) return __builtin_amdgcn_readlane(v, i);
  return __shfl(v, (threadIdx.x & 32) + i);
}

// One part of the sorted rows, eight columns a thread.
template <int kMode, bool kWide>
__device__ __forceinline__ void sum_part(const SumParams& p) {
  const int per = 256 / p.width, l32 = threadIdx.x & 31;
  const int slab = (int)(blockIdx.x % p.slabs), block = (int)(blockIdx.x / p.slabs);
  int part = block * per + threadIdx.x / p.width;
  if constexpr (kWide) part = __builtin_amdgcn_readfirstlane(part);
  const int64_t my_col = 8 * ((int64_t)slab * p.width + threadIdx.x % p.width);
  const int total = *p.total, first = part * kPart;
  // (threads past the last column or the last row stay: lanes look at rows for
  // each other)
  if (kWide && first >= total) return;
  const int n = first >= total ? 0 : first + kPart < total ? kPart : total - first;   // rows of the part
  const bool stored = my_col < p.cols && n > 0;
  const int64_t col = my_col < p.cols ? my_col : 0;
  float* partial = p.partial + 2 * (int64_t)part * p.cols + col;
  // lane i looks at row i
  const int at = n == 0 ? 0 : first + (l32 < n ? l32 : n - 1);
  int32_t key = 0, row = 0, next = -1, before = -1;
  if (total > 0) {
    key = p.key[at];
    row = p.order[at];
    if (at + 1 < total) next = p.key[at + 1];
    if (first > 0 && n > 0) before = p.key[first - 1];
  }
  const bool ends_here = l32 < n && (next != key || l32 == n - 1);
  const uint64_t ballot = __ballot(ends_here);
  const uint32_t ends = (uint32_t)(kWide || !(threadIdx.x & 32) ? ballot : ballot >> 32);   // rows that end a run, or the part
  const bool goes_on = n > 0 && of_row<kWide>(next, n > 0 ? n - 1 : 0) == of_row<kWide>(key, n > 0 ? n - 1 : 0);
  uint4 raw[kPart];
#pragma unroll
  for (int i = 0; i < kPart; ++i) raw[i] = load_stream16(p.dy + (int64_t)of_row<kWide>(row, i) * p.cols + col);
  // what dw holds, four rows ahead
  constexpr int kAhead = 4;
  Old old[kAhead];
  auto look_ahead = [&](int i) __attribute__((always_inline)) {
    if constexpr (kMode == kF32Add) {
      const int32_t v = of_row<kWide>(key, i);
      if ((ends >> i) & 1) old[i % kAhead] = load_old(p, v, col);
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) look_ahead(i);
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  bool head = before == of_row<kWide>(key, 0);   // the run at hand began in an earlier part
#pragma unroll
  for (int i = 0; i < kPart; ++i) {   // (rows from n on are in no run that ends)
    float f[8];
    unpack8(raw[i], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += f[e];
    const int32_t v = of_row<kWide>(key, i);
    if ((ends >> i) & 1) {
      if (stored) {
        if (head) store_partial(partial, s);
        else if (i == n - 1 && goes_on) store_partial(partial + p.cols, s);
        else store_row<kMode>(p, v, col, s, old[i % kAhead]);
      }
      head = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = 0.0f;
    }
    if (i + kAhead < kPart) look_ahead(i + kAhead);
  }
}

// No rows: a gradient of zeros.
__global__ __launch_bounds__(256) void zero_kernel(uint8_t* p, int64_t bytes) {
  for (int64_t at = 16 * ((int64_t)blockIdx.x * 256 + threadIdx.x); at < bytes; at += 4096 * (int64_t)gridDim.x)
    *reinterpret_cast<uint4*>(p + at) = make_uint4(0, 0, 0, 0);
}

constexpr int kFillRows = 16;   // rows of dW that a block looks through

// Zeros for those of kFillRows rows of dW whose token does not occur.
template <int kMode>
__device__ __forceinline__ void fill_rows(const SumParams& p, int64_t v0) {
  __shared__ int32_t present[kFillRows];
  const int t = threadIdx.x;
  if (t < kFillRows) {
    const int64_t v = v0 + t;
    const int total = *p.total;
    int lo = 0, hi = total;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (p.key[mid] < v) lo = mid + 1;
      else hi = mid;
    }
    present[t] = v >= p.fill_to || (lo < total && p.key[lo] == v);
  }
  __syncthreads();
  const int64_t bytes = p.cols * (kMode == kBF16 ? 2 : 4);
  for (int r = 0; r < kFillRows; ++r) {
    if (present[r]) continue;
    uint8_t* row = (uint8_t*)p.dw + (v0 + r) * bytes;
    for (int64_t at = 16 * t; at < bytes; at += 4096) *reinterpret_cast<uint4*>(row + at) = make_uint4(0, 0, 0, 0);
  }
}

// The first blocks sum, the others fill.
template <int kMode>
__global__ __launch_bounds__(256) void sum_kernel(const SumParams p) {
  if ((int)blockIdx.x >= p.sum_blocks) fill_rows<kMode>(p, p.fill_from + (int64_t)kFillRows * (blockIdx.x - p.sum_blocks));
  else if (p.width >= 64) sum_part<kMode, true>(p);
  else sum_part<kMode, false>(p);
}

// Joins a run that begins in a part and goes on behind it; kWide as above.
template <int kMode, bool kWide>
__device__ __forceinline__ void join_part(const SumParams& p) {
  const int per = 256 / p.width, lane = threadIdx.x & 63;
  const int slab = (int)(blockIdx.x % p.slabs), block = (int)(blockIdx.x / p.slabs);
  int part = block * per + threadIdx.x / p.width;
  if constexpr (kWide) part = __builtin_amdgcn_readfirstlane(part);
  const int64_t my_col = 8 * ((int64_t)slab * p.width + threadIdx.x % p.width);
  const bool stored = my_col < p.cols;
  const int64_t col = stored ? my_col : 0;
  const int total = *p.total, first = part * kPart, next = first + kPart;
  if (next >= total) return;
  const int32_t key = p.key[next - 1];
  if (p.key[next] != key) return;
  if (p.key[first] == key && first > 0 && p.key[first - 1] == key) return;   // it began before
  // The parts behind this one that it reaches into: those whose first row has
  // its token.
  int more = 1;
  if constexpr (kWide) {
    for (;; more += 64) {
      const int64_t at = next + (int64_t)kPart * (more + lane);
      const uint64_t in = __ballot(at < total && p.key[at < total ? at : next] == key);
      if (~in != 0) {
        more += __builtin_ctzll(~in);
        break;
      }
    }
  } else {
    while (next + kPart * more < total && p.key[next + kPart * more] == key) ++more;
  }
  Old old;
  if constexpr (kMode == kF32Add) old = load_old(p, key, col);
  float s[8];
  auto load = [&](int64_t slot, float (&f)[8]) {
    const float4* from = reinterpret_cast<const float4*>(p.partial + slot * p.cols + col);
    const float4 a = from[0], b = from[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  };
  load(2 * (int64_t)part + 1, s);
  for (int q = 1; q <= more; q += 8) {   // eight loads in flight
    float f[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) load(2 * (int64_t)(part + (q + i < more ? q + i : more)), f[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = q + i <= more ? s[e] + f[i][e] : s[e];
  }
  if (stored) store_row<kMode>(p, key, col, s, old);
}

template <int kMode>
__global__ __launch_bounds__(256) void join_kernel(const SumParams p) {
  if ((int)blockIdx.x >= p.sum_blocks) fill_rows<kMode>(p, p.fill_from + (int64_t)kFillRows * (blockIdx.x - p.sum_blocks));
  else if (p.width >= 64) join_part<kMode, true>(p);
  else join_part<kMode, false>(p);
}

template <int kMode>
hipError_t launch_sums(SumParams& p, int64_t late, hipStream_t stream) {
  void* args[] = {&p};
  auto blocks = [&] { return (unsigned)(p.sum_blocks + (p.fill_to - p.fill_from + kFillRows - 1) / kFillRows); };
  hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&sum_kernel<kMode>), dim3(blocks()), dim3(256), args, 0, stream);
  p.fill_from = p.fill_to;
  p.fill_to += late;
  if (e == hipSuccess)
    e = hipLaunchKernel(reinterpret_cast<const void*>(&join_kernel<kMode>), dim3(blocks()), dim3(256), args, 0, stream);
  return e;
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

  // Rows of dw without a token are zeroed in all three launches, so that the
  // memory is busy while the rows are sorted and while runs are joined: the
  // first ones before it is known which have a token (8192 x 4096 over 32000
  // rows in BF16: 75.3 us, 79.5 with all of them beside the sums; 2048 columns
  // over 50001 rows in FP32: 85.5, 93.8).
  const int64_t row_bytes = cols * (mode == kBF16 ? 2 : 4), most = kFill / row_bytes;
  const int64_t early = mode == kF32Add ? 0 : vocab / 4 < most ? vocab / 4 : most, late = early;
  hipError_t e = hipSuccess;
  if (rows > 0) {
    SortParams q = {a->tokens, s.run_key, s.run_order, s.count, rows, vocab, (uint8_t*)dw, early * row_bytes,
                    (int32_t)up(rows, kSortBlock)};
    void* args[] = {&q};
    const int64_t fill = up(q.fill_bytes, 65536);
    e = hipLaunchKernel(reinterpret_cast<const void*>(&sort_kernel), dim3((unsigned)(q.sort_blocks + fill)), dim3(1024),
                        args, 0, stream);
  }
  if (e == hipSuccess && s.runs > 1) {
    MergeParams m = {s.run_key, s.run_order, s.count, s.key, s.order, s.total, s.runs};
    void* args[] = {&m};
    e = hipLaunchKernel(reinterpret_cast<const void*>(&merge_kernel), dim3((unsigned)up(rows, 256)), dim3(256), args, 0,
                        stream);
  }
  SumParams p;
  memset(&p, 0, sizeof(p));
  p.dy = a->dy;
  p.key = s.key;
  p.order = s.order;
  p.total = s.total;
  p.partial = s.partial;
  p.dw = dw;
  p.cols = cols;
  p.vocab = vocab;
  p.parts = s.parts;
  p.width = 32;
  while (p.width < 256 && 8 * p.width < cols) p.width *= 2;
  p.slabs = (int32_t)up(cols, 8 * p.width);
  p.sum_blocks = (int32_t)(up(s.parts, 256 / p.width) * p.slabs);
  p.scale = a->scale;
  p.fill_from = early;
  p.fill_to = mode == kF32Add ? early : vocab - late;
  if (e == hipSuccess && rows == 0) {
    const int64_t bytes = vocab * row_bytes, blocks = up(bytes, 4096);
    void* zero[] = {&dw, (void*)&bytes};
    e = hipLaunchKernel(reinterpret_cast<const void*>(&zero_kernel), dim3((unsigned)(blocks < 16384 ? blocks : 16384)),
                        dim3(256), zero, 0, stream);
  } else if (e == hipSuccess) {
    e = mode == kBF16 ? launch_sums<kBF16>(p, late, stream)
        : mode == kF32 ? launch_sums<kF32>(p, late, stream) : launch_sums<kF32Add>(p, late, stream);
  }
  return e == hipSuccess ? COAT_OK : hip_fail(e);
}

}  // extern "C"
