// Embedding and its gradient (include/fp8lin_train.h has the definitions).
//
// Lookup: HBM-bound, a row read and a row written for each token (8192 tokens of
// 8192 columns from fp32: 58 us, 6.9 TB/s of both, frequent rows from the caches).
//
// Gradient.  Tokens are sorted by id, stably, so that the rows of an id lie
// together in the tokens' order; then rows are added without atomics, in an
// order that does not depend on the launch.  The sort is a radix sort by digits
// of up to nine bits.  Up to kTile tokens it is one workgroup's, in LDS, while
// the others of its launch write the gradient's zeros; more tokens take three
// launches a digit.  The sums: sorted positions are cut into chunks of kChunk; a
// chunk writes the ids that lie whole in it, and leaves the sums of those that
// reach past its ends in the workspace, which a last kernel adds in order.
// HBM-bound by the gradient's writing: vocab x d floats, and dout read once (4095
// tokens, 32000 x 5120: 144 us, of which 111 clear; 2048 tokens, 50257 x 768: 36).
// Tiles add the later digits' launches, beside which nothing is cleared, and places
// that few workgroups find (32768 tokens, 32000 x 4096: 270 us, 152 at 5.2 TB/s).
#include <algorithm>

#include "norm_kernel.h"
#include "quotient.h"

namespace fp8lin {
namespace {

__device__ __forceinline__ int64_t id_at(const void* ids, bool wide, int64_t t) {
  return wide ? static_cast<const int64_t*>(ids)[t] : (int64_t)static_cast<const int32_t*>(ids)[t];
}
// A unit's element in its row, and what is left of the row there.
struct Unit {
  int64_t row;
  int col, left;
};

template <int DT>
__device__ __forceinline__ void store_past(void* p, int64_t i, const float (&v)[4]) {
  if constexpr (DT == FP8_IN_FP32)
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(static_cast<float*>(p) + i));
  else
    __builtin_nontemporal_store(u32x2{bf16x2(v[0], v[1]), bf16x2(v[2], v[3])},
                                reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + i));
}

// ---------------------------------------------------------------- lookup
struct LookupArgs {
  const void* ids;
  bool wide;
  int64_t tokens, vocab;
  const void* table;
  int d, units;  // units of four elements of a row
  float scale;
  void* out;
  uint32_t first;
};

// Units of all rows in turn, U of a lane, a workgroup's width apart.  Large
// outputs are stored past the caches, which keep the table's frequent rows (8192
// rows of 4096 bf16 from 50257: 22 -> 19 us; loads past the caches took 35).
template <int TT, int OT, bool WHOLE, int U>
__global__ __launch_bounds__(256) void embedding_fwd_kernel(LookupArgs a) {
  const int64_t base = (int64_t)(a.first + blockIdx.x) * (256 * U);
  const int64_t row0 = quotient(base, a.units);
  const int rem = (int)(base - row0 * a.units) + threadIdx.x;
  Raw<TT> raw[U];
  Unit at[U];
  bool there[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t x = (uint32_t)rem + 256 * i, r = x / (uint32_t)a.units;
    at[i].row = row0 + r;
    at[i].col = 4 * (int)(x - r * (uint32_t)a.units);
    at[i].left = a.d - at[i].col;
    there[i] = at[i].row < a.tokens;
    raw[i] = Raw<TT>{};
    if (there[i]) {
      const int64_t id = id_at(a.ids, a.wide, at[i].row);
      if (id >= 0 && id < a.vocab) raw[i] = load_raw<TT, WHOLE, false>(a.table, id * a.d + at[i].col, at[i].left);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (!there[i]) continue;
    float v[4];
    unpack<TT>(raw[i], v);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] *= a.scale;
    const int64_t to = at[i].row * a.d + at[i].col;
    if constexpr (U > 1 && WHOLE) store_past<OT>(a.out, to, v);
    else store_as<OT, WHOLE>(a.out, to, at[i].left, v);
  }
}

// ---------------------------------------------------------------- sort
constexpr int kSortWaves = 16, kSortThreads = 64 * kSortWaves;
constexpr int kItems = 16;                       // of a lane
constexpr int kTile = kSortThreads * kItems;     // tokens of a workgroup
constexpr int kMaxDigit = 9, kBins = 1 << kMaxDigit;

struct SortArgs {
  const void* ids;
  bool wide;
  int64_t tokens, vocab;
  int passes, bits;           // digits, and the bits of each
  uint32_t *key, *order;      // sorted; a key of vocab: no token of the table
  uint32_t *key2, *order2;    // more than one tile: between passes
  uint32_t* hist;             // [bins][tiles]
  int tiles;
  float* zero;                // cleared by the workgroups behind the tiles', or null
  int64_t zeros;              // floats
};

__device__ __forceinline__ uint32_t key_at(const SortArgs& a, int64_t t) {
  const int64_t id = id_at(a.ids, a.wide, t);
  return id >= 0 && id < a.vocab ? (uint32_t)id : (uint32_t)a.vocab;
}

// Workgroups past the sorting ones clear the gradient, one store a lane: many
// short workgroups sweep the memory in order (655 MB in 105 us, 6.2 TB/s; a
// resident grid that strides over it 147).
__device__ __forceinline__ void clear_share(const SortArgs& a, int sorting) {
  const int64_t groups = (int64_t)gridDim.x - sorting, units = (a.zeros + 3) / 4;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t i = ((int64_t)blockIdx.x - sorting) * kSortThreads + threadIdx.x; i < units; i += groups * kSortThreads) {
    if (4 * i + 4 <= a.zeros) {
      *reinterpret_cast<f32x4*>(a.zero + 4 * i) = zero;
    } else {
      for (int64_t j = 4 * i; j < a.zeros; ++j) a.zero[j] = 0.0f;
    }
  }
}

// A wave's LDS operations complete in order; this keeps the compiler to it.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

struct SortShared {
  uint16_t count[kSortWaves][kBins];  // of a wave's items with that digit, then their first place
  uint32_t wave_total[kSortWaves];
};

// The places of a tile's n items when they are sorted by one digit, stably.
// Items lie wave by wave, `items` of a lane: item (wave, i, lane) is number wave
// * 64 * items + 64 i + lane.  first_of: receives the first place of each digit.
__device__ __forceinline__ void digit_places(const uint32_t (&key)[kItems], int items, int n, int shift,
                                             int bits, SortShared& s, uint32_t (&place)[kItems], uint32_t* first_of) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, bins = 1 << bits;
  for (int b = lane; b < bins; b += 64) s.count[wave][b] = 0;
  wave_fence();
  const uint64_t below = ((uint64_t)1 << lane) - 1;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (i >= items) break;
    const bool there = wave * 64 * items + 64 * i + lane < n;
    const uint32_t digit = (key[i] >> shift) & (bins - 1);
    uint64_t same = __ballot(there);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((digit >> b) & 1);
      same &= (digit >> b) & 1 ? set : ~set;
    }
    const uint32_t before = there ? s.count[wave][digit] : 0;
    place[i] = before + __popcll(same & below);
    wave_fence();
    if (there && (same & below) == 0) s.count[wave][digit] = (uint16_t)(before + __popcll(same));
    wave_fence();
  }
  __syncthreads();
  // first places: digits in order, within a digit the waves in order
  uint32_t total = 0;
  if ((int)threadIdx.x < bins)
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = s.count[w][threadIdx.x];
      s.count[w][threadIdx.x] = (uint16_t)total;
      total += c;
    }
  uint32_t upto = total;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = __shfl_up(upto, off, 64);
    if (lane >= off) upto += o;
  }
  if (lane == 63) s.wave_total[wave] = upto;
  __syncthreads();
  uint32_t base = upto - total;
  for (int w = 0; w < wave; ++w) base += s.wave_total[w];
  if ((int)threadIdx.x < bins) first_of[threadIdx.x] = base;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const uint32_t digit = (key[i] >> shift) & (bins - 1);
    if (i < items && wave * 64 * items + 64 * i + lane < n) place[i] += s.count[wave][digit] + first_of[digit];
  }
}

// Up to kTile tokens: every digit in LDS.
__global__ __launch_bounds__(kSortThreads) void embedding_sort_kernel(SortArgs a) {
  __shared__ SortShared s;
  __shared__ uint32_t first_of[kBins];
  __shared__ uint32_t keys[kTile];
  __shared__ uint16_t orders[kTile];
  if (blockIdx.x > 0) return clear_share(a, 1);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = (int)a.tokens;
  const int items = (n + kSortThreads - 1) / kSortThreads, mine = wave * 64 * items + lane;
  auto there = [&](int i) { return i < items && mine + 64 * i < n; };
  uint32_t key[kItems], order[kItems], place[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    order[i] = mine + 64 * i;
    key[i] = there(i) ? key_at(a, mine + 64 * i) : 0xFFFFFFFFu;
  }
  for (int pass = 0; pass < a.passes; ++pass) {
    digit_places(key, items, n, pass * a.bits, a.bits, s, place, first_of);
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (there(i)) {
        keys[place[i]] = key[i];
        orders[place[i]] = (uint16_t)order[i];
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (there(i)) {
        key[i] = keys[mine + 64 * i];
        order[i] = orders[mine + 64 * i];
      }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kItems; ++i)
    if (there(i)) {
      a.key[mine + 64 * i] = key[i];
      a.order[mine + 64 * i] = order[i];
    }
}

// More tokens.  A pass: how many items of each digit a tile has, where the
// digits of the tiles start, and the items to their places.
struct Pass {
  const uint32_t *key, *order;  // null: the first pass, from the ids
  uint32_t *to_key, *to_order;
  int shift, bits;
};
__device__ __forceinline__ uint32_t pass_key(const SortArgs& a, const Pass& p, int64_t t) {
  return p.key ? p.key[t] : key_at(a, t);
}
__global__ __launch_bounds__(kSortThreads) void embedding_count_kernel(SortArgs a, Pass p) {
  __shared__ uint32_t count[kBins];
  if ((int)blockIdx.x >= a.tiles) return clear_share(a, a.tiles);
  const int bins = 1 << p.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) count[b] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * kTile, t1 = min(t0 + kTile, a.tokens);
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kSortThreads)
    atomicAdd(&count[(pass_key(a, p, t) >> p.shift) & (bins - 1)], 1u);  // (a count: its order does not matter)
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) a.hist[(int64_t)b * a.tiles + blockIdx.x] = count[b];
}
__global__ __launch_bounds__(kSortThreads) void embedding_scan_kernel(SortArgs a, Pass p) {
  __shared__ uint32_t wave_total[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = ((int64_t)1 << p.bits) * a.tiles;
  uint32_t base = 0;
  for (int64_t i0 = 0; i0 < n; i0 += kSortThreads) {
    const int64_t i = i0 + threadIdx.x;
    const uint32_t v = i < n ? a.hist[i] : 0;
    uint32_t upto = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t o = __shfl_up(upto, off, 64);
      if (lane >= off) upto += o;
    }
    if (lane == 63) wave_total[wave] = upto;
    __syncthreads();
    uint32_t before = base;
    for (int w = 0; w < kSortWaves; ++w) {
      if (w < wave) before += wave_total[w];
      base += wave_total[w];
    }
    if (i < n) a.hist[i] = before + upto - v;
    __syncthreads();
  }
}
__global__ __launch_bounds__(kSortThreads) void embedding_place_kernel(SortArgs a, Pass p) {
  __shared__ SortShared s;
  __shared__ uint32_t first_of[kBins];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, bins = 1 << p.bits;
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int n = (int)min((int64_t)kTile, a.tokens - t0), mine = wave * 64 * kItems + lane;
  uint32_t key[kItems], order[kItems], place[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const bool there = mine + 64 * i < n;
    key[i] = there ? pass_key(a, p, t0 + mine + 64 * i) : 0xFFFFFFFFu;
    order[i] = there && p.order ? p.order[t0 + mine + 64 * i] : (uint32_t)(t0 + mine + 64 * i);
  }
  digit_places(key, kItems, n, p.shift, p.bits, s, place, first_of);
#pragma unroll
  for (int i = 0; i < kItems; ++i)
    if (mine + 64 * i < n) {
      const uint32_t digit = (key[i] >> p.shift) & (bins - 1);
      const uint32_t to = a.hist[(int64_t)digit * a.tiles + blockIdx.x] + place[i] - first_of[digit];
      p.to_key[to] = key[i];
      p.to_order[to] = order[i];
    }
}

// ---------------------------------------------------------------- sums
constexpr int kChunk = 16;  // sorted positions, whose rows are all on their way at once

struct SumArgs {
  const void* dout;
  const uint32_t *key, *order;
  int64_t tokens, vocab, d;
  float scale;
  bool accumulate;
  float* dtable;
  float* part;     // [chunks][2][d]: sums that reach past the chunk's first, its last position
  int64_t chunks;
  float* span;     // [chunks / kSpan][d]: sums of spans of chunks, or null
  int cols;        // waves across a row, 256 columns each
  uint32_t first;
};

template <bool WHOLE>
__device__ __forceinline__ void store_sum(const SumArgs& a, uint32_t id, int col, int left, const float (&sum)[4]) {
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = sum[e] * a.scale;
  const int64_t at = (int64_t)id * a.d + col;
  if (a.accumulate) {
    float was[4];
    unpack<FP8_IN_FP32>(load_raw<FP8_IN_FP32, WHOLE, false>(a.dtable, at, left), was);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += was[e];
  }
  store_as<FP8_IN_FP32, WHOLE>(a.dtable, at, left, v);
}

// A chunk and 256 columns a wave.  The chunk's ids and rows are scalars.
template <int DT, bool WHOLE>
__global__ __launch_bounds__(256) void embedding_sum_kernel(SumArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t g = (int64_t)(a.first + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t chunk = quotient(g, a.cols), p0 = chunk * kChunk;
  if (chunk >= a.chunks) return;
  const int col = ((int)(g - chunk * a.cols) * 64 + lane) * 4, left = (int)a.d - col;
  const int n = (int)min((int64_t)kChunk, a.tokens - p0);
  // lane i: the id at position p0 - 1 + i (none before the first and after the
  // last position), and the row at p0 + i
  const int64_t at = p0 - 1 + lane;
  constexpr uint32_t kNoId = 0xFFFFFFFFu;
  const uint32_t my_key = lane < n + 2 && at >= 0 && at < a.tokens ? a.key[at] : kNoId;
  const uint32_t my_row = lane < n ? a.order[p0 + lane] : 0;
  auto key = [&](int i) { return (uint32_t)__builtin_amdgcn_readlane((int)my_key, i + 1); };
  Raw<DT> raw[kChunk];
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    raw[i] = Raw<DT>{};
    const int64_t row = (uint32_t)__builtin_amdgcn_readlane((int)my_row, i);
    if (i < n && key(i) < (uint32_t)a.vocab && left > 0)
      raw[i] = load_raw<DT, WHOLE, true>(a.dout, row * a.d + col, left);
  }
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  bool from_before = key(-1) == key(0);  // the run goes on from the chunk before
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    if (i < n && key(i) < (uint32_t)a.vocab) {
      float v[4];
      unpack<DT>(raw[i], v);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += v[e];
      const bool goes_on = key(i + 1) == key(i);
      if (!goes_on || i + 1 == n) {
        if (left > 0) {
          if (from_before) store_as<FP8_IN_FP32, WHOLE>(a.part, (2 * chunk) * a.d + col, left, sum);
          else if (goes_on) store_as<FP8_IN_FP32, WHOLE>(a.part, (2 * chunk + 1) * a.d + col, left, sum);
          else store_sum<WHOLE>(a, key(i), col, left, sum);
        }
        from_before = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = 0.0f;
      }
    }
  }
}

// Rows of partial sums on their way at once.
constexpr int kAhead = 16;
// Of many tokens an id may have very many (padding that is a token): the chunks of
// a span that it fills are added before the join, all spans at the same time
// (65536 rows of 1024, all of one id: 1323 -> 126 us; 16384 of 768: 144 -> 63, and
// 59 -> 61 where no id fills a span, which is the launch: none for fewer tokens).
constexpr int kSpan = 64, kManyChunks = 512;

// Whether span s lies in a run of `id` that its first chunk is a part of.
__device__ __forceinline__ bool fills_span(const SumArgs& a, int64_t s, uint32_t id) {
  return (s + 1) * kSpan <= a.chunks && a.key[min((s + 1) * kSpan * kChunk, a.tokens) - 1] == id;
}

template <bool WHOLE>
__global__ __launch_bounds__(256) void embedding_span_kernel(SumArgs a) {
  const int64_t g = (int64_t)(a.first + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t s = quotient(g, a.cols), p0 = s * kSpan * kChunk;
  if ((s + 1) * kSpan > a.chunks || s == 0) return;
  const int col = ((int)(g - s * a.cols) * 64 + (int)(threadIdx.x & 63)) * 4, left = (int)a.d - col;
  const uint32_t id = a.key[p0];
  if (left <= 0 || id >= (uint32_t)a.vocab || a.key[p0 - 1] != id || !fills_span(a, s, id)) return;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c0 = 0; c0 < kSpan; c0 += kAhead) {
    Raw<FP8_IN_FP32> raw[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      raw[i] = load_raw<FP8_IN_FP32, WHOLE, false>(a.part, 2 * (s * kSpan + c0 + i) * a.d + col, left);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float v[4];
      unpack<FP8_IN_FP32>(raw[i], v);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += v[e];
    }
  }
  store_as<FP8_IN_FP32, WHOLE>(a.span, s * a.d + col, left, sum);
}

// Ids whose rows begin in one chunk and end in another: the chunks' sums, or those
// of whole spans, in order, a wave for 256 columns.
template <bool WHOLE>
__global__ __launch_bounds__(256) void embedding_join_kernel(SumArgs a) {
  const int64_t g = (int64_t)(a.first + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t chunk = quotient(g, a.cols), p0 = chunk * kChunk, p1 = p0 + kChunk;
  if (chunk + 1 >= a.chunks) return;  // nothing goes on from the last one
  const int lane = threadIdx.x & 63, col = ((int)(g - chunk * a.cols) * 64 + lane) * 4, left = (int)a.d - col;
  const uint32_t id = a.key[p1 - 1];
  if (id >= (uint32_t)a.vocab || a.key[p1] != id) return;
  if (p0 > 0 && a.key[p0 - 1] == id && a.key[p0] == id) return;  // begun in an earlier one
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (left > 0) unpack<FP8_IN_FP32>(load_raw<FP8_IN_FP32, WHOLE, false>(a.part, (2 * chunk + 1) * a.d + col, left), sum);
  for (int64_t c0 = chunk + 1; c0 < a.chunks && a.key[c0 * kChunk] == id;) {
    const bool spans = a.span && c0 % kSpan == 0 && fills_span(a, c0 / kSpan, id);
    const int64_t unit = spans ? kSpan : 1, step = spans ? a.d : 2 * a.d;
    const float* from = spans ? a.span + c0 / kSpan * a.d : a.part + 2 * c0 * a.d;
    // how many there are, a lane each (sorted: they come first); chunks up to
    // where the next span begins
    const int64_t c = c0 + lane * unit;
    const int most = (int)min((int64_t)kAhead, spans || !a.span ? kAhead : kSpan - c0 % kSpan);
    const bool there = lane < most && c < a.chunks && (spans ? fills_span(a, c / kSpan, id) : a.key[c * kChunk] == id);
    const int taken = __popcll(__ballot(there));
    Raw<FP8_IN_FP32> raw[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      raw[i] = Raw<FP8_IN_FP32>{};
      if (i < taken && left > 0) raw[i] = load_raw<FP8_IN_FP32, WHOLE, false>(from, i * step + col, left);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float v[4];
      unpack<FP8_IN_FP32>(raw[i], v);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += v[e];
    }
    c0 += taken * unit;
  }
  if (left > 0) store_sum<WHOLE>(a, id, col, left, sum);
}

int64_t aligned(int64_t bytes) { return (bytes + 255) & ~(int64_t)255; }
struct GradPlan {
  int64_t tiles, chunks;
  int passes, bits;
  int64_t spans;                                              // 0: the join takes chunks alone
  int64_t key, order, key2, order2, hist, part, span, bytes;  // offsets
};
GradPlan plan_of(int64_t tokens, int64_t vocab, int64_t d) {
  GradPlan p{};
  p.tiles = (tokens + kTile - 1) / kTile;
  p.chunks = (tokens + kChunk - 1) / kChunk;
  int bits = 1;
  while ((vocab >> bits) != 0) ++bits;  // keys 0 .. vocab
  p.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  p.bits = (bits + p.passes - 1) / p.passes;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t r = at;
    at += aligned(bytes);
    return r;
  };
  p.key = take(4 * tokens);
  p.order = take(4 * tokens);
  if (p.tiles > 1) {
    p.key2 = take(4 * tokens);
    p.order2 = take(4 * tokens);
    p.hist = take(4 * ((int64_t)1 << p.bits) * p.tiles);
  }
  const int64_t row = 4 * ((d + 3) & ~(int64_t)3);
  p.part = take(2 * p.chunks * row);
  p.spans = p.chunks > kManyChunks ? p.chunks / kSpan : 0;
  p.span = take(p.spans * row);
  p.bytes = at;
  return p;
}

}  // namespace

hipError_t launch_embedding_fwd(const void* ids, bool wide, int64_t tokens, const void* table, int table_dtype,
                                int64_t vocab, int64_t d, float scale, void* out, int out_dtype, hipStream_t stream) {
  LookupArgs a{ids, wide, tokens, vocab, table, (int)d, (int)((d + 3) / 4), scale, out, 0};
  const int64_t units = tokens * a.units;
  auto run = [&](auto tt, auto ot, auto whole, auto u) {
    constexpr int U = decltype(u)::value;
    in_stretches((units + 256 * U - 1) / (256 * U), 256, [&](uint32_t first, uint32_t count) {
      a.first = first;
      hipLaunchKernelGGL((embedding_fwd_kernel<decltype(tt)::value, decltype(ot)::value, decltype(whole)::value, U>),
                         dim3(count), dim3(256), 0, stream, a);
    });
  };
  using std::integral_constant;
  auto sized = [&](auto tt, auto ot, auto whole) {
    if (units > 1024 * 1024) run(tt, ot, whole, integral_constant<int, 4>{});
    else run(tt, ot, whole, integral_constant<int, 1>{});
  };
  auto typed = [&](auto tt, auto ot) {
    if (d % 4 == 0) sized(tt, ot, std::true_type{});
    else sized(tt, ot, std::false_type{});
  };
  constexpr integral_constant<int, FP8_IN_BF16> b16{};
  constexpr integral_constant<int, FP8_IN_FP32> f32{};
  if (table_dtype == FP8_IN_BF16) out_dtype == FP8_IN_BF16 ? typed(b16, b16) : typed(b16, f32);
  else out_dtype == FP8_IN_BF16 ? typed(f32, b16) : typed(f32, f32);
  return hipGetLastError();
}

int64_t embedding_bwd_workspace_bytes(int64_t tokens, int64_t vocab, int64_t d) {
  return plan_of(tokens, vocab, d).bytes;
}

hipError_t launch_embedding_bwd(const EmbeddingGrad& g, void* ws, hipStream_t stream) {
  const GradPlan p = plan_of(g.tokens, g.vocab, g.d);
  uint8_t* w = static_cast<uint8_t*>(ws);
  auto words = [&](int64_t at) { return reinterpret_cast<uint32_t*>(w + at); };
  SortArgs s{};
  s.ids = g.ids, s.wide = g.wide, s.tokens = g.tokens, s.vocab = g.vocab;
  s.passes = p.passes, s.bits = p.bits, s.tiles = (int)p.tiles;
  s.key = words(p.key), s.order = words(p.order);
  s.key2 = words(p.key2), s.order2 = words(p.order2), s.hist = words(p.hist);
  int clearing = 0;
  if (!g.accumulate) {
    s.zero = g.dtable;
    s.zeros = g.vocab * g.d;
    clearing = (int)std::min<int64_t>(1 << 21, (s.zeros + 4 * kSortThreads - 1) / (4 * kSortThreads));
  }
  if (p.tiles <= 1) {
    hipLaunchKernelGGL(embedding_sort_kernel, dim3(1 + clearing), dim3(kSortThreads), 0, stream, s);
  } else {
    Pass pass{nullptr, nullptr, nullptr, nullptr, 0, p.bits};
    for (int i = 0; i < p.passes; ++i) {
      const bool last_here = (p.passes - 1 - i) % 2 == 0;  // the last pass ends in key, order
      pass.to_key = last_here ? s.key : s.key2;
      pass.to_order = last_here ? s.order : s.order2;
      pass.shift = i * p.bits;
      hipLaunchKernelGGL(embedding_count_kernel, dim3((uint32_t)p.tiles + (i == 0 ? clearing : 0)), dim3(kSortThreads),
                         0, stream, s, pass);
      hipLaunchKernelGGL(embedding_scan_kernel, dim3(1), dim3(kSortThreads), 0, stream, s, pass);
      hipLaunchKernelGGL(embedding_place_kernel, dim3((uint32_t)p.tiles), dim3(kSortThreads), 0, stream, s, pass);
      pass.key = pass.to_key;
      pass.order = pass.to_order;
    }
  }
  SumArgs a{};
  a.dout = g.dout, a.key = s.key, a.order = s.order;
  a.tokens = g.tokens, a.vocab = g.vocab, a.d = g.d;
  a.scale = g.scale, a.accumulate = g.accumulate, a.dtable = g.dtable;
  a.part = reinterpret_cast<float*>(w + p.part);
  a.chunks = p.chunks;
  a.span = p.spans > 0 ? reinterpret_cast<float*>(w + p.span) : nullptr;
  a.cols = (int)((g.d + 255) / 256);
  auto launch = [&](auto kernel, int64_t waves) {
    in_stretches((waves + 3) / 4, 256, [&](uint32_t first, uint32_t count) {
      a.first = first;
      hipLaunchKernelGGL(kernel, dim3(count), dim3(256), 0, stream, a);
    });
  };
  const bool whole = g.d % 4 == 0;
  if (g.dout_dtype == FP8_IN_BF16)
    launch(whole ? embedding_sum_kernel<FP8_IN_BF16, true> : embedding_sum_kernel<FP8_IN_BF16, false>,
           p.chunks * a.cols);
  else
    launch(whole ? embedding_sum_kernel<FP8_IN_FP32, true> : embedding_sum_kernel<FP8_IN_FP32, false>,
           p.chunks * a.cols);
  if (p.spans > 0) launch(whole ? embedding_span_kernel<true> : embedding_span_kernel<false>, p.spans * a.cols);
  launch(whole ? embedding_join_kernel<true> : embedding_join_kernel<false>, (p.chunks - 1) * a.cols);
  return hipGetLastError();
}

}  // namespace fp8lin
