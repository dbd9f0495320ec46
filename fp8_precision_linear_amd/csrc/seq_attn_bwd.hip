// Attention over packed sequences, backward: seq_attn.h has the mathematics.
//
// Probabilities are recomputed from q, k and lse, so nothing of the size of the
// logits is stored.  Two kinds of workgroups, each the owner of what it sums, so
// that no sum depends on an order of atomics: seven products where a kernel that
// adds dq from every key tile would need five.
//
// dq.  As the forward: 128 query rows of one head a workgroup, 32 a wave, q and
// dout in registers; keys and values through LDS.
//
// dk, dv.  128 keys of a key head at a time, 32 a wave, k and v in registers;
// the queries and dout of all its heads through LDS.
//
// A workgroup takes a tile of rows (of keys) where there are enough of them.
// Otherwise -- few heads, short batches -- the tiles' walks, of very different
// lengths under a causal mask, are laid one behind the other for each head and cut
// into equal shares, so that all workgroups run at the same time and end
// together; a cut walk's partial sums are joined in order by a last kernel.
//
// Both kinds run in one launch, behind a small one that leaves -lse log2(e) and
// -delta of every row and head.
//
// Large calls: two causal sequences of 3500-4096, 64 heads on 8 of 128, 1820-1870 us,
// 930 TFLOP/s of the seven products (50 us are the first kernel's, at HBM's rate, 29
// the join's); two of 4096, 32 heads of 128, everything seen, MFMA busy 48% of the
// SIMDs' cycles and the other vector instructions 30%, with little overlap, at 1.6 GHz
// (the power limit), no bank conflicts.  Heads of 256 hold one wave a SIMD: three of
// 2000, 16 on 4, 800 us.  Small calls are the launches' latency and the partial sums:
// 2 x 1024, 12 heads of 64, 45 us.
#include <algorithm>

#include "seq_attn.h"

namespace fp8lin {
namespace {

// Query rows of a tile of the dk, dv kernel.
template <int D>
constexpr int kQueriesOf = D == 256 ? 32 : 64;

// A key tile's walk: tiles of query rows from `lo` on, of each head of the group.
struct Walk {
  int lo, tiles;
};
template <int D>
__device__ __forceinline__ Walk walk_of(const SeqAttnArgs& a, int n, int k0) {
  constexpr int kQueries = kQueriesOf<D>;
  const int lo = a.causal ? k0 : 0;
  const int64_t hi = a.window ? (int64_t)min(k0 + kSeqRows, n) - 1 + a.window : n;
  return {lo, ((int)min((int64_t)n, hi) - lo + kQueries - 1) / kQueries};
}

// The keys that rows [row0, row0 + kSeqRows) walk over.
template <int D>
__device__ __forceinline__ Walk keys_of(const SeqAttnArgs& a, int n, int row0) {
  constexpr int kKeys = kQueriesOf<D>;
  const int hi = a.causal ? min(n, row0 + kSeqRows) : n;
  const int lo = a.window ? max(0, row0 - a.window + 1) & ~(kKeys - 1) : 0;
  return {lo, (hi - lo + kKeys - 1) / kKeys};
}

// What a tile costs beside its walk, in tiles of the walk: loads that wait for one
// another, the last stores, masked tiles.
template <int D>
constexpr int kEntry = D == 64 ? 4 : 3;

// The lines of a head: where each tile's walk over the queries starts on that of
// all key tiles, and its walk over the keys on that of all row tiles.  Written by
// one workgroup, a sequence a lane, sequences in order.
template <int D>
__device__ void write_line(const SeqAttnArgs& a) {
  __shared__ int64_t part[4][3];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t tiles0 = 0, its0 = 0, keys0 = 0;
  for (int i0 = 0; i0 < a.batch; i0 += 256) {
    const int i = i0 + threadIdx.x;
    int first = 0, n = 0;
    if (i < a.batch) {
      first = max(0, min(a.cu[i], a.tokens));
      n = min(max(first, min(a.cu[i + 1], a.tokens)) - first, a.max_len);
    }
    int64_t its = 0, keys = 0;
    for (int k0 = 0; k0 < n; k0 += kSeqRows) {
      its += (int64_t)walk_of<D>(a, n, k0).tiles * a.group + kEntry<D>;
      keys += keys_of<D>(a, n, k0).tiles + kEntry<D>;
    }
    const int64_t mine[3] = {(n + kSeqRows - 1) / kSeqRows, its, keys};
    int64_t upto[3] = {mine[0], mine[1], mine[2]};
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const int64_t o = __shfl_up(upto[c], off, 64);
        if (lane >= off) upto[c] += o;
      }
    __syncthreads();  // the chunk before is done with `part`
    if (lane == 63)
#pragma unroll
      for (int c = 0; c < 3; ++c) part[wave][c] = upto[c];
    __syncthreads();
    int64_t at = tiles0 + upto[0] - mine[0], start = its0 + upto[1] - its, start_q = keys0 + upto[2] - keys;
    for (int v = 0; v < 4; ++v) {
      if (v < wave) at += part[v][0], start += part[v][1], start_q += part[v][2];
      tiles0 += part[v][0];
      its0 += part[v][1];
      keys0 += part[v][2];
    }
    for (int k0 = 0; k0 < n; k0 += kSeqRows, ++at) {
      if (at >= a.most_tiles) break;  // (overlapping sequences: past what there is room for)
      a.line[at] = {start, start_q, first, n, k0, 0};
      start += (int64_t)walk_of<D>(a, n, k0).tiles * a.group + kEntry<D>;
      start_q += keys_of<D>(a, n, k0).tiles + kEntry<D>;
    }
  }
  if (threadIdx.x == 0) *a.line_end = {its0, keys0, 0, 0, 0, (int)min(tiles0, (int64_t)a.most_tiles)};
}

// Share j of a line: from here to share j + 1's start.
__device__ __forceinline__ int64_t share_start(int64_t total, int shares, int64_t j) { return quotient(total * j, shares); }

// A value that is the same in every lane, as a scalar.
__device__ __forceinline__ int64_t scalar(int64_t v) {
  return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// A workgroup's part of a line: [pos, end), from tile `at` on.
struct Share {
  int64_t pos, end;
  int at, tiles;
};
template <bool ROWS>
__device__ __forceinline__ Share share_of(const SeqAttnArgs& a, int shares, int j) {
  Share r;
  // (read before the number of tiles is known: the line has room for all)
  const SeqLine mine = a.line[min((int)threadIdx.x, a.most_tiles - 1)];
  const int64_t total = scalar(ROWS ? a.line_end->start_q : a.line_end->start);
  r.pos = share_start(total, shares, j);
  r.end = share_start(total, shares, j + 1);
  r.tiles = __builtin_amdgcn_readfirstlane(a.line_end->count);
  // the tile that the share begins in: the last that starts at or before it
  int at = __syncthreads_count((int)threadIdx.x < r.tiles && (ROWS ? mine.start_q : mine.start) <= r.pos) - 1;
  for (int i0 = 256; i0 < r.tiles; i0 += 256) {
    const int i = i0 + (int)threadIdx.x;
    const SeqLine& l = a.line[min(i, r.tiles - 1)];
    at += __syncthreads_count(i < r.tiles && (ROWS ? l.start_q : l.start) <= r.pos);
  }
  r.at = __builtin_amdgcn_readfirstlane(at);
  return r;
}
// What it takes of a tile's walk: [begin, stop) of `length`.
struct Piece {
  int64_t begin, stop, length;
  __device__ __forceinline__ bool whole() const { return stop - begin == length; }
};
template <int D>
__device__ __forceinline__ Piece piece_of(Share& s, int64_t start, int64_t length) {
  start = scalar(start) + kEntry<D>;
  const Piece p = {max((int64_t)0, s.pos - start), min(length, s.end - start), length};
  s.pos = start + length;
  return p;
}
// Where its partial sums go: a share cuts at most two walks, the one it begins
// inside of (slot 0) and the one it ends in (slot 1).
template <int D>
__device__ __forceinline__ int64_t slot_of(uint32_t group, const Piece& p, int row) {
  return ((2 * (int64_t)group + (p.begin == 0)) * kSeqRows + row) * D;
}

// The tile of a workgroup that takes a whole one, the last first or the first; of
// ragged batches (ragged_places) from the line.
template <bool LAST_FIRST>
__device__ __forceinline__ SeqLine whole_tile(const SeqAttnArgs& a, int place) {
  SeqLine tile = {};
  if (a.rest > 0) {
    const int at = LAST_FIRST ? a.most_tiles - 1 - place : place;
    if (at < a.line_end->count) tile = a.line[at];
  } else {
    const Seq s = seq_of(a, place % a.batch);
    const int nth = place / a.batch;
    tile.first = s.first, tile.n = s.n, tile.k0 = (LAST_FIRST ? a.tiles - 1 - nth : nth) * kSeqRows;
  }
  return tile;
}

// What a row's gradients are formed from: -lse log2(e), or NaN where the forward's
// results are not finite, which makes everything that the row sees NaN, and
// -delta.  D / 8 lanes a row; one more workgroup writes the line of key tiles.
template <int D>
__global__ __launch_bounds__(256) void seq_attn_stats_kernel(SeqAttnArgs a) {
  constexpr int kLanes = D / 8;
  uint32_t x = a.first + blockIdx.x;
  if ((a.shares > 0 || a.rest > 0) && x-- == 0) return write_line<D>(a);
  const uint32_t i = x * (256 / kLanes) + threadIdx.x / kLanes;  // of tokens * q_heads, fewer than 2^31
  const int64_t token = i / (uint32_t)a.q_heads;
  if (token >= a.tokens) return;
  const int head = (int)(i - token * a.q_heads), d = 8 * (threadIdx.x % kLanes);
  const v8b g = *reinterpret_cast<const v8b*>(a.dout + token * a.dout_stride + head * D + d);
  const v8b o = *reinterpret_cast<const v8b*>(a.out + (int64_t)i * D + d);
  float delta = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) delta = fmaf((float)g[e], (float)o[e], delta);
#pragma unroll
  for (int off = 1; off < kLanes; off <<= 1) delta += __shfl_xor(delta, off, 64);
  if (d != 0) return;
  const float lse = a.lse[i];
  const bool fine = lse - lse == 0.0f && delta - delta == 0.0f;
  const int64_t to = head * (int64_t)a.tokens + token;
  a.lse2[to] = fine ? lse * -1.44269504088896340736f : NAN;
  a.delta[to] = -delta;
}

// Sub-tiles of 32 rows (keys) whose products run side by side: two where the
// registers hold them.
template <int D>
constexpr int kSubs = D == 64 ? 2 : 1;

// LDS of a workgroup.
template <int D>
struct GradShared {
  static constexpr int kRows = kQueriesOf<D>;  // of a tile, for either kind
  __attribute__((aligned(1024))) uint8_t ring[2][2][kRows * D * 2];  // [buffer][keys, values or queries, dout]
  __attribute__((aligned(16))) float stats[2][2][64];                // [buffer][-lse2, -delta]
  int bad_key[kRows];
  int found[4];
};

// CUT: the workgroup has a share of the line, otherwise one tile.
template <int D, bool CUT>
__device__ __forceinline__ void dq_group(const SeqAttnArgs& a, GradShared<D>& lds, uint32_t x) {
  constexpr int J = D / 16, DT = D / 32, kKeys = GradShared<D>::kRows, SUB = kSubs<D>, kStep = 32 * SUB;
  using Load = TileLoad<D, kKeys>;
  int* const found = lds.found;
  int* const bad_key = lds.bad_key;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  const int nth = x % a.q_heads, place = x / a.q_heads;
  const int kv_head = nth % a.heads, head = kv_head * a.group + nth / a.heads;
  Share share = {0, 1, 0, 1};
  if constexpr (CUT) share = share_of<true>(a, a.row_shares, place);

  const uint32_t ring0 = lds_addr(lds.ring);
  const int64_t ks = a.k_stride * 2, vs = a.v_stride * 2;
  const Load load_k(lane, wave, (uint32_t)ks), load_v(lane, wave, (uint32_t)vs);
  const uint32_t by_row = row_place<D>(lane), by_column = column_place<D>(lane);

  for (; share.pos < share.end && share.at < share.tiles; ++share.at) {
    SeqLine tile = {};
    if constexpr (CUT) {
      tile = a.line[share.at];
    } else {
      tile = whole_tile<true>(a, place);  // late rows see most
    }
    const Seq s = {__builtin_amdgcn_readfirstlane(tile.first), __builtin_amdgcn_readfirstlane(tile.n)};
    const int row0 = __builtin_amdgcn_readfirstlane(tile.k0);
    if (row0 >= s.n) return;  // (not one of a line)
    const Walk walk = keys_of<D>(a, s.n, row0);
    Piece piece = {0, walk.tiles, walk.tiles};
    if constexpr (CUT) piece = piece_of<D>(share, tile.start_q, walk.tiles);
    if (piece.stop <= piece.begin) return;  // the share ends at the entry
    const int klo = walk.lo + (int)piece.begin * kKeys;
    const int khi = min(a.causal ? min(s.n, row0 + kSeqRows) : s.n, walk.lo + (int)piece.stop * kKeys);

    const uint16_t* kp = a.k + (int64_t)(s.first + klo) * a.k_stride + kv_head * D;
    const uint16_t* vp = a.v + (int64_t)(s.first + klo) * a.v_stride + kv_head * D;
    auto issue = [&](int T, int buf) {
      load_k.issue(kp + (int64_t)(T - klo) * a.k_stride, ks, s.n - T, ring0 + buf * 2 * Load::kBytes, wave);
      load_v.issue(vp + (int64_t)(T - klo) * a.v_stride, vs, s.n - T, ring0 + (2 * buf + 1) * Load::kBytes, wave);
    };
    issue(klo, 0);

    const int wrow = row0 + 32 * wave, row = wrow + r32;
    v8b q[J], g[J];
#pragma unroll
    for (int j = 0; j < J; ++j) q[j] = g[j] = v8b{};
    if (row < s.n) {
      const uint16_t* qp = a.q + (int64_t)(s.first + row) * a.q_stride + head * D + 8 * h;
      const uint16_t* gp = a.dout + (int64_t)(s.first + row) * a.dout_stride + head * D + 8 * h;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        q[j] = *reinterpret_cast<const v8b*>(qp + 16 * j);
        g[j] = *reinterpret_cast<const v8b*>(gp + 16 * j);
      }
    }
    const int64_t stat = (int64_t)head * a.tokens + s.first + min(row, s.n - 1);
    const float minus_lse2 = a.lse2[stat], minus_delta = a.delta[stat];

    const int hi = a.causal ? min(row + 1, s.n) : s.n, lo = a.window ? row - a.window + 1 : 0;
    const int whi = wrow >= s.n ? 0 : (a.causal ? min(wrow + 32, s.n) : s.n);
    const int wlo = a.window ? wrow - a.window + 1 : 0;
    const int all_hi = a.causal ? min(s.n, row0 + 1) : s.n;
    const int all_lo = a.window ? min(row0 + kSeqRows, s.n) - a.window : 0;

    v16f dq[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) dq[d] = zero16();

    // kStep keys from position K on, in LDS at `keys` and `values`
    auto consume = [&](bool masked, bool any_bad, int K, uint32_t keys, uint32_t values, int slot) {
      v16f t[SUB], dp[SUB];
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub) {
        t[sub] = zero16();
#pragma unroll
        for (int e = 0; e < 16; ++e) dp[sub][e] = minus_delta;
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) {
          t[sub] = mma(lds_row(((keys + by_row) ^ (32 * j)) + sub * 64 * D), q[j], t[sub]);
          dp[sub] = mma(lds_row(((values + by_row) ^ (32 * j)) + sub * 64 * D), g[j], dp[sub]);
        }
        if (D > 64 && j % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
      if (any_bad) {
        asm volatile("");
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
          for (int e = 0; e < 16; ++e) t[sub][e] = bad_key[slot + 32 * sub + result_row(e, h)] ? NAN : t[sub][e];
      }
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
        for (int e = 0; e < 16; ++e) dp[sub][e] *= __builtin_amdgcn_exp2f(fmaf(t[sub][e], a.scale_log2, minus_lse2));
      if (masked) {
        asm volatile("");
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int key = K + 32 * sub + result_row(e, h);
            dp[sub][e] = key >= lo && key < hi ? dp[sub][e] : 0.0f;
          }
      }
      v8b ds[2 * SUB];
#pragma unroll
      for (int c = 0; c < 2 * SUB; ++c) ds[c] = operand(dp[c >> 1], c & 1);
      if (D > 64) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 0; c < 2 * SUB; ++c)
#pragma unroll
        for (int d = 0; d < DT; ++d) dq[d] = mma(column_step<D>(keys + by_column + c * 32 * D, d), ds[c], dq[d]);
    };

    int buf = 0;
    for (int T = klo; T < khi; T += kKeys, buf ^= 1) {
      wait_vmcnt<0>();
      bare_barrier();
      if (T + kKeys < khi) issue(T + kKeys, buf ^ 1);
      const uint32_t keys = ring0 + buf * 2 * Load::kBytes, values = keys + Load::kBytes;
      bool any_bad = false;
      if (T + kKeys > all_hi || T < all_lo) {
        any_bad = has_bad<Load::kBytes>(keys, found);
        if (any_bad) {
          if (threadIdx.x < kKeys) bad_key[threadIdx.x] = 0;
          clear_bad<Load::kBytes>(keys, 2 * D, bad_key);
        }
      }
#pragma unroll
      for (int slot = 0; slot < kKeys; slot += kStep) {
        const int K = T + slot;
        if (K >= whi || K + kStep <= wlo) continue;
        const bool whole = K + kStep <= min(s.n, a.causal ? wrow + 1 : s.n) && (!a.window || K > wrow + 31 - a.window);
        consume(!whole, any_bad, K, keys + slot * 2 * D, values + slot * 2 * D, slot);
      }
    }

    if constexpr (CUT) bare_barrier();  // every wave is done with the ring
    if (row >= s.n) {
      if constexpr (CUT) continue;
      else return;
    }
    if (!CUT || piece.whole()) {
      uint16_t* to = a.dq + (int64_t)(s.first + row) * a.dq_stride + head * D;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint2*>(to + 32 * d + 8 * u + 4 * h) =
              make_uint2(pack_bf16(dq[d][4 * u] * a.scale, dq[d][4 * u + 1] * a.scale),
                         pack_bf16(dq[d][4 * u + 2] * a.scale, dq[d][4 * u + 3] * a.scale));
    } else {
      float* part = a.part_q + slot_of<D>(x, piece, 32 * wave + r32) + 4 * h;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<v4f*>(part + 32 * d + 8 * u) =
              v4f{dq[d][4 * u], dq[d][4 * u + 1], dq[d][4 * u + 2], dq[d][4 * u + 3]};
    }
    if constexpr (!CUT) return;
  }
}

// Which of the two sums a workgroup forms.  With heads of 256 one: the two sums
// alone would fill the registers (spilled, 2000 tokens of 16 heads on 4 took 1100
// us; two kinds of workgroups, which form p twice, 420).
constexpr int kDk = 1, kDv = 2;

// x: the workgroup among those of its kind.
template <int D, int SUMS, bool CUT>
__device__ __forceinline__ void dkv_group(const SeqAttnArgs& a, GradShared<D>& lds, uint32_t x) {
  constexpr int J = D / 16, DT = D / 32, kQueries = kQueriesOf<D>, SUB = kSubs<D>, kStep = 32 * SUB;
  constexpr bool kWantK = (SUMS & kDk) != 0, kWantV = (SUMS & kDv) != 0;
  using Load = TileLoad<D, kQueries>;
  int* const found = lds.found;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  const int kv_head = x % a.heads, place = x / a.heads;
  Share share = {0, 1, 0, 1};
  if constexpr (CUT) share = share_of<false>(a, a.shares, place);

  const uint32_t ring0 = lds_addr(lds.ring), stats0 = lds_addr(lds.stats);
  const int64_t qs = a.q_stride * 2, gs = a.dout_stride * 2;
  const Load load_q(lane, wave, (uint32_t)qs), load_g(lane, wave, (uint32_t)gs);
  const uint32_t by_row = row_place<D>(lane), by_column = column_place<D>(lane);

  for (; share.pos < share.end && share.at < share.tiles; ++share.at) {
    SeqLine tile = {};
    if constexpr (CUT) {
      tile = a.line[share.at];
    } else {
      tile = whole_tile<false>(a, place);  // early keys are seen most
    }
    const Seq s = {__builtin_amdgcn_readfirstlane(tile.first), __builtin_amdgcn_readfirstlane(tile.n)};
    const int k0 = __builtin_amdgcn_readfirstlane(tile.k0);
    if (k0 >= s.n) return;  // (not one of a line)
    const Walk walk = walk_of<D>(a, s.n, k0);
    Piece piece = {0, (int64_t)walk.tiles * a.group, (int64_t)walk.tiles * a.group};
    if constexpr (CUT) piece = piece_of<D>(share, tile.start, piece.length);
    if (piece.stop <= piece.begin) return;  // the share ends at the entry
    const int64_t its = piece.stop - piece.begin;

    const int wkey = k0 + 32 * wave, key = wkey + r32;
    v8b k[J], v[J];
#pragma unroll
    for (int j = 0; j < J; ++j) k[j] = v[j] = v8b{};
    if (key < s.n) {
      const uint16_t* kp = a.k + (int64_t)(s.first + key) * a.k_stride + kv_head * D + 8 * h;
      const uint16_t* vp = a.v + (int64_t)(s.first + key) * a.v_stride + kv_head * D + 8 * h;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        k[j] = *reinterpret_cast<const v8b*>(kp + 16 * j);
        if constexpr (kWantK) v[j] = *reinterpret_cast<const v8b*>(vp + 16 * j);
      }
    }
    // the queries that see the lane's key
    const int lo = a.causal ? key : 0;
    const int hi = a.window ? (int)min((int64_t)s.n, (int64_t)key + a.window) : s.n;

    v16f dk[DT], dv[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) dk[d] = dv[d] = zero16();

    auto issue = [&](int group, int t, int buf) {
      const int head = kv_head * a.group + group, T = walk.lo + t * kQueries, left = s.n - T;
      const int64_t token = s.first + T;
      load_q.issue(a.q + token * a.q_stride + head * D, qs, left, ring0 + buf * 2 * Load::kBytes, wave);
      load_g.issue(a.dout + token * a.dout_stride + head * D, gs, left, ring0 + (2 * buf + 1) * Load::kBytes, wave);
      // every wave brings all of the rows' statistics: the same words to the same place
      const int64_t row = (int64_t)head * a.tokens + token + min(lane, left - 1);
      dma4(a.lse2 + row, stats0 + buf * 512);
      if constexpr (kWantK) dma4(a.delta + row, stats0 + buf * 512 + 256);
    };

    // kStep query rows from Q on, in LDS at `queries` and `grads`
    auto consume = [&](bool masked, int Q, uint32_t queries, uint32_t grads, const float* stat) {
      v16f t[SUB], dp[SUB];
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub) {
        t[sub] = zero16();
        if constexpr (kWantK) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const v4f w = *reinterpret_cast<const v4f*>(stat + 64 + 32 * sub + 8 * u + 4 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e) dp[sub][4 * u + e] = w[e];
          }
        }
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) {
          t[sub] = mma(lds_row(((queries + by_row) ^ (32 * j)) + sub * 64 * D), k[j], t[sub]);
          if constexpr (kWantK) dp[sub] = mma(lds_row(((grads + by_row) ^ (32 * j)) + sub * 64 * D), v[j], dp[sub]);
        }
        if (D > 64 && j % 2 == 1) __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const v4f w = *reinterpret_cast<const v4f*>(stat + 32 * sub + 8 * u + 4 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            t[sub][4 * u + e] = __builtin_amdgcn_exp2f(fmaf(t[sub][4 * u + e], a.scale_log2, w[e]));
        }
      if (masked) {
        asm volatile("");
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int row = Q + 32 * sub + result_row(e, h);
            const bool seen = row >= lo && row < hi;
            t[sub][e] = seen ? t[sub][e] : 0.0f;
            if constexpr (kWantK) dp[sub][e] = seen ? dp[sub][e] : 0.0f;
          }
      }
      v8b p[2 * SUB], ds[2 * SUB];
#pragma unroll
      for (int c = 0; c < 2 * SUB; ++c) {
        if constexpr (kWantV) p[c] = operand(t[c >> 1], c & 1);
      }
      if constexpr (kWantK) {
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) dp[sub] *= t[sub];
#pragma unroll
        for (int c = 0; c < 2 * SUB; ++c) ds[c] = operand(dp[c >> 1], c & 1);
      }
      if (D > 64) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 0; c < 2 * SUB; ++c)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          if constexpr (kWantV) dv[d] = mma(column_step<D>(grads + by_column + c * 32 * D, d), p[c], dv[d]);
          if constexpr (kWantK) dk[d] = mma(column_step<D>(queries + by_column + c * 32 * D, d), ds[c], dk[d]);
          if (D > 64 && d % 2 == 1) __builtin_amdgcn_sched_barrier(0);
        }
    };

    int group = (int)quotient(piece.begin, walk.tiles), t = (int)(piece.begin - (int64_t)group * walk.tiles), buf = 0;
    issue(group, t, 0);
    for (int64_t it = 0; it < its; ++it, buf ^= 1) {
      const int T = walk.lo + t * kQueries;
      wait_vmcnt<0>();
      bare_barrier();
      if (++t == walk.tiles) t = 0, ++group;
      if (it + 1 < its) issue(group, t, buf ^ 1);
      const uint32_t queries = ring0 + buf * 2 * Load::kBytes, grads = queries + Load::kBytes;
      // rows that some key of the workgroup is not seen by
      if ((a.causal && T < min(k0 + kSeqRows, s.n) - 1) || T + kQueries > s.n ||
          (a.window && T + kQueries > (int64_t)k0 + a.window)) {
        if (has_bad<2 * Load::kBytes>(queries, found)) clear_bad<2 * Load::kBytes>(queries, 2 * D, nullptr);
      }
#pragma unroll
      for (int slot = 0; slot < kQueries; slot += kStep) {
        const int Q = T + slot;
        if (wkey >= s.n || Q >= s.n || (a.causal && Q + kStep - 1 < wkey)) continue;
        if (a.window && Q >= (int64_t)wkey + 31 + a.window) continue;
        const bool whole = Q + kStep <= s.n && (!a.causal || Q >= wkey + 31) &&
                           (!a.window || Q + kStep - 1 < (int64_t)wkey + a.window);
        consume(!whole, Q, queries + slot * 2 * D, grads + slot * 2 * D, &lds.stats[buf][0][slot]);
      }
    }
    if constexpr (CUT) bare_barrier();  // every wave is done with the ring

    if (key >= s.n) {
      if constexpr (CUT) continue;
      else return;
    }
    if (!CUT || piece.whole()) {
      const int64_t token = s.first + key;
      uint16_t* to_k = a.dk + token * a.dk_stride + kv_head * D + 4 * h;
      uint16_t* to_v = a.dv + token * a.dv_stride + kv_head * D + 4 * h;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = 4 * u;
          if constexpr (kWantK)
            *reinterpret_cast<uint2*>(to_k + 32 * d + 8 * u) =
                make_uint2(pack_bf16(dk[d][e] * a.scale, dk[d][e + 1] * a.scale),
                           pack_bf16(dk[d][e + 2] * a.scale, dk[d][e + 3] * a.scale));
          if constexpr (kWantV)
            *reinterpret_cast<uint2*>(to_v + 32 * d + 8 * u) =
                make_uint2(pack_bf16(dv[d][e], dv[d][e + 1]), pack_bf16(dv[d][e + 2], dv[d][e + 3]));
        }
    } else {
      const int64_t to = slot_of<D>(x, piece, 32 * wave + r32) + 4 * h;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = 4 * u;
          if constexpr (kWantK)
            *reinterpret_cast<v4f*>(a.part_k + to + 32 * d + 8 * u) = v4f{dk[d][e], dk[d][e + 1], dk[d][e + 2], dk[d][e + 3]};
          if constexpr (kWantV)
            *reinterpret_cast<v4f*>(a.part_v + to + 32 * d + 8 * u) = v4f{dv[d][e], dv[d][e + 1], dv[d][e + 2], dv[d][e + 3]};
        }
    }
    if constexpr (!CUT) return;
  }
}

// The kind whose workgroups take longest comes first.
template <int D, bool CUT_KEYS, bool CUT_ROWS>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void seq_attn_grad_kernel(SeqAttnArgs a) {
  __shared__ GradShared<D> lds;
  uint32_t x = a.first + blockIdx.x;
  if (x >= a.dq_first) {
    const uint32_t y = x - a.dq_first;
    if constexpr (D == 256) {
      if (y < a.dkv_groups) return dkv_group<D, kDk, CUT_KEYS>(a, lds, y);
      if (y < 2 * a.dkv_groups) return dkv_group<D, kDv, CUT_KEYS>(a, lds, y - a.dkv_groups);
      x -= 2 * a.dkv_groups;
    } else {
      if (y < a.dkv_groups) return dkv_group<D, kDk | kDv, CUT_KEYS>(a, lds, y);
      x -= a.dkv_groups;
    }
  }
  dq_group<D, CUT_ROWS>(a, lds, x);
}

// Adds the sums of the tiles whose walks were cut, share by share: a lane four
// dimensions of a row.  Of dk and dv, or (ROWS) of dq.
template <int D, bool ROWS>
__device__ __forceinline__ void join_group(const SeqAttnArgs& a, uint32_t x) {
  constexpr int kRows = 1024 / D, kParts = kSeqRows / kRows;
  const int heads = ROWS ? a.q_heads : a.heads, shares = ROWS ? a.row_shares : a.shares;
  const int nth = x % heads, head = ROWS ? (nth % a.heads) * a.group + nth / a.heads : nth;
  x /= heads;
  const int at = x / kParts, row = (int)(x % kParts) * kRows + threadIdx.x / (D / 4), d = 4 * (threadIdx.x % (D / 4));
  const SeqLine end = *a.line_end, tile = a.line[at];  // (one of `most_tiles`)
  if (at >= end.count) return;
  const Seq s = {tile.first, tile.n};
  const int64_t total = ROWS ? end.start_q : end.start, start = ROWS ? tile.start_q : tile.start;
  const int64_t length = ROWS ? keys_of<D>(a, s.n, tile.k0).tiles : (int64_t)walk_of<D>(a, s.n, tile.k0).tiles * a.group;
  // the shares that hold the walk's first and last tile
  const int64_t walk = start + kEntry<D>;
  const int64_t j0 = quotient((walk + 1) * shares - 1, total), j1 = quotient((walk + length) * shares - 1, total);
  if (j0 == j1 || row >= s.n - tile.k0) return;
  // slots: the first share's second one, the others' first
  const int64_t step = (int64_t)heads * 2 * kSeqRows * D;
  const int64_t from = ((2 * (j0 * heads + nth)) * kSeqRows + row) * D + d;
  const float* const part = ROWS ? a.part_q : a.part_k;
  v4f sum = *reinterpret_cast<const v4f*>(part + from + kSeqRows * D), v = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (!ROWS) v = *reinterpret_cast<const v4f*>(a.part_v + from + kSeqRows * D);
  const bool some_empty = total < shares;
  for (int64_t j = j0 + 1; j <= j1; j += 4) {
    v4f pk[4], pv[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool there = j + c <= j1 && !(some_empty && share_start(total, shares, j + c) ==
                                                            share_start(total, shares, j + c + 1));
      pk[c] = pv[c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      if (there) {
        pk[c] = *reinterpret_cast<const v4f*>(part + from + (j + c - j0) * step);
        if constexpr (!ROWS) pv[c] = *reinterpret_cast<const v4f*>(a.part_v + from + (j + c - j0) * step);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      sum += pk[c];
      v += pv[c];
    }
  }
  const int64_t token = s.first + tile.k0 + row;
  sum *= a.scale;
  uint16_t* to = ROWS ? a.dq + token * a.dq_stride : a.dk + token * a.dk_stride;
  *reinterpret_cast<uint2*>(to + head * D + d) = make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
  if constexpr (!ROWS)
    *reinterpret_cast<uint2*>(a.dv + token * a.dv_stride + head * D + d) =
        make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
template <int D>
__global__ __launch_bounds__(256) void seq_attn_join_kernel(SeqAttnArgs a) {
  const uint32_t x = a.first + blockIdx.x, dkv = (uint32_t)a.most_tiles * a.heads * (kSeqRows * D / 1024);
  if (x < dkv) join_group<D, false>(a, x);
  else join_group<D, true>(a, x - dkv);
}

// Fewest tiles of a share's walks (were every query to see every key): a share
// costs some 5 us beside its tiles, of 1 to 2 us each.
constexpr int64_t kLeastShare = 4;

// From the shape alone, so that the workspace does not depend on the mask.
struct BwdPlan {
  int64_t most_tiles;
  int shares, row_shares;  // of a key head's line (dk, dv) and a head's (dq); 0: whole tiles
  int64_t share_tiles;     // tiles of a share of dk and dv, about
  int64_t stat, part, part_q, line, bytes;  // bytes of each
};
BwdPlan plan_of(const SeqAttnShape& s) {
  BwdPlan p{};
  const int64_t tiles = (s.max_len + kSeqRows - 1) / kSeqRows;
  p.most_tiles = std::min((int64_t)s.tokens / kSeqRows + s.batch, tiles * s.batch);
  // Workgroups that run at once on 256 CUs.  Twice as many tiles: one each, whose
  // neighbours walk the same rows at the same time (four sequences of 4096, 32
  // heads: tiles 2086 us, shares 2356).
  const int64_t resident = s.head_dim == 256 ? 256 : 512, queries = s.head_dim == 256 ? 32 : 64;
  const int64_t length = (s.max_len + queries - 1) / queries, work = p.most_tiles * length;
  const bool cut_rows = p.most_tiles * s.q_heads < 2 * resident;
  if (p.most_tiles * s.heads < 2 * resident) {
    // Where dq is cut too, all run at once: four products here and three there
    // (heads of 256: two and three, here twice).
    const int64_t slots = !cut_rows ? resident : s.head_dim == 256 ? resident * 5 / 16 : resident * 4 / 7;
    const int64_t walks = work * (s.q_heads / s.heads);
    p.shares = (int)std::max<int64_t>(1, std::min(slots / s.heads, walks / kLeastShare));
    p.share_tiles = walks / p.shares;
    if (cut_rows) {
      const int64_t rows = s.head_dim == 256 ? resident * 6 / 16 : resident * 3 / 7;
      p.row_shares = (int)std::max<int64_t>(1, std::min(rows / s.q_heads, work / kLeastShare));
    }
  }
  auto aligned = [](int64_t bytes) { return (bytes + 255) & ~(int64_t)255; };
  p.stat = aligned((int64_t)s.tokens * s.q_heads * 4);
  p.part = (int64_t)p.shares * s.heads * 2 * kSeqRows * s.head_dim * 4;
  p.part_q = (int64_t)p.row_shares * s.q_heads * 2 * kSeqRows * s.head_dim * 4;
  p.line = aligned((p.most_tiles + 1) * (int64_t)sizeof(SeqLine));
  p.bytes = 2 * p.stat + 2 * p.part + p.part_q + p.line;
  return p;
}

template <int D>
void run_bwd(SeqAttnArgs& a, int64_t share_tiles, hipStream_t stream) {
  auto launch = [&](auto kernel, int64_t groups) {
    in_stretches(groups, 256, [&](uint32_t first, uint32_t count) {
      a.first = first;
      hipLaunchKernelGGL(kernel, dim3(count), dim3(256), 0, stream, a);
    });
  };
  launch(seq_attn_stats_kernel<D>, ((int64_t)a.tokens * a.q_heads * (D / 8) + 255) / 256 + (a.shares > 0 || a.rest > 0));
  const int64_t tiles = a.rest > 0 ? a.most_tiles : (int64_t)a.tiles * a.batch;
  const int64_t dkv = a.shares > 0 ? (int64_t)a.heads * a.shares : tiles * a.heads;
  const int64_t dq = (a.row_shares > 0 ? a.row_shares : tiles) * a.q_heads;
  a.dkv_groups = (uint32_t)dkv;
  a.dq_first = a.shares > 0 && share_tiles < (a.max_len + kQueriesOf<D> - 1) / kQueriesOf<D> ? (uint32_t)dq : 0;
  const int64_t groups = (D == 256 ? 2 : 1) * dkv + dq;
  // (kernels of their own: the loop over a share's tiles costs whole tiles 3%)
  if (a.row_shares > 0) launch(seq_attn_grad_kernel<D, true, true>, groups);
  else if (a.shares > 0) launch(seq_attn_grad_kernel<D, true, false>, groups);
  else launch(seq_attn_grad_kernel<D, false, false>, groups);
  const int64_t joins = (int64_t)a.most_tiles * (kSeqRows * D / 1024);
  if (a.shares > 1 || a.row_shares > 1)
    launch(seq_attn_join_kernel<D>, joins * a.heads + (a.row_shares > 1 ? joins * a.q_heads : 0));
}

}  // namespace

int64_t seq_attn_bwd_workspace_bytes(const SeqAttnShape& s) { return plan_of(s).bytes; }

hipError_t launch_seq_attn_bwd(SeqAttnArgs a, int head_dim, void* ws, hipStream_t stream) {
  const BwdPlan p = plan_of({a.batch, a.tokens, a.max_len, a.q_heads, a.heads, head_dim});
  a.shares = p.shares;
  a.row_shares = p.row_shares;
  a.most_tiles = (int)p.most_tiles;
  a.tiles = (a.max_len + kSeqRows - 1) / kSeqRows;
  a.rest = ragged_places(a.tokens, a.batch, a.tiles);
  uint8_t* at = static_cast<uint8_t*>(ws);
  auto take = [&](int64_t bytes) {
    uint8_t* r = at;
    at += bytes;
    return r;
  };
  a.line = reinterpret_cast<SeqLine*>(take(p.line));
  a.line_end = a.line + p.most_tiles;
  a.lse2 = reinterpret_cast<float*>(take(p.stat));
  a.delta = reinterpret_cast<float*>(take(p.stat));
  a.part_k = reinterpret_cast<float*>(take(p.part));
  a.part_v = reinterpret_cast<float*>(take(p.part));
  a.part_q = reinterpret_cast<float*>(take(p.part_q));
  if (head_dim == 64) run_bwd<64>(a, p.share_tiles, stream);
  else if (head_dim == 128) run_bwd<128>(a, p.share_tiles, stream);
  else run_bwd<256>(a, p.share_tiles, stream);
  return hipGetLastError();
}

}  // namespace fp8lin
