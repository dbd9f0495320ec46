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
// the queries and dout of all its heads through LDS.  A workgroup takes a key
// tile where there are enough of them.  Otherwise -- few key heads, short
// batches -- the tiles' walks over the queries, of very different lengths under a
// causal mask, are laid one behind the other for each key head and cut into
// equal shares, one for each workgroup that runs at the same time, and the rows'
// walks over the keys into chunks; a cut walk's partial sums are joined in order
// by a last kernel.
//
// Both kinds run in one launch, behind a small one that leaves -lse log2(e) and
// -delta of every row and head.
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

// The line of all key tiles of a head: where each one's walk starts on it, in
// query tiles.  Written by one workgroup, a sequence a lane, sequences in order.
template <int D>
__device__ void write_line(const SeqAttnArgs& a) {
  __shared__ int64_t part[4][2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t tiles0 = 0, its0 = 0;
  for (int i0 = 0; i0 < a.batch; i0 += 256) {
    const int i = i0 + threadIdx.x;
    int n = 0;
    if (i < a.batch) {
      const int first = max(0, min(a.cu[i], a.tokens));
      n = min(max(first, min(a.cu[i + 1], a.tokens)) - first, a.max_len);
    }
    int64_t its = 0;
    for (int k0 = 0; k0 < n; k0 += kSeqRows) its += (int64_t)walk_of<D>(a, n, k0).tiles * a.group;
    int64_t t = (n + kSeqRows - 1) / kSeqRows, w = its;
    const int64_t my_tiles = t;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t ot = __shfl_up(t, off, 64), ow = __shfl_up(w, off, 64);
      if (lane >= off) t += ot, w += ow;
    }
    __syncthreads();  // the chunk before is done with `part`
    if (lane == 63) part[wave][0] = t, part[wave][1] = w;
    __syncthreads();
    int64_t at = tiles0 + t - my_tiles, start = its0 + w - its;
    for (int v = 0; v < 4; ++v) {
      if (v < wave) at += part[v][0], start += part[v][1];
      tiles0 += part[v][0];
      its0 += part[v][1];
    }
    for (int k0 = 0; k0 < n; k0 += kSeqRows, ++at) {
      if (at >= a.most_tiles) break;  // (overlapping sequences: past what there is room for)
      a.line[at] = {start, i, k0};
      start += (int64_t)walk_of<D>(a, n, k0).tiles * a.group;
    }
  }
  if (threadIdx.x == 0) {
    a.line_end->start = its0;
    a.line_end->seq = (int)min(tiles0, (int64_t)a.most_tiles);
  }
}

// Share j of a line of `total` query tiles: from here to share j + 1's.
__device__ __forceinline__ int64_t share_start(int64_t total, int shares, int64_t j) { return total * j / shares; }

// What a row's gradients are formed from: -lse log2(e), or NaN where the forward's
// results are not finite, which makes everything that the row sees NaN, and
// -delta.  D / 8 lanes a row; one more workgroup writes the line of key tiles.
template <int D>
__global__ __launch_bounds__(256) void seq_attn_stats_kernel(SeqAttnArgs a) {
  constexpr int kLanes = D / 8;
  uint32_t x = a.first + blockIdx.x;
  if (a.shares > 0 && x-- == 0) return write_line<D>(a);
  const int64_t i = (int64_t)x * (256 / kLanes) + threadIdx.x / kLanes, token = i / a.q_heads;
  if (token >= a.tokens) return;
  const int head = (int)(i - token * a.q_heads), d = 8 * (threadIdx.x % kLanes);
  const v8b g = *reinterpret_cast<const v8b*>(a.dout + token * a.dout_stride + head * D + d);
  const v8b o = *reinterpret_cast<const v8b*>(a.out + i * D + d);
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

// The keys that rows [row0, row0 + kSeqRows) read, and the chunks of them.
struct KeySpan {
  int lo, hi, chunks;
};
template <int D>
__device__ __forceinline__ KeySpan keys_of(const SeqAttnArgs& a, int n, int row0) {
  constexpr int kKeys = kQueriesOf<D>;
  KeySpan r;
  r.hi = a.causal ? min(n, row0 + kSeqRows) : n;
  r.lo = a.window ? max(0, row0 - a.window + 1) & ~(kKeys - 1) : 0;
  r.chunks = a.dq_chunk > 0 ? ((r.hi - r.lo + kKeys - 1) / kKeys + a.dq_chunk - 1) / a.dq_chunk : 1;
  return r;
}

template <int D>
__device__ __forceinline__ void dq_group(const SeqAttnArgs& a, GradShared<D>& lds, uint32_t x) {
  constexpr int J = D / 16, DT = D / 32, kKeys = GradShared<D>::kRows, SUB = kSubs<D>, kStep = 32 * SUB;
  using Load = TileLoad<D, kKeys>;
  int* const found = lds.found;
  int* const bad_key = lds.bad_key;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  const int kv_head = x % a.heads;
  x /= a.heads;
  const int head = kv_head * a.group + x % a.group;
  x /= a.group;
  const int chunk = x % a.dq_splits;
  x /= a.dq_splits;
  const Seq s = seq_of(a, x % a.batch);
  const int row0 = (a.tiles - 1 - (int)(x / a.batch)) * kSeqRows;  // late rows see most: first
  if (row0 >= s.n) return;
  const KeySpan span = keys_of<D>(a, s.n, row0);
  if (chunk >= span.chunks) return;
  const int klo = span.lo + chunk * a.dq_chunk * kKeys;
  const int khi = span.chunks == 1 ? span.hi : min(span.hi, klo + a.dq_chunk * kKeys);

  const uint32_t ring0 = lds_addr(lds.ring);
  const int64_t ks = a.k_stride * 2, vs = a.v_stride * 2;
  const Load load_k(lane, wave, (uint32_t)ks), load_v(lane, wave, (uint32_t)vs);
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
  const uint32_t by_row = row_place<D>(lane), by_column = column_place<D>(lane);

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

  if (row >= s.n) return;
  if (span.chunks > 1) {
    float* part = a.part_q + (((int64_t)chunk * a.tokens + s.first + row) * a.q_heads + head) * D + 4 * h;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *reinterpret_cast<v4f*>(part + 32 * d + 8 * u) =
            v4f{dq[d][4 * u], dq[d][4 * u + 1], dq[d][4 * u + 2], dq[d][4 * u + 3]};
    return;
  }
  uint16_t* to = a.dq + (int64_t)(s.first + row) * a.dq_stride + head * D;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<uint2*>(to + 32 * d + 8 * u + 4 * h) =
          make_uint2(pack_bf16(dq[d][4 * u] * a.scale, dq[d][4 * u + 1] * a.scale),
                     pack_bf16(dq[d][4 * u + 2] * a.scale, dq[d][4 * u + 3] * a.scale));
}

// A value that is the same in every lane, as a scalar.
__device__ __forceinline__ int64_t scalar(int64_t v) {
  return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// Which of the two sums a workgroup forms.  With heads of 256 one: the two sums
// alone would fill the registers (spilled, 2000 tokens of 16 heads on 4 took 1100
// us; two kinds of workgroups, which form p twice, 420).
constexpr int kDk = 1, kDv = 2;

// x: the workgroup among those of its kind.
template <int D, int SUMS>
__device__ __forceinline__ void dkv_group(const SeqAttnArgs& a, GradShared<D>& lds, uint32_t x) {
  constexpr int J = D / 16, DT = D / 32, kQueries = kQueriesOf<D>, SUB = kSubs<D>, kStep = 32 * SUB;
  constexpr bool kWantK = (SUMS & kDk) != 0, kWantV = (SUMS & kDv) != 0;
  using Load = TileLoad<D, kQueries>;
  int* const found = lds.found;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  const int kv_head = x % a.heads, place = x / a.heads;
  // a share of the head's line, or one key tile
  int64_t pos = 0, end = 1;
  int at = 0, key_tiles = 1;
  if (a.shares > 0) {
    const int64_t total = scalar(a.line_end->start);
    pos = share_start(total, a.shares, place);
    end = share_start(total, a.shares, place + 1);
    if (pos >= end) return;
    key_tiles = __builtin_amdgcn_readfirstlane(a.line_end->seq);
    at = -1;  // the key tile that the share begins in: the last that starts at or before it
    for (int i0 = 0; i0 < key_tiles; i0 += 256) {
      const int i = i0 + (int)threadIdx.x;
      at += __syncthreads_count(i < key_tiles && a.line[min(i, key_tiles - 1)].start <= pos);
    }
    at = __builtin_amdgcn_readfirstlane(at);
  }

  const uint32_t ring0 = lds_addr(lds.ring), stats0 = lds_addr(lds.stats);
  const int64_t qs = a.q_stride * 2, gs = a.dout_stride * 2;
  const Load load_q(lane, wave, (uint32_t)qs), load_g(lane, wave, (uint32_t)gs);
  const uint32_t by_row = row_place<D>(lane), by_column = column_place<D>(lane);

  for (; pos < end && at < key_tiles; ++at) {
    SeqLine tile = {0, place % a.batch, place / a.batch * kSeqRows};  // early keys are seen most: first
    if (a.shares > 0) tile = a.line[at];
    const Seq s = seq_of(a, __builtin_amdgcn_readfirstlane(tile.seq));
    const int k0 = __builtin_amdgcn_readfirstlane(tile.k0);
    if (k0 >= s.n) return;  // (not one of a line)
    const Walk walk = walk_of<D>(a, s.n, k0);
    // (a walk has fewer than 2^31 tiles: at most 2^30 / 32 for each head)
    const int64_t start = scalar(tile.start);
    const int64_t length = (int64_t)walk.tiles * a.group, begin = pos - start;
    const int64_t stop = a.shares > 0 ? min(length, end - start) : length, its = stop - begin;
    pos = start + stop;

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

    int group = (int)(begin / walk.tiles), t = (int)(begin % walk.tiles), buf = 0;
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
    bare_barrier();  // every wave is done with the ring

    if (key >= s.n) continue;
    if (its == length) {
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
      // a share cuts at most two walks: the one it begins inside of (0), the one it ends in (1)
      const int64_t slot = 2 * (int64_t)x + (begin == 0);
      const int64_t to = (slot * kSeqRows + 32 * wave + r32) * D + 4 * h;
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
  }
}

// The kind whose workgroups take longest comes first.
template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void seq_attn_grad_kernel(SeqAttnArgs a) {
  __shared__ GradShared<D> lds;
  uint32_t x = a.first + blockIdx.x;
  if (x >= a.dq_first) {
    const uint32_t y = x - a.dq_first;
    if constexpr (D == 256) {
      if (y < a.dkv_groups) return dkv_group<D, kDk>(a, lds, y);
      if (y < 2 * a.dkv_groups) return dkv_group<D, kDv>(a, lds, y - a.dkv_groups);
      x -= 2 * a.dkv_groups;
    } else {
      if (y < a.dkv_groups) return dkv_group<D, kDk | kDv>(a, lds, y);
      x -= a.dkv_groups;
    }
  }
  dq_group<D>(a, lds, x);
}

// dq of rows whose keys were cut, chunk by chunk; x counts (part of a tile, head).
template <int D>
__device__ __forceinline__ void join_dq(const SeqAttnArgs& a, uint32_t x) {
  constexpr int kRows = 1024 / D, kParts = kSeqRows / kRows;
  const int head = x % a.q_heads;
  x /= a.q_heads;
  const int at = x / kParts, d = 4 * (threadIdx.x % (D / 4));
  if (at >= a.line_end->seq) return;
  const SeqLine tile = a.line[at];
  const Seq s = seq_of(a, tile.seq);
  const int chunks = keys_of<D>(a, s.n, tile.k0).chunks, row = tile.k0 + (x % kParts) * kRows + threadIdx.x / (D / 4);
  if (chunks == 1 || row >= s.n) return;
  const int64_t step = (int64_t)a.tokens * a.q_heads * D, token = s.first + row;
  const float* from = a.part_q + (token * a.q_heads + head) * D + d;
  v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c = 0; c < chunks; c += 4) {
    v4f p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const v4f*>(from + min(c + i, chunks - 1) * step);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < chunks) sum += p[i];
  }
  sum *= a.scale;
  *reinterpret_cast<uint2*>(a.dq + token * a.dq_stride + head * D + d) =
      make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
}

// Adds the sums of the key tiles whose walks were cut, share by share: a lane
// four dimensions of a key.
template <int D>
__global__ __launch_bounds__(256) void seq_attn_join_kernel(SeqAttnArgs a) {
  constexpr int kKeys = 1024 / D, kParts = kSeqRows / kKeys;
  uint32_t x = a.first + blockIdx.x;
  const uint32_t dkv = (uint32_t)a.most_tiles * a.heads * kParts;
  if (x >= dkv) return join_dq<D>(a, x - dkv);
  const int kv_head = x % a.heads;
  x /= a.heads;
  const int at = x / kParts, key = (int)(x % kParts) * kKeys + threadIdx.x / (D / 4), d = 4 * (threadIdx.x % (D / 4));
  if (at >= a.line_end->seq) return;
  const SeqLine tile = a.line[at];
  const Seq s = seq_of(a, tile.seq);
  const int64_t total = a.line_end->start, last = tile.start + (int64_t)walk_of<D>(a, s.n, tile.k0).tiles * a.group - 1;
  // the shares that hold the walk's first and last tile
  const int64_t j0 = ((tile.start + 1) * a.shares - 1) / total, j1 = ((last + 1) * a.shares - 1) / total;
  if (j0 == j1 || key >= s.n - tile.k0) return;
  // slots: the first share's second one, the others' first
  const int64_t step = (int64_t)a.heads * 2 * kSeqRows * D;
  const int64_t from = ((2 * (j0 * a.heads + kv_head)) * kSeqRows + key) * D + d;
  v4f k = *reinterpret_cast<const v4f*>(a.part_k + from + kSeqRows * D);
  v4f v = *reinterpret_cast<const v4f*>(a.part_v + from + kSeqRows * D);
  // (where the line is shorter than its shares are many, some are empty)
  for (int64_t j = j0 + 1; j <= j1; j += 4) {
    v4f pk[4], pv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool there = j + i <= j1 && share_start(total, a.shares, j + i) < share_start(total, a.shares, j + i + 1);
      pk[i] = pv[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      if (there) {
        pk[i] = *reinterpret_cast<const v4f*>(a.part_k + from + (j + i - j0) * step);
        pv[i] = *reinterpret_cast<const v4f*>(a.part_v + from + (j + i - j0) * step);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k += pk[i];
      v += pv[i];
    }
  }
  const int64_t token = s.first + tile.k0 + key;
  k *= a.scale;
  *reinterpret_cast<uint2*>(a.dk + token * a.dk_stride + kv_head * D + d) =
      make_uint2(pack_bf16(k[0], k[1]), pack_bf16(k[2], k[3]));
  *reinterpret_cast<uint2*>(a.dv + token * a.dv_stride + kv_head * D + d) =
      make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// Fewest query tiles of a share (were every query to see every key), and fewest
// key tiles of a chunk of dq.
constexpr int64_t kLeastShare = 8, kLeastChunk = 6;

// From the shape alone, so that the workspace does not depend on the mask.
struct BwdPlan {
  int64_t most_tiles;
  int shares;            // 0: whole key tiles
  int64_t share_tiles;   // query tiles of a share, about
  int chunk, splits;     // key tiles of a chunk of dq, and the most of them; 0, 1: whole
  int64_t stat, part, part_q, line, bytes;  // bytes of each
};
BwdPlan plan_of(const SeqAttnShape& s) {
  BwdPlan p{};
  const int64_t tiles = (s.max_len + kSeqRows - 1) / kSeqRows;
  p.most_tiles = std::min((int64_t)s.tokens / kSeqRows + s.batch, tiles * s.batch);
  // Workgroups that run at once on 256 CUs.  Twice as many key tiles: one each,
  // whose neighbours walk the same queries at the same time (four sequences of
  // 4096, 32 heads: tiles 2086 us, shares 2356).
  const int64_t resident = s.head_dim == 256 ? 256 : 512, queries = s.head_dim == 256 ? 32 : 64;
  const int64_t length = (s.max_len + queries - 1) / queries, work = p.most_tiles * length * (s.q_heads / s.heads);
  p.splits = 1;
  if (p.most_tiles * s.heads < 2 * resident) {
    p.shares = (int)std::max<int64_t>(1, std::min(resident / s.heads, work / kLeastShare));
    p.share_tiles = work / p.shares;
    const int64_t splits = std::min(2 * resident / (p.most_tiles * s.q_heads), length / kLeastChunk);
    if (splits > 1) {
      p.chunk = (int)((length + splits - 1) / splits);
      p.splits = (int)((length + p.chunk - 1) / p.chunk);
    }
  }
  auto aligned = [](int64_t bytes) { return (bytes + 255) & ~(int64_t)255; };
  p.stat = aligned((int64_t)s.tokens * s.q_heads * 4);
  p.part = (int64_t)p.shares * s.heads * 2 * kSeqRows * s.head_dim * 4;
  p.part_q = p.splits > 1 ? (int64_t)p.splits * s.tokens * s.q_heads * s.head_dim * 4 : 0;
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
  launch(seq_attn_stats_kernel<D>, ((int64_t)a.tokens * a.q_heads * (D / 8) + 255) / 256 + (a.shares > 0));
  const int64_t tiles = (int64_t)a.tiles * a.batch;
  const int64_t dkv = a.shares > 0 ? (int64_t)a.heads * a.shares : tiles * a.heads;
  const int64_t dq = tiles * a.q_heads * a.dq_splits;
  const int64_t dq_tiles = a.dq_chunk > 0 ? a.dq_chunk : (a.max_len + kQueriesOf<D> - 1) / kQueriesOf<D>;
  a.dkv_groups = (uint32_t)dkv;
  a.dq_first = a.shares > 0 && share_tiles < dq_tiles ? (uint32_t)dq : 0;
  launch(seq_attn_grad_kernel<D>, (D == 256 ? 2 : 1) * dkv + dq);
  const int64_t joins = (int64_t)a.most_tiles * (kSeqRows * D / 1024);
  if (a.shares > 1 || a.dq_splits > 1)
    launch(seq_attn_join_kernel<D>, joins * a.heads + (a.dq_splits > 1 ? joins * a.q_heads : 0));
}

}  // namespace

int64_t seq_attn_bwd_workspace_bytes(const SeqAttnShape& s) { return plan_of(s).bytes; }

hipError_t launch_seq_attn_bwd(SeqAttnArgs a, int head_dim, void* ws, hipStream_t stream) {
  const BwdPlan p = plan_of({a.batch, a.tokens, a.max_len, a.q_heads, a.heads, head_dim});
  a.shares = p.shares;
  a.dq_chunk = p.chunk;
  a.dq_splits = p.splits;
  a.most_tiles = (int)p.most_tiles;
  a.tiles = (a.max_len + kSeqRows - 1) / kSeqRows;
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
