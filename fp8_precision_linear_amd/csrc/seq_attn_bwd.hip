// Attention over packed sequences, backward: seq_attn.h has the mathematics.
//
// Probabilities are recomputed from q, k and lse, so nothing of the size of the
// logits is stored.  Two kernels, each the owner of what it sums, so that no sum
// depends on an order of atomics: seven products where one kernel that adds dq
// from every key tile would need five.
//
// dq.  As the forward: 128 query rows of one head a workgroup, 32 a wave, q and
// dout in registers; keys and values through LDS.  It runs first and leaves, for
// each row, -lse log2(e) and -delta for the other kernel.
//
// dk, dv.  128 keys of a key head a workgroup, 32 a wave, k and v in registers;
// the queries and dout of all its heads through LDS.  Where the key tiles are
// too few to fill the chip, a tile's walk over the queries is cut into chunks
// whose partial sums a third kernel joins in order.
#include <algorithm>

#include "seq_attn.h"

namespace fp8lin {
namespace {

// What a row's gradients are formed from; NaN where the forward's results are
// not finite, which makes everything that the row sees NaN.
struct RowStat {
  float minus_lse2, minus_delta;
};
__device__ __forceinline__ RowStat row_stat(float lse, float delta) {
  const bool fine = lse - lse == 0.0f && delta - delta == 0.0f;
  return {fine ? lse * -1.44269504088896340736f : NAN, -delta};
}

template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void seq_attn_dq_kernel(SeqAttnArgs a) {
  constexpr int J = D / 16, DT = D / 32, kKeys = D == 256 ? 32 : 64;
  using Load = TileLoad<D, kKeys>;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[2][2][Load::kBytes];  // [buffer][keys, values]
  __shared__ int found[4];
  __shared__ int bad_key[kKeys];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  uint32_t x = a.first + blockIdx.x;
  const int kv_head = x % a.heads;
  x /= a.heads;
  const int head = kv_head * a.group + x % a.group;
  x /= a.group;
  const Seq s = seq_of(a, x % a.batch);
  const int row0 = (a.tiles - 1 - (int)(x / a.batch)) * kSeqRows;
  if (row0 >= s.n) return;
  const int khi = a.causal ? min(s.n, row0 + kSeqRows) : s.n;
  const int klo = a.window ? max(0, row0 - a.window + 1) & ~(kKeys - 1) : 0;

  const uint32_t ring0 = lds_addr(ring);
  const int64_t ks = a.k_stride * 2, vs = a.v_stride * 2;
  const Load load_k(lane, wave, (uint32_t)ks), load_v(lane, wave, (uint32_t)vs);
  const uint16_t* kp = a.k + (int64_t)(s.first + klo) * a.k_stride + kv_head * D;
  const uint16_t* vp = a.v + (int64_t)(s.first + klo) * a.v_stride + kv_head * D;
  auto issue = [&](int T, int buf) {
    load_k.issue(kp + (int64_t)(T - klo) * a.k_stride, ks, s.n - T, ring0 + buf * 2 * Load::kBytes, wave);
    load_v.issue(vp + (int64_t)(T - klo) * a.v_stride, vs, s.n - T, ring0 + (2 * buf + 1) * Load::kBytes, wave);
  };

  const int wrow = row0 + 32 * wave, row = wrow + r32;
  v8b q[J], g[J];
  float delta = 0.0f;
#pragma unroll
  for (int j = 0; j < J; ++j) q[j] = g[j] = v8b{};
  const int64_t cell = (int64_t)(s.first + min(row, s.n - 1)) * a.q_heads + head;
  if (row < s.n) {
    const uint16_t* qp = a.q + (int64_t)(s.first + row) * a.q_stride + head * D + 8 * h;
    const uint16_t* gp = a.dout + (int64_t)(s.first + row) * a.dout_stride + head * D + 8 * h;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      q[j] = *reinterpret_cast<const v8b*>(qp + 16 * j);
      g[j] = *reinterpret_cast<const v8b*>(gp + 16 * j);
      const v8b o = *reinterpret_cast<const v8b*>(a.out + cell * D + 8 * h + 16 * j);
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = fmaf((float)g[j][e], (float)o[e], delta);
    }
  }
  delta = swap32_sum(delta);
  const RowStat stat = row_stat(a.lse[cell], delta);
  if (row < s.n && h == 0) {
    const int64_t at = (int64_t)head * a.tokens + s.first + row;
    a.lse2[at] = stat.minus_lse2;
    a.delta[at] = stat.minus_delta;
  }
  issue(klo, 0);

  const int hi = a.causal ? min(row + 1, s.n) : s.n, lo = a.window ? row - a.window + 1 : 0;
  const int whi = wrow >= s.n ? 0 : (a.causal ? min(wrow + 32, s.n) : s.n);
  const int wlo = a.window ? wrow - a.window + 1 : 0;
  const int all_hi = a.causal ? min(s.n, row0 + 1) : s.n;
  const int all_lo = a.window ? min(row0 + kSeqRows, s.n) - a.window : 0;

  v16f dq[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) dq[d] = zero16();
  const uint32_t by_row = row_place<D>(lane), by_column = column_place<D>(lane);

  // 32 keys from position K on, in LDS at `keys` and `values`
  auto consume = [&](bool masked, bool any_bad, int K, uint32_t keys, uint32_t values, int slot) {
    v16f t = zero16(), dp;
#pragma unroll
    for (int e = 0; e < 16; ++e) dp[e] = stat.minus_delta;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      t = mma(lds_row((keys + by_row) ^ (32 * j)), q[j], t);
      dp = mma(lds_row((values + by_row) ^ (32 * j)), g[j], dp);
      if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
    if (any_bad) {
      asm volatile("");
#pragma unroll
      for (int e = 0; e < 16; ++e) t[e] = bad_key[slot + result_row(e, h)] ? NAN : t[e];
    }
    v16f ds;
#pragma unroll
    for (int e = 0; e < 16; ++e) ds[e] = __builtin_amdgcn_exp2f(fmaf(t[e], a.scale_log2, stat.minus_lse2)) * dp[e];
    if (masked) {
      asm volatile("");
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int key = K + result_row(e, h);
        ds[e] = key >= lo && key < hi ? ds[e] : 0.0f;
      }
    }
    v8b b[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) b[c] = operand(ds, c);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int d = 0; d < DT; ++d) dq[d] = mma(column_step<D>(keys + by_column + c * 32 * D, d), b[c], dq[d]);
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
    for (int sub = 0; sub < kKeys / 32; ++sub) {
      const int K = T + 32 * sub;
      if (K >= whi || K + 32 <= wlo) continue;
      const bool whole = K + 32 <= min(s.n, a.causal ? wrow + 1 : s.n) && (!a.window || K > wrow + 31 - a.window);
      consume(!whole, any_bad, K, keys + sub * 64 * D, values + sub * 64 * D, 32 * sub);
    }
  }

  if (row >= s.n) return;
  uint16_t* to = a.dq + (int64_t)(s.first + row) * a.dq_stride + head * D;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<uint2*>(to + 32 * d + 8 * u + 4 * h) =
          make_uint2(pack_bf16(dq[d][4 * u] * a.scale, dq[d][4 * u + 1] * a.scale),
                     pack_bf16(dq[d][4 * u + 2] * a.scale, dq[d][4 * u + 3] * a.scale));
}

// Query rows of a tile of the dk, dv kernel.
template <int D>
constexpr int kQueriesOf = D == 256 ? 32 : 64;

// A key tile's walk: tiles of query rows [lo, hi) of each head of the group.
struct Walk {
  int lo, tiles, chunks;
};
template <int D>
__device__ __forceinline__ Walk walk_of(const SeqAttnArgs& a, const Seq& s, int k0) {
  constexpr int kQueries = kQueriesOf<D>;
  Walk w;
  w.lo = a.causal ? k0 : 0;
  const int64_t hi = a.window ? (int64_t)min(k0 + kSeqRows, s.n) - 1 + a.window : s.n;
  w.tiles = ((int)min((int64_t)s.n, hi) - w.lo + kQueries - 1) / kQueries;
  w.chunks = (int)(((int64_t)w.tiles * a.group + a.chunk - 1) / a.chunk);
  return w;
}

template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void seq_attn_dkv_kernel(SeqAttnArgs a) {
  constexpr int J = D / 16, DT = D / 32, kQueries = kQueriesOf<D>;
  using Load = TileLoad<D, kQueries>;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[2][2][Load::kBytes];  // [buffer][queries, dout]
  __shared__ __attribute__((aligned(1024))) float stats[2][2][64];             // [buffer][-lse2, -delta]
  __shared__ int found[4];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  uint32_t x = a.first + blockIdx.x;
  const int kv_head = x % a.heads;
  x /= a.heads;
  const int split = x % a.splits;
  x /= a.splits;
  const Seq s = seq_of(a, x % a.batch);
  const int k0 = (int)(x / a.batch) * kSeqRows;  // early keys are seen most: first
  if (k0 >= s.n) return;
  const Walk walk = walk_of<D>(a, s, k0);
  if (split >= walk.chunks) return;
  const int it0 = split * a.chunk, its = (int)min((int64_t)a.chunk, (int64_t)walk.tiles * a.group - it0);

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
      v[j] = *reinterpret_cast<const v8b*>(vp + 16 * j);
    }
  }
  // the queries that see the lane's key
  const int lo = a.causal ? key : 0;
  const int hi = a.window ? (int)min((int64_t)s.n, (int64_t)key + a.window) : s.n;

  v16f dk[DT], dv[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) dk[d] = dv[d] = zero16();

  const uint32_t ring0 = lds_addr(ring), stats0 = lds_addr(stats);
  const int64_t qs = a.q_stride * 2, gs = a.dout_stride * 2;
  const Load load_q(lane, wave, (uint32_t)qs), load_g(lane, wave, (uint32_t)gs);
  auto issue = [&](int group, int t, int buf) {
    const int head = kv_head * a.group + group, T = walk.lo + t * kQueries, left = s.n - T;
    const int64_t token = s.first + T;
    load_q.issue(a.q + token * a.q_stride + head * D, qs, left, ring0 + buf * 2 * Load::kBytes, wave);
    load_g.issue(a.dout + token * a.dout_stride + head * D, gs, left, ring0 + (2 * buf + 1) * Load::kBytes, wave);
    // every wave brings all of the rows' statistics: the same words to the same place
    const int64_t at = (int64_t)head * a.tokens + token + min(lane, left - 1);
    dma4(a.lse2 + at, stats0 + buf * 512);
    dma4(a.delta + at, stats0 + buf * 512 + 256);
  };
  const uint32_t by_row = row_place<D>(lane), by_column = column_place<D>(lane);

  // 32 query rows from Q on, in LDS at `queries` and `grads`
  auto consume = [&](bool masked, int Q, uint32_t queries, uint32_t grads, const float* stat) {
    v16f t = zero16(), dp;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const v4f w = *reinterpret_cast<const v4f*>(stat + 64 + 8 * u + 4 * h);
#pragma unroll
      for (int e = 0; e < 4; ++e) dp[4 * u + e] = w[e];
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      t = mma(lds_row((queries + by_row) ^ (32 * j)), k[j], t);
      dp = mma(lds_row((grads + by_row) ^ (32 * j)), v[j], dp);
      if (j % 2 == 1) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const v4f w = *reinterpret_cast<const v4f*>(stat + 8 * u + 4 * h);
#pragma unroll
      for (int e = 0; e < 4; ++e) t[4 * u + e] = __builtin_amdgcn_exp2f(fmaf(t[4 * u + e], a.scale_log2, w[e]));
    }
    if (masked) {
      asm volatile("");
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int row = Q + result_row(e, h);
        const bool seen = row >= lo && row < hi;
        t[e] = seen ? t[e] : 0.0f;
        dp[e] = seen ? dp[e] : 0.0f;
      }
    }
    v8b p[2], ds[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) p[c] = operand(t, c);
    dp *= t;
#pragma unroll
    for (int c = 0; c < 2; ++c) ds[c] = operand(dp, c);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        dv[d] = mma(column_step<D>(grads + by_column + c * 32 * D, d), p[c], dv[d]);
        dk[d] = mma(column_step<D>(queries + by_column + c * 32 * D, d), ds[c], dk[d]);
        if (d % 2 == 1) __builtin_amdgcn_sched_barrier(0);
      }
  };

  int group = it0 / walk.tiles, t = it0 % walk.tiles, buf = 0;
  issue(group, t, 0);
  for (int it = 0; it < its; ++it, buf ^= 1) {
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
    for (int sub = 0; sub < kQueries / 32; ++sub) {
      const int Q = T + 32 * sub;
      if (wkey >= s.n || Q >= s.n || (a.causal && Q + 31 < wkey)) continue;
      if (a.window && Q >= (int64_t)wkey + 31 + a.window) continue;
      const bool whole = Q + 32 <= s.n && (!a.causal || Q >= wkey + 31) &&
                         (!a.window || Q + 31 < (int64_t)wkey + a.window);
      consume(!whole, Q, queries + sub * 64 * D, grads + sub * 64 * D, &stats[buf][0][32 * sub]);
    }
  }

  if (key >= s.n) return;
  const int64_t token = s.first + key;
  if (walk.chunks == 1) {
    uint16_t* to_k = a.dk + token * a.dk_stride + kv_head * D + 4 * h;
    uint16_t* to_v = a.dv + token * a.dv_stride + kv_head * D + 4 * h;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = 4 * u;
        *reinterpret_cast<uint2*>(to_k + 32 * d + 8 * u) =
            make_uint2(pack_bf16(dk[d][e] * a.scale, dk[d][e + 1] * a.scale),
                       pack_bf16(dk[d][e + 2] * a.scale, dk[d][e + 3] * a.scale));
        *reinterpret_cast<uint2*>(to_v + 32 * d + 8 * u) =
            make_uint2(pack_bf16(dv[d][e], dv[d][e + 1]), pack_bf16(dv[d][e + 2], dv[d][e + 3]));
      }
    return;
  }
  const int64_t at = (((int64_t)split * a.tokens + token) * a.heads + kv_head) * D + 4 * h;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = 4 * u;
      *reinterpret_cast<v4f*>(a.part_k + at + 32 * d + 8 * u) = v4f{dk[d][e], dk[d][e + 1], dk[d][e + 2], dk[d][e + 3]};
      *reinterpret_cast<v4f*>(a.part_v + at + 32 * d + 8 * u) = v4f{dv[d][e], dv[d][e + 1], dv[d][e + 2], dv[d][e + 3]};
    }
}

// Adds the chunks' sums of key tiles that were split, in order.
template <int D>
__global__ __launch_bounds__(256) void seq_attn_join_kernel(SeqAttnArgs a) {
  uint32_t x = a.first + blockIdx.x;
  const int kv_head = x % a.heads;
  x /= a.heads;
  const Seq s = seq_of(a, x % a.batch);
  const int k0 = (int)(x / a.batch) * kSeqRows;
  if (k0 >= s.n) return;
  const int chunks = walk_of<D>(a, s, k0).chunks;
  if (chunks == 1) return;
  const int keys = min(kSeqRows, s.n - k0);
  const int64_t step = (int64_t)a.tokens * a.heads * D;
  for (int i = threadIdx.x; i < keys * (D / 4); i += 256) {
    const int64_t token = s.first + k0 + i / (D / 4);
    const int d = 4 * (i % (D / 4));
    const int64_t at = (token * a.heads + kv_head) * D + d;
    v4f k = *reinterpret_cast<const v4f*>(a.part_k + at), v = *reinterpret_cast<const v4f*>(a.part_v + at);
    for (int c = 1; c < chunks; ++c) {
      k += *reinterpret_cast<const v4f*>(a.part_k + at + c * step);
      v += *reinterpret_cast<const v4f*>(a.part_v + at + c * step);
    }
    k *= a.scale;
    *reinterpret_cast<uint2*>(a.dk + token * a.dk_stride + kv_head * D + d) =
        make_uint2(pack_bf16(k[0], k[1]), pack_bf16(k[2], k[3]));
    *reinterpret_cast<uint2*>(a.dv + token * a.dv_stride + kv_head * D + d) =
        make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  }
}

// How the walks of the key tiles are cut: chunk in query tiles, the most chunks
// of one.  From the shape alone, so that the workspace does not depend on the mask.
struct Cut {
  int chunk, splits;
};
Cut cut_of(const SeqAttnShape& s) {
  const int64_t queries = s.head_dim == 256 ? 32 : 64;
  const int64_t longest = (s.max_len + queries - 1) / queries * (s.q_heads / s.heads);  // of a key tile's walk
  const int64_t key_tiles = (s.tokens + kSeqRows - 1) / kSeqRows;                       // about, of all sequences
  // enough chunks for four workgroups a CU, none shorter than eight tiles
  const int64_t want = 1024, have = key_tiles * s.heads;
  const int64_t splits = std::max<int64_t>(1, std::min(want / std::max<int64_t>(have, 1), longest / 8));
  const int64_t chunk = (longest + splits - 1) / splits;
  return {(int)chunk, (int)((longest + chunk - 1) / chunk)};
}

int64_t aligned(int64_t bytes) { return (bytes + 255) & ~(int64_t)255; }
int64_t stat_bytes(const SeqAttnShape& s) { return aligned((int64_t)s.tokens * s.q_heads * 4); }
int64_t part_bytes(const SeqAttnShape& s, int splits) {
  return aligned((int64_t)splits * s.tokens * s.heads * s.head_dim * 4);
}

template <int D>
void run_bwd(SeqAttnArgs& a, hipStream_t stream) {
  auto launch = [&](auto kernel, int64_t groups) {
    in_stretches(groups, 256, [&](uint32_t first, uint32_t count) {
      a.first = first;
      hipLaunchKernelGGL(kernel, dim3(count), dim3(256), 0, stream, a);
    });
  };
  const int64_t tiles = (int64_t)a.tiles * a.batch;
  launch(seq_attn_dq_kernel<D>, tiles * a.q_heads);
  launch(seq_attn_dkv_kernel<D>, tiles * a.heads * a.splits);
  if (a.splits > 1) launch(seq_attn_join_kernel<D>, tiles * a.heads);
}

}  // namespace

int64_t seq_attn_bwd_workspace_bytes(const SeqAttnShape& s) {
  const Cut c = cut_of(s);
  return 2 * stat_bytes(s) + (c.splits > 1 ? 2 * part_bytes(s, c.splits) : 0);
}

hipError_t launch_seq_attn_bwd(SeqAttnArgs a, int head_dim, void* ws, hipStream_t stream) {
  const SeqAttnShape s{a.batch, a.tokens, a.max_len, a.q_heads, a.heads, head_dim};
  const Cut c = cut_of(s);
  a.chunk = c.chunk;
  a.splits = c.splits;
  a.tiles = (a.max_len + kSeqRows - 1) / kSeqRows;
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.lse2 = reinterpret_cast<float*>(p);
  a.delta = reinterpret_cast<float*>(p + stat_bytes(s));
  a.part_k = reinterpret_cast<float*>(p + 2 * stat_bytes(s));
  a.part_v = reinterpret_cast<float*>(p + 2 * stat_bytes(s) + part_bytes(s, c.splits));
  if (head_dim == 64) run_bwd<64>(a, stream);
  else if (head_dim == 128) run_bwd<128>(a, stream);
  else run_bwd<256>(a, stream);
  return hipGetLastError();
}

}  // namespace fp8lin
