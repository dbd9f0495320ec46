// Attention over the paged FP8 cache: which kernel takes a batch, how its keys
// are split, and the join of split results (attn_common.h, attn_rows.hip,
// attn_tile.hip).
#include <climits>
#include <cmath>

#include "attn_common.h"

namespace fp8lin {
namespace {

struct AttnPlan {
  int max_new;          // most new tokens of a sequence that is served
  bool few;             // the rows kernel
  int row_blocks;       // of 16, rows kernel
  int tile_rows;        // rows per row tile
  int row_tiles;        // most of any sequence
  int shares;           // rows kernel: workgroups of the even shares, or 0
  int chunk, splits;    // tile kernel
  int64_t base;         // workgroups without a split
  int64_t most_splits;  // tile kernel, whatever the window
};

// Tile kernel: workgroups wanted in flight, two for each of 256 CUs, and the
// fewest tiles of a chunk.  Where whole row tiles leave CUs without work, short
// chunks pay (247 tokens of 16 heads of 256 on 808 cached: chunks of 4 tiles 33
// us, of 6 38, of 10 47); where they do not, the join costs more than a second
// workgroup a CU saves (two prompts of up to 1303 tokens, 32 heads of 64 on 8:
// two chunks 42 us, whole 27).
constexpr int64_t kWantTiles = 512, kCUs = 256, kLeastTiles = 4, kLeastTilesFull = 32;
// Rows kernel: even shares where a segment may hold more tiles than this.  The
// join costs some 8 us, and a segment's tiles 2 to 3 us for every four: one
// sequence of 1000 tokens, 8 heads of 128, whole 13.6 us and in shares 12.5, of
// 1500 17.2 and 12.7, of 2500 23.7 and 12.8; 32 sequences of 500 to 1000 tokens
// 17.2 and 23.1, of 750 to 1500 21.8 and 25.5, of 1250 to 2500 29.6 and 32.2.
constexpr int64_t kWholeTiles = 24;

// Rows of a key head up to which a sequence is the rows kernel's.
constexpr int kFewRows = 32;
// max_new: most new tokens of the sequences that the plan is for.
AttnPlan plan_of(const fp8_kv_cache_t& c, const fp8_kv_batch_t& b, int q_heads, int window, int max_new) {
  AttnPlan p{};
  const int64_t rows = (int64_t)max_new * (q_heads / c.heads);
  p.max_new = max_new;
  p.few = rows <= kFewRows;
  p.row_blocks = rows <= 16 || c.head_dim == 256 ? 1 : 2;
  p.tile_rows = p.few ? 16 * p.row_blocks : kAttnTileRows;
  p.row_tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
  p.base = (int64_t)p.row_tiles * b.batch * c.heads;
  p.chunk = kAttnTile, p.splits = 1, p.most_splits = 1;
  if (p.few) {
    const int resident = attn_rows_resident(c.head_dim, p.row_blocks);
    if ((b.max_len + kAttnTile - 1) / kAttnTile > kWholeTiles && p.base < 16 * (int64_t)resident) p.shares = resident;
    return p;
  }
  int64_t span = b.max_len;  // most keys of a row tile
  if (window > 0) span = span < (int64_t)window + max_new + kAttnTile ? span : (int64_t)window + max_new + kAttnTile;
  const int64_t tiles = span > 0 ? (span + kAttnTile - 1) / kAttnTile : 1;
  const int64_t want = (kWantTiles + p.base - 1) / p.base;
  int64_t per = (tiles + want - 1) / want;
  const int64_t fewest = p.base < kCUs ? kLeastTiles : kLeastTilesFull;
  per = per < fewest ? fewest : per;
  p.splits = (int)((tiles + per - 1) / per);
  p.chunk = (int)(per * kAttnTile);
  const int64_t least = fewest * kAttnTile, full = (b.max_len + least - 1) / least;
  p.most_splits = want < full ? want : (full > 0 ? full : 1);
  return p;
}

// Mixed batches: sequences of few rows beside some of many get the rows kernel, in
// launches of their own, where a workgroup of the tile kernel would walk their
// keys for longer than that takes: a tile of 64 keys costs it about 1 us, the
// launches 30 us and the caches' reading at 5 TB/s.  Half as much again is asked,
// since the walk may hide behind the longer sequences' work.  A prompt of 512
// tokens beside one token on 131071, 64 heads on 8 of 128: one kernel 2370 us, two
// 91, on 8000 154 and 43, on 2000 47 and 39 (left to one); a prompt of 2000 beside
// one token on 3000, 32 heads: one kernel 82 us, two 96, on 8000 170 and 100.
//
// Returns the most new tokens of a sequence that the rows kernel takes, or 0
// where the rule says no or the batch's bounds leave no room for such a sequence.
int mixed_new(const fp8_kv_cache_t& c, const fp8_kv_batch_t& b, int q_heads, int window) {
  const int n = kFewRows / (q_heads / c.heads);
  if (n == 0 || b.max_new <= n || (int64_t)b.tokens > (int64_t)(b.batch - 1) * b.max_new + n) return 0;
  auto pays = [&](int w) {
    const double keys = w > 0 && w < b.max_len ? w : b.max_len;
    const double apart = 30.0 + keys * b.batch * c.heads * c.head_dim * 2 / 5e6;  // us
    const double walk = plan_of(c, b, q_heads, w, b.max_new).chunk / kAttnTile;
    return walk > 1.5 * apart;
  };
  // (a workspace is made without knowing the window)
  return pays(0) && (window == 0 || pays(window)) ? n : 0;
}

// Rows of partial results.
int64_t part_rows(const AttnPlan& p, const fp8_kv_batch_t& b, int q_heads, int64_t splits) {
  return p.few ? 2 * (int64_t)p.shares * p.tile_rows : splits * b.tokens * q_heads;
}

// Workspace of a plan whose batch is cut into up to `splits` chunks: partial
// outputs, references and sums, and for even shares the segments' workgroups.  A
// multiple of 16.
int64_t plan_bytes(const AttnPlan& p, const fp8_kv_cache_t& c, const fp8_kv_batch_t& b, int q_heads, int64_t splits) {
  if (p.shares == 0 && splits == 1) return 0;
  const int64_t n = part_rows(p, b, q_heads, splits) * (c.head_dim + 2) * 4 + (p.shares ? p.base * 8 : 0);
  return (n + 15) / 16 * 16;
}

// The join of a (new token, query head) whose keys were split into parts
// (chunks, or shares): out = sum_c w_c out_c / sum_c w_c, w_c = l_c 2^(m_c - M),
// with M the largest reference of a part that sees keys (one that sees none has
// l = 0 and out = 0; a weight that underflows still carries a NaN on).  The
// parts' references and sums stay apart until here: added to a large reference a
// sum would be rounded away.  out is kept divided by the weights' sum throughout,
// since a value times a sum could pass fp32's range.
// A row of D / 4 lanes joins `few` parts alone, several rows a workgroup; many
// parts are dealt to all rows of a workgroup, which meet in LDS in order.
constexpr int kJoin = 256;
constexpr int kFewParts = 16;
__global__ __launch_bounds__(kJoin) void attn_join_kernel(AttnArgs a, int tile_rows, bool few, int max_new) {
  __shared__ v4f so[kJoin];
  __shared__ float ss[kJoin], st[kJoin];
  const int D = a.cache.head_dim, lanes = D / 4, t = threadIdx.x;
  const int64_t index = few ? (int64_t)blockIdx.x * (kJoin / lanes) + t / lanes : blockIdx.x;
  const int head = index % a.q_heads;
  const uint32_t x = index / a.q_heads;
  const int i = x % a.batch.batch, nth = x / a.batch.batch;
  if (nth >= max_new) return;
  const int row = nth * a.group + head % a.group, tile = row / tile_rows;
  int2 w{0, 0};
  if (a.shares) w = a.segments[((int64_t)i * a.row_tiles + tile) * a.cache.heads + head / a.group];
  const KVSeq s = kv_seq(a.batch, a.cache.block_size, i);
  if (nth >= s.n || !attn_serves(a, s)) return;
  const int64_t at = (int64_t)(s.first + nth) * a.q_heads + head;
  // part c's row of part_o and part_sum: first for c = 0, then from `base` by step
  int64_t first = at, base = at, step = (int64_t)a.batch.tokens * a.q_heads;
  int chunks;
  if (a.shares) {
    chunks = w.y - w.x + 1;
    first = (2 * (int64_t)w.x + 1) * tile_rows + row % tile_rows;
    base = 2 * (int64_t)w.x * tile_rows + row % tile_rows;
    step = 2 * tile_rows;
  } else {
    chunks = attn_span(a, s, tile * tile_rows, tile_rows).chunks;
  }
  if (chunks <= 1) return;
  const int share = few ? 0 : t / lanes, shares = few ? 1 : kJoin / lanes, d = 4 * (t % lanes);
  // four parts at a time, their results and sums loaded together
  constexpr int kAhead = 4;
  float top = -INFINITY, total = 0.0f;
  v4f sum{0, 0, 0, 0};
  for (int c0 = share; c0 < chunks; c0 += kAhead * shares) {
    float2 ml[kAhead];
    v4f v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int c = c0 + u * shares;
      const int real = c < chunks ? c : c0;
      const int64_t p = real == 0 ? first : base + real * step;
      ml[u] = a.part_sum[p];
      if (c >= chunks) ml[u].y = 0.0f;
      v[u] = *reinterpret_cast<const v4f*>(a.part_o + p * D + d);
    }
    float up = top;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) up = ml[u].y == 0.0f ? up : fmaxf(up, ml[u].x);
    const float before = total == 0.0f ? 0.0f : total * __builtin_amdgcn_exp2f(top - up);
    float w[kAhead];
    top = up, total = before;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      w[u] = ml[u].y == 0.0f ? 0.0f : ml[u].y * __builtin_amdgcn_exp2f(ml[u].x - top);
      total += w[u];
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    sum *= before * inv;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) sum += v[u] * (w[u] * inv);
  }
  if (!few) {
    so[t] = sum;
    ss[t] = total;
    st[t] = top;
    __syncthreads();
    if (t >= lanes) return;
    float most = total;  // what the weights may add up to
    for (int k = 1; k < shares; ++k) {
      top = fmaxf(top, st[k * lanes + t]);
      most += ss[k * lanes + t];
    }
    const float down = most == 0.0f ? 0.0f : 1.0f / most;
    sum = v4f{0, 0, 0, 0};
    total = 0.0f;
    for (int k = 0; k < shares; ++k) {
      const float part = st[k * lanes + t];
      const float f = part == -INFINITY ? 0.0f : ss[k * lanes + t] * __builtin_amdgcn_exp2f(part - top);
      sum += so[k * lanes + t] * (f * down);
      total += f;
    }
    sum *= total == 0.0f ? 0.0f : most / total;
  }
  *reinterpret_cast<uint2*>(a.out + at * D + d) = make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
  if (d == 0 && a.lse) a.lse[at] = row_lse(top, total);
}

}  // namespace

int64_t kv_attention_workspace_bytes(const fp8_kv_cache_t& c, const fp8_kv_batch_t& b, int q_heads) {
  // the kernels number a key head's rows in 32 bits, up to the end of a tile
  if ((int64_t)b.max_new * (q_heads / c.heads) > 0x7FFFFFFF - kAttnTileRows) return FP8_ERR_SIZE;
  // tiles of a sequence over its heads are counted in 32 bits
  if ((int64_t)c.heads * (b.max_len / kAttnTile + 1) > 0x7FFFFFFF) return FP8_ERR_SIZE;
  // the window may shorten the span and so raise the split, up to most_splits, and
  // leave a mixed batch to one kernel
  const AttnPlan p = plan_of(c, b, q_heads, 0, b.max_new);
  if (p.base > 0x7FFFFFFF / p.most_splits) return FP8_ERR_SIZE;
  // the join's workgroups
  if ((p.shares || p.most_splits > 1) && (int64_t)b.batch * b.max_new > 0x7FFFFFFF / q_heads) return FP8_ERR_SIZE;
  const int64_t bytes = plan_bytes(p, c, b, q_heads, p.most_splits);
  const int few = mixed_new(c, b, q_heads, 0);
  return bytes + (few ? plan_bytes(plan_of(c, b, q_heads, 0, few), c, b, q_heads, 1) : 0);
}

hipError_t launch_kv_attention(const AttnProblem& pr, void* ws, hipStream_t stream) {
  AttnArgs a{};
  a.cache = pr.cache;
  a.batch = pr.batch;
  a.q = pr.q;
  a.q_stride = pr.q_stride;
  a.q_heads = pr.q_heads;
  a.group = pr.q_heads / pr.cache.heads;
  a.block_shift = __builtin_ctz(pr.cache.block_size);
  a.scale = pr.scale;
  a.scale_log2 = pr.scale == 0.0f ? 1.0f : fabsf(pr.scale) * 1.44269504088896340736f;
  a.causal = pr.causal;
  a.window = pr.window;
  a.out = pr.out;
  a.lse = pr.lse;
  // the launches of a plan, for sequences of `least` to `most` rows of a key head
  auto run = [&](const AttnPlan& p, int least, int most) -> hipError_t {
    a.least = least;
    a.most = most;
    a.part_o = static_cast<float*>(ws);
    const int64_t parts = part_rows(p, pr.batch, pr.q_heads, p.splits);
    a.part_sum = reinterpret_cast<float2*>(a.part_o + parts * pr.cache.head_dim);
    a.segments = reinterpret_cast<int2*>(a.part_sum + parts);
    ws = static_cast<char*>(ws) + plan_bytes(p, pr.cache, pr.batch, pr.q_heads, p.splits);
    a.shares = p.shares;
    a.chunk = p.chunk;
    a.splits = p.splits;
    a.row_tiles = p.row_tiles;
    hipError_t e = hipSuccess;
    in_stretches(p.shares ? p.shares : p.base * p.splits, kAttnThreads, [&](uint32_t first, uint32_t count) {
      if (e != hipSuccess) return;
      a.first = first;
      e = p.few ? launch_attn_rows(a, p.row_blocks, count, stream) : launch_attn_tile(a, count, stream);
    });
    if (e != hipSuccess || (p.splits == 1 && p.shares == 0)) return e;
    const int64_t joins = (int64_t)pr.batch.batch * p.max_new * pr.q_heads;
    // shares: a segment's parts are about its tiles over a share's
    const int64_t parts_most = p.shares ? (p.base < p.shares ? (p.shares + p.base - 1) / p.base + 1 : 3) : p.splits;
    const bool few = parts_most <= kFewParts;
    const int per = few ? kJoin / (pr.cache.head_dim / 4) : 1;
    hipLaunchKernelGGL(attn_join_kernel, dim3((uint32_t)((joins + per - 1) / per)), dim3(kJoin), 0, stream, a,
                       p.tile_rows, few, p.max_new);
    return hipGetLastError();
  };
  const AttnPlan whole = plan_of(pr.cache, pr.batch, pr.q_heads, pr.window, pr.batch.max_new);
  const int few = mixed_new(pr.cache, pr.batch, pr.q_heads, pr.window);
  if (!few) return run(whole, 0, INT_MAX);
  const hipError_t e = run(whole, kFewRows + 1, INT_MAX);
  if (e != hipSuccess) return e;
  return run(plan_of(pr.cache, pr.batch, pr.q_heads, pr.window, few), 0, kFewRows);
}

}  // namespace fp8lin
