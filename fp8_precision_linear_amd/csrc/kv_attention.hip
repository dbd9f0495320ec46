// Attention over the paged FP8 cache: which kernel takes a batch, how its keys
// are split, and the join of split results (attn_common.h, attn_rows.hip,
// attn_tile.hip).
#include "attn_common.h"

namespace fp8lin {
namespace {

struct AttnPlan {
  bool few;          // the rows kernel
  int row_blocks;    // of 16, rows kernel
  int tile_rows;     // rows per row tile
  int row_tiles;     // most of any sequence
  int chunk, splits;
  int64_t base;         // workgroups without a split
  int64_t most_splits;  // whatever the window
};

// Workgroups wanted in flight: four (rows) or two (tiles) for each of 256 CUs.
constexpr int64_t kWantRows = 1024, kWantTiles = 512;

AttnPlan plan_of(const fp8_kv_cache_t& c, const fp8_kv_batch_t& b, int q_heads, int window) {
  AttnPlan p{};
  const int64_t rows = (int64_t)b.max_new * (q_heads / c.heads);
  p.few = rows <= 32;
  p.row_blocks = rows <= 16 || c.head_dim == 256 ? 1 : 2;
  p.tile_rows = p.few ? 16 * p.row_blocks : kAttnTileRows;
  p.row_tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
  p.base = (int64_t)p.row_tiles * b.batch * c.heads;
  int64_t span = b.max_len;  // most keys of a row tile
  if (window > 0) span = span < (int64_t)window + b.max_new + kAttnTile ? span : (int64_t)window + b.max_new + kAttnTile;
  const int64_t tiles = span > 0 ? (span + kAttnTile - 1) / kAttnTile : 1;
  // no chunk below four tiles (one for each wave of the rows kernel)
  const int64_t want = ((p.few ? kWantRows : kWantTiles) + p.base - 1) / p.base;
  int64_t per = (tiles + want - 1) / want;
  per = (per + 3) / 4 * 4;
  p.splits = (int)((tiles + per - 1) / per);
  p.chunk = (int)(per * kAttnTile);
  const int64_t full = ((int64_t)b.max_len + 4 * kAttnTile - 1) / (4 * kAttnTile);
  p.most_splits = want < full ? want : (full > 0 ? full : 1);
  return p;
}

// One workgroup per new token: joins the chunks of each of its heads that was
// split.  out = sum_c 2^(lse_c - L) out_c, L = log2 sum_c 2^lse_c.
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int tile_rows) {
  const int i = blockIdx.x % a.batch.batch, nth = blockIdx.x / a.batch.batch;
  const KVSeq s = kv_seq(a.batch, a.cache.block_size, i);
  if (nth >= s.n) return;
  const int D = a.cache.head_dim, G = a.group, upr = D / 4;
  const int64_t row0 = (int64_t)(s.first + nth) * a.q_heads;
  const int64_t step = (int64_t)a.batch.tokens * a.q_heads;
  for (int x = threadIdx.x; x < a.q_heads * upr; x += 256) {
    const int head = x / upr, d = 4 * (x % upr);
    const int tile = (nth * G + head % G) / tile_rows;
    const int chunks = attn_span(a, s, tile * tile_rows, tile_rows).chunks;
    if (chunks == 1) continue;
    const int64_t at = row0 + head;
    float top = -INFINITY;
    for (int c = 0; c < chunks; ++c) top = fmaxf(top, a.part_lse[c * step + at]);
    float total = 0.0f;
    v4f sum{0, 0, 0, 0};
    for (int c = 0; c < chunks; ++c) {
      const float lse = a.part_lse[c * step + at];
      // a chunk without visible keys has lse = -inf and adds nothing
      const float f = lse == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(lse - top);
      total += f;
      sum += *reinterpret_cast<const v4f*>(a.part_o + (c * step + at) * D + d) * f;
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    *reinterpret_cast<uint2*>(a.out + at * D + d) =
        make_uint2(pack_bf16(sum[0] * inv, sum[1] * inv), pack_bf16(sum[2] * inv, sum[3] * inv));
    if (d == 0 && a.lse) a.lse[at] = total == 0.0f ? -INFINITY : (top + log2f(total)) * 0.693147180559945309f;
  }
}

}  // namespace

int64_t kv_attention_workspace_bytes(const fp8_kv_cache_t& c, const fp8_kv_batch_t& b, int q_heads) {
  // the window may shorten the span and so raise the split, up to this
  const AttnPlan p = plan_of(c, b, q_heads, 0);
  if (p.base > 0x7FFFFFFF / p.most_splits) return FP8_ERR_SIZE;
  if (p.most_splits == 1) return 0;
  return p.most_splits * b.tokens * q_heads * (c.head_dim + 1) * 4;
}

hipError_t launch_kv_attention(const AttnProblem& pr, void* ws, hipStream_t stream) {
  const AttnPlan p = plan_of(pr.cache, pr.batch, pr.q_heads, pr.window);
  AttnArgs a{};
  a.cache = pr.cache;
  a.batch = pr.batch;
  a.q = pr.q;
  a.q_stride = pr.q_stride;
  a.q_heads = pr.q_heads;
  a.group = pr.q_heads / pr.cache.heads;
  a.scale_log2 = pr.scale * 1.44269504088896340736f;
  a.causal = pr.causal;
  a.window = pr.window;
  a.out = pr.out;
  a.lse = pr.lse;
  a.part_o = static_cast<float*>(ws);
  a.part_lse = a.part_o + (int64_t)p.splits * pr.batch.tokens * pr.q_heads * pr.cache.head_dim;
  a.chunk = p.chunk;
  a.splits = p.splits;
  a.row_tiles = p.row_tiles;
  const uint32_t groups = (uint32_t)(p.base * p.splits);
  hipError_t e = p.few ? launch_attn_rows(a, p.row_blocks, groups, stream)
                       : launch_attn_tile(a, groups, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t tokens = (int64_t)pr.batch.batch * pr.batch.max_new;
  hipLaunchKernelGGL(attn_join_kernel, dim3((uint32_t)tokens), dim3(256), 0, stream, a, p.tile_rows);
  return hipGetLastError();
}

}  // namespace fp8lin
