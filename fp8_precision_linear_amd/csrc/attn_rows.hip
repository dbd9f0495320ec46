// Attention of a few query rows (single tokens, short drafts) over the paged
// FP8 cache: attn_common.h has the mathematics.
//
// HBM-bound: every cached byte of the (sequence, key head) is read once and
// serves the group's query rows, 16 per MFMA tile.  Workgroups of four waves
// take the keys of one segment, or an even share of all of them; the waves take
// its tiles of 64 keys in turn, each with its own running maximum, sum and O,
// and meet in LDS at the end.  Keys and values go from memory straight to
// registers: a load instruction covers whole 64-byte runs, and the next tile's
// keys are in flight during this tile's softmax, its values during the next
// one's logits.
//
// 131071 tokens of 8 heads of 128: 268 MB in 50-52 us (5.3 TB/s), and 6 us of
// join; 32 sequences of 1000 to 8191 tokens: 302 MB in 65-68 us (4.5 TB/s: the
// start, the walk to a share's first segment and the meeting in LDS cost some
// 10 us of it), and 5 us of join.  One workgroup per segment instead of even
// shares took 107 us over the 32.
#include "attn_common.h"

namespace fp8lin {
namespace {

constexpr int kWaves = kAttnWaves;

// Waves of one SIMD (registers allow that many).
template <int D, int RB>
constexpr int kOcc = D * RB >= 256 ? 1 : (D * RB == 128 ? 2 : 3);

// A workgroup's keys.  Directly: all keys of its (sequence, row tile, head).
// Shared: the tiles of all segments -- (sequence, row tile, head) in that
// order -- form one line that the workgroups cut into equal shares, so that
// ragged lengths and any batch size load every CU alike; a segment cut by a
// share's end leaves partial results, joined afterwards.
struct Segment {
  int pair;         // sequence * row_tiles + row tile
  int head;
  int first, last;  // this workgroup's tiles [first, last) of the segment
};

// A pair's sequence and its tiles (0: no such rows; at least 1 otherwise).
struct Pair {
  KVSeq s;
  int tiles;
};
template <int ROWS>
__device__ __forceinline__ Pair pair_of(const AttnArgs& a, int p) {
  Pair r{{0, 0, 0, 0}, 0};
  if (p >= a.batch.batch * a.row_tiles) return r;
  const int i = a.row_tiles == 1 ? p : p / a.row_tiles;
  r.s = kv_seq(a.batch, a.cache.block_size, i);
  const int row0 = (p - i * a.row_tiles) * ROWS;
  if (row0 >= r.s.n * a.group || !attn_serves(a, r.s)) return r;
  const AttnSpan span = attn_span(a, r.s, row0, ROWS);
  r.tiles = max(1, (span.hi - span.lo + kAttnTile - 1) / kAttnTile);
  return r;
}
__device__ __forceinline__ Pair pair_from(const Pair& p, int lane) {
  return {{__builtin_amdgcn_readlane(p.s.first, lane), __builtin_amdgcn_readlane(p.s.n, lane),
           __builtin_amdgcn_readlane(p.s.start, lane), __builtin_amdgcn_readlane(p.s.len, lane)},
          __builtin_amdgcn_readlane(p.tiles, lane)};
}

// A tile that some rows do not see whole: no code of an invisible slot may turn
// 0 * code into NaN, so NaN (and infinity) codes become zeros; where a row does
// see such a token, its output becomes NaN.  Those are counted by a product of
// visibility with "is bad".  see(rb, e): whether this lane's row of block rb
// sees key e of its granule.
template <int FMT, int RB, int DT, typename F>
__device__ __forceinline__ void clean_values(uint4 (&v)[DT], v4f (&o)[RB][DT], F&& see) {
  uint32_t bad = 0;
#pragma unroll
  for (int d = 0; d < DT; ++d)
    bad |= bad_bytes<FMT>(v[d].x) | bad_bytes<FMT>(v[d].y) | bad_bytes<FMT>(v[d].z) | bad_bytes<FMT>(v[d].w);
  if (!__any(bad != 0)) return;
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    v8h s[2];
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e >> 3][e & 7] = see(rb, e) ? (_Float16)1.0f : (_Float16)0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      __builtin_amdgcn_sched_barrier(0);
      uint4 w = v[d];
      // or the masks above stay in registers until here
      asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
      v4f n{0, 0, 0, 0};
      n = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones_f16(bad_bytes<FMT>(w.x), bad_bytes<FMT>(w.y)), s[0], n, 0, 0, 0);
      n = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones_f16(bad_bytes<FMT>(w.z), bad_bytes<FMT>(w.w)), s[1], n, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[rb][d][e] = n[e] > 0.0f ? NAN : o[rb][d][e];
    }
  }
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    asm volatile("" : "+v"(v[d].x), "+v"(v[d].y), "+v"(v[d].z), "+v"(v[d].w));
    v[d].x &= ~bad_bytes<FMT>(v[d].x);
    v[d].y &= ~bad_bytes<FMT>(v[d].y);
    v[d].z &= ~bad_bytes<FMT>(v[d].z);
    v[d].w &= ~bad_bytes<FMT>(v[d].w);
  }
}

template <int D, int FMT, int RB, bool ONE>
__global__ __launch_bounds__(64 * kWaves, (kOcc<D, RB>)) void attn_rows_kernel(AttnArgs a) {
  constexpr int kRows = 16 * RB;
  constexpr int J = D / 64;   // 64-dimension steps of the logits
  constexpr int DT = D / 16;  // 16-dimension tiles of the output
  constexpr int kPitch = D + 4;
  __shared__ float so[kWaves][16][kPitch];
  __shared__ float sm[kWaves][kRows], sl[kWaves][kRows];
  __shared__ int sb[kWaves];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int BS = a.cache.block_size, H = a.cache.heads, G = a.group;

  Segment seg;
  Pair pair;
  int64_t at = 0, end = 1, share = 0;  // this workgroup's stretch of the line of tiles
  if (a.shares) {
    // prefix sums over the pairs, 64 at a time: the line's length first, then
    // the pair that holds tile `at` (a second reading only past 64 pairs)
    const int pairs = a.batch.batch * a.row_tiles;
    Pair mine;
    int64_t upto = 0, base = 0, total = 0;
    auto scan = [&](int p) {
      mine = pair_of<kRows>(a, p + lane);
      upto = (int64_t)mine.tiles * H;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int64_t v = __shfl_up(upto, off, 64);
        if (lane >= off) upto += v;
      }
      upto += base;
      base = __shfl(upto, 63, 64);
    };
    for (int p = 0; p < pairs; p += 64) scan(p);
    total = base;
    share = max((int64_t)kWaves, (total + a.shares - 1) / a.shares);
    at = blockIdx.x * share;
    end = min(total, at + share);
    if (at >= end) return;
    int p = 0;
    if (pairs > 64) {
      base = 0;
      for (;; p += 64) {
        if (p >= pairs) return;  // the device's lengths changed under the call
        scan(p);
        if (base > at) break;
      }
    }
    const int k = __builtin_ctzll(__ballot(upto > at));
    pair = pair_from(mine, k);
    seg.pair = p + k;
    const int64_t rel = at - (__shfl(upto, k, 64) - (int64_t)pair.tiles * H);
    seg.head = __builtin_amdgcn_readfirstlane((int)((uint32_t)rel / (uint32_t)pair.tiles));
    seg.first = __builtin_amdgcn_readfirstlane((int)((uint32_t)rel % (uint32_t)pair.tiles));
  } else {
    const AttnPlace pl = attn_place(a);
    seg.pair = pl.seq * a.row_tiles + pl.row_tile;
    seg.head = pl.head;
    seg.first = 0;
    pair = pair_from(pair_of<kRows>(a, seg.pair), 0);
    if (pair.tiles == 0) return;
    end = pair.tiles;
  }

  for (;;) {
    seg.last = (int)min((int64_t)pair.tiles, seg.first + (end - at));
    const int sequence = a.row_tiles == 1 ? seg.pair : seg.pair / a.row_tiles;
    const int row0 = (seg.pair - sequence * a.row_tiles) * kRows, head = seg.head;
    const KVSeq s = pair.s;
    const int rows = s.n * G;
    const AttnSpan span = attn_span(a, s, row0, kRows);
    const int kbeg = span.lo + seg.first * kAttnTile, kend = min(span.hi, span.lo + seg.last * kAttnTile);

    // Operand roles.  Logits: row r16 of sub-tile `sub` is the key
    // 16 (r16 / 4) + 4 sub + r16 % 4 of the tile; then S^T's four results of
    // sub-tile `sub` in lane (r16, g) are the keys 16 g + 4 sub + 0..3.
    // ONE: blocks hold whole tiles, so a tile has one block, the same in every
    // lane; otherwise each granule of 16 keys has its own.
    const int gk = r16 >> 2;
    auto block_of = [&](int pos) {
      return pos < kend ? kv_block(a.cache, a.batch, sequence, pos >> a.block_shift) : -1;
    };
    auto cell = [&](int block) { return (int64_t)max(block, 0) * H + head; };
    const uint32_t k_lane = ((ONE ? 16 * gk : 0) + (r16 & 3)) * D + 16 * g, v_lane = r16 * BS + (ONE ? 16 * g : 0);
    uint4 kreg[4][J], vreg[DT];
    auto load_k = [&](int T, int block) {
      const uint8_t* p = a.cache.k + cell(block) * BS * D + ((T + (ONE ? 0 : 16 * gk)) & (BS - 1)) * D;
#pragma unroll
      for (int sub = 0; sub < 4; ++sub)
#pragma unroll
        for (int j = 0; j < J; ++j) kreg[sub][j] = *reinterpret_cast<const uint4*>((p + 4 * sub * D + 64 * j) + k_lane);
    };
    auto load_v = [&](int T, int block) {
      const uint8_t* p = a.cache.v + cell(block) * BS * D + ((T + (ONE ? 0 : 16 * g)) & (BS - 1));
#pragma unroll
      for (int d = 0; d < DT; ++d) vreg[d] = *reinterpret_cast<const uint4*>((p + 16 * d * BS) + v_lane);
    };
    auto uniform = [](int v) { return ONE ? __builtin_amdgcn_readfirstlane(v) : v; };

    constexpr int kStep = kWaves * kAttnTile;
    int T = kbeg + wave * kAttnTile;
    int bk = -1, bv = -1, kb = 0, vb = 0;
    auto ids = [&](int T, int& k, int& v) {
      v = block_of(ONE ? T : T + 16 * g);
      k = ONE ? v : block_of(T + 16 * gk);
    };
    int nbk, nbv;
    if (T < kend) ids(T, bk, bv);
    ids(T + kStep, nbk, nbv);
    if (T < kend) {
      bk = uniform(bk), bv = uniform(bv);
      load_k(T, bk);
      load_v(T, bv);
      kb = a.cache.k_bias[cell(bv)];
      vb = a.cache.v_bias[cell(bv)];
    }

    // this lane's rows: queries and visible keys [lo, hi)
    v8b q[RB][J][2];
    int lo[RB], hi[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int row = row0 + 16 * rb + r16;
      lo[rb] = -0x7FFFFFFF, hi[rb] = 0x7FFFFFFF;  // past the last row: anything, not stored
#pragma unroll
      for (int j = 0; j < J; ++j) q[rb][j][0] = q[rb][j][1] = v8b{};
      if (row < rows) {
        const int pos = s.start + row / G;
        hi[rb] = a.causal ? min(pos + 1, s.len) : s.len;
        if (a.window) lo[rb] = pos - a.window + 1;
        const uint16_t* qp = a.q + (int64_t)(s.first + row / G) * a.q_stride + (head * G + row % G) * D + 16 * g;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            q[rb][j][c] = __builtin_bit_cast(
                v8b, sign_queries(*reinterpret_cast<const uint4*>(qp + 64 * j + 8 * c), a.scale));
      }
    }

    v4f o[RB][DT];
    float m[RB], l[RB];
    int bref = kNoBias;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      m[rb] = kNoRef, l[rb] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[rb][d] = v4f{0, 0, 0, 0};
    }

    for (; T < kend; T += kStep) {
      // logits
      v4f sacc[RB][4];
#pragma unroll
      for (int sub = 0; sub < 4; ++sub) {
        __builtin_amdgcn_sched_barrier(0);  // widen a sub-tile at a time: registers
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) sacc[rb][sub] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const uint4 w = kreg[sub][j];
          const v8b k0 = widen_bf16<FMT>(w.x, w.y), k1 = widen_bf16<FMT>(w.z, w.w);
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) {
            sacc[rb][sub] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, q[rb][j][0], sacc[rb][sub], 0, 0, 0);
            sacc[rb][sub] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, q[rb][j][1], sacc[rb][sub], 0, 0, 0);
          }
        }
      }
      const int block = bv;
      const float kscale = key_scale(a.scale_log2, kb);
      const int vbias = block >= 0 ? vb : kNoBias;
      // the next tile's keys, and the block numbers of the one after
      const bool more = T + kStep < kend;
      if (more) {
        bk = uniform(nbk), bv = uniform(nbv);
        load_k(T + kStep, bk);
        kb = a.cache.k_bias[cell(bv)];
        vb = a.cache.v_bias[cell(bv)];
        ids(T + 2 * kStep, nbk, nbv);
      }

      bool inside = block >= 0;
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) inside = inside && T + kAttnTile <= hi[rb] && T >= lo[rb];
      const bool masked = !__all(inside);
      v8h p[RB][2];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        if (masked) {
          const int first = T + 16 * g;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (block < 0 || first + e < lo[rb] || first + e >= hi[rb]) sacc[rb][e >> 2][e & 3] = -INFINITY;
        }
        float top = sacc[rb][0][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = raw_max(top, sacc[rb][e >> 2][e & 3]);
        top = swap16_max(swap32_max(top * kscale));
        const bool move = top - m[rb] > kLazy;
        if (__any(move)) {
          const float to = move ? reference_for(top) : m[rb];
          const float f = __builtin_amdgcn_exp2f(m[rb] - to);
          m[rb] = to;
          l[rb] *= f;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[rb][d] *= f;
        }
        float t[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          t[e] = __builtin_amdgcn_exp2f(rounded(sacc[rb][e >> 2][e & 3], kscale) - m[rb]);
          l[rb] += t[e];
        }
        p[rb][0] = pack_f16(t);
        p[rb][1] = pack_f16(t + 8);
      }

      // values, at the scale of the smallest bias so far
      const int low = __builtin_amdgcn_readfirstlane(ONE ? vbias : swap16_min(swap32_min(vbias)));
      if (low < bref) {
        if (bref != kNoBias) {
          const float f = pow2_scale(low - bref);
#pragma unroll
          for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int d = 0; d < DT; ++d) o[rb][d] *= f;
        }
        bref = low;
      }
      const float vscale = pow2_scale(min(bref, 1000) - min(vbias, 1000) + kHead<FMT>);
      if (masked) clean_values<FMT, RB, DT>(vreg, o, [&](int rb, int e) {
        return !(block < 0 || T + 16 * g + e < lo[rb] || T + 16 * g + e >= hi[rb]);
      });
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        if (d % 2 == 0) __builtin_amdgcn_sched_barrier(0);
        const uint4 w = vreg[d];
        const v8h v0 = widen_f16<FMT>(w.x, w.y, vscale), v1 = widen_f16<FMT>(w.z, w.w, vscale);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          o[rb][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p[rb][0], o[rb][d], 0, 0, 0);
          o[rb][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p[rb][1], o[rb][d], 0, 0, 0);
        }
      }
      if (more) load_v(T + kStep, bv);
    }

    // the waves' results meet: row r of the workgroup, four waves in order
    const bool whole = seg.first == 0 && seg.last == pair.tiles;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (seg.first == 0);  // of a partial result
    if (a.shares && seg.first == 0 && threadIdx.x == 0)
      a.segments[(int64_t)seg.pair * H + head] =
          make_int2(blockIdx.x, (int)min((int64_t)a.shares - 1, (at + pair.tiles - 1) / share));
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      l[rb] = swap16_sum(swap32_sum(l[rb]));
      if (g == 0) {
        sm[wave][16 * rb + r16] = m[rb];
        sl[wave][16 * rb + r16] = l[rb];
      }
    }
    if (lane == 0) sb[wave] = bref;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      if (rb > 0) __syncthreads();
#pragma unroll
      for (int d = 0; d < DT; ++d) *reinterpret_cast<v4f*>(&so[wave][r16][16 * d + 4 * g]) = o[rb][d];
      __syncthreads();
      int low = sb[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) low = min(low, sb[w]);
      for (int x = threadIdx.x; x < 16 * (D / 4); x += 64 * kWaves) {
        const int r = x / (D / 4), d = 4 * (x % (D / 4));
        const int row = row0 + 16 * rb + r;
        if (row >= rows) continue;
        float top = sm[0][16 * rb + r];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sm[w][16 * rb + r]);
        float total = 0.0f;
        v4f sum{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float f = __builtin_amdgcn_exp2f(sm[w][16 * rb + r] - top);
          total += sl[w][16 * rb + r] * f;
          sum += *reinterpret_cast<const v4f*>(&so[w][r][d]) * (sb[w] == kNoBias ? 0.0f : f * pow2_scale(low - sb[w]));
        }
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum[e] = total == 0.0f ? 0.0f : __builtin_ldexpf(nan_if_infinite<FMT>(sum[e]) * inv, -(low + kHead<FMT>));
        if (whole) {
          const int64_t to = (int64_t)(s.first + row / G) * a.q_heads + head * G + row % G;
          *reinterpret_cast<uint2*>(a.out + to * D + d) =
              make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
          if (d == 0 && a.lse) a.lse[to] = row_lse(top, total);
        } else {
          const int64_t to = slot * kRows + 16 * rb + r;
          *reinterpret_cast<v4f*>(a.part_o + to * D + d) = sum;
          if (d == 0) a.part_sum[to] = make_float2(top, total);
        }
      }
    }

    // the next segment of the share
    at += seg.last - seg.first;
    if (at >= end) return;
    __syncthreads();  // LDS is free again
    seg.first = 0;
    if (++seg.head == H) {
      seg.head = 0;
      do {
        if (++seg.pair >= a.batch.batch * a.row_tiles) return;
        pair = pair_from(pair_of<kRows>(a, seg.pair), 0);
      } while (pair.tiles == 0);
    }
  }
}

template <int D, int RB>
void run(const AttnArgs& a, uint32_t groups, hipStream_t stream) {
  const dim3 grid(groups), block(64 * kWaves);
  const bool one = a.cache.block_size >= kAttnTile;
  if (a.cache.fmt == FP8_E4M3) {
    if (one) hipLaunchKernelGGL((attn_rows_kernel<D, FP8_E4M3, RB, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((attn_rows_kernel<D, FP8_E4M3, RB, false>), grid, block, 0, stream, a);
  } else {
    if (one) hipLaunchKernelGGL((attn_rows_kernel<D, FP8_E5M2, RB, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((attn_rows_kernel<D, FP8_E5M2, RB, false>), grid, block, 0, stream, a);
  }
}

}  // namespace

int attn_rows_resident(int head_dim, int row_blocks) {
  const int d = head_dim * row_blocks;
  return 256 * (d >= 256 ? kOcc<256, 1> : (d == 128 ? kOcc<128, 1> : kOcc<64, 1>));
}

hipError_t launch_attn_rows(const AttnArgs& a, int row_blocks, uint32_t groups, hipStream_t stream) {
  const int D = a.cache.head_dim;
  if (D == 256) run<256, 1>(a, groups, stream);
  else if (D == 128 && row_blocks == 1) run<128, 1>(a, groups, stream);
  else if (D == 128) run<128, 2>(a, groups, stream);
  else if (row_blocks == 1) run<64, 1>(a, groups, stream);
  else run<64, 2>(a, groups, stream);
  return hipGetLastError();
}

}  // namespace fp8lin
