// Attention of many query rows (prompts, chunks of them) over the paged FP8
// cache: attn_common.h has the mathematics.
//
// MFMA- and VALU-bound: two prompts of 1777 to 2048 tokens on 1500 to 2048
// cached, 64 heads of 128 on 8: 312 GFLOP in 333-354 us, 880-940 TFLOP/s, where
// a large bf16 product of a library reaches 1205 and converts nothing.  Heads of
// 256 leave one wave a SIMD (the output alone takes 128 registers), which then
// waits out what two would overlap.
//
// A workgroup of four waves takes 128 rows (token, head
// of the group) of one sequence and key head; each wave owns 32 of them on the
// 32x32x16 MFMA and keeps its queries, logits and O in registers.  Tiles of 64
// keys and values go through LDS by DMA, as codes, in a ring of four, one
// barrier a tile.  Each wave widens the codes it reads (half the LDS bytes that
// widened tiles would cost).
//
// LDS, 16-byte chunks swizzled so that the 16 lanes of a read address 16
// different bank groups (64 banks): keys [64][D], chunk c of row r at
// c ^ fk(r); values [D][64], chunk c of row d at c ^ ((d >> 2) & 3).  The DMA
// writes LDS linearly, so the swizzle sits in the lanes' source addresses.
#include "attn_common.h"
#include "lds_dma.h"

namespace fp8lin {
namespace {

constexpr int kWaves = kAttnWaves;
// Tiles in LDS: three on their way while one is consumed.  (With one on its way
// short prompts, whose workgroups have a CU to themselves, waited for every
// tile: 740 tokens of 40 heads took 102 us.)
constexpr int kRing = 4;
// Tiles whose block numbers and biases are held in LDS at a time.  The main
// loop then asks nothing of memory but tiles, whose arrival it counts.
constexpr int kStretch = 64;
// A lane's 32 probabilities of a tile may add up to this before its row's
// reference moves: 32 keys level with the maximum that set it (2^kShift each)
// stay below, and none can pass fp16's range.
constexpr float kMostPart = 32768.0f;
// References from here on have their logits rounded (attn_common.h).
constexpr float kHuge = 0x1p22f;

// Bits of a key row that tell apart the rows 16 lanes of a fragment read
// ({0..7, 16..23} or {8..15, 24..31} of 32) and share a bank window.
template <int D>
__device__ __forceinline__ int fk(int r) {
  if constexpr (D == 64) return ((r >> 2) & 1) | (((r >> 4) & 1) << 1);
  else if constexpr (D == 128) return ((r >> 1) & 3) | (((r >> 4) & 1) << 2);
  else return (r & 7) | (((r >> 4) & 1) << 3);
}

typedef int v4i __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v4i lds_read16(uint32_t at) {
  return *(__attribute__((address_space(3))) const v4i*)(uintptr_t)at;
}

__device__ __forceinline__ void lds_write16(uint32_t at, v4i v) {
  *(__attribute__((address_space(3))) v4i*)(uintptr_t)at = v;
}

// ONE: blocks hold whole tiles, so a tile has one block; otherwise each of its
// four granules of 16 keys has its own.
template <int D, int FMT, bool ONE>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void attn_tile_kernel(AttnArgs a) {
  constexpr int NB = ONE ? 1 : 4;
  constexpr int J = D / 32;   // 32-dimension steps of the logits
  constexpr int DT = D / 32;  // 32-dimension tiles of the output
  constexpr int kTileBytes = kAttnTile * D;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kRing][2][kTileBytes];  // [buffer][keys, values]
  __shared__ __attribute__((aligned(16))) int table[3][kStretch * NB];  // blocks, key biases, value biases
  __shared__ int found[kWaves];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  const AttnPlace at = attn_place(a);
  const int BS = a.cache.block_size, H = a.cache.heads, G = a.group;
  const KVSeq s = kv_seq_uniform(a.batch, BS, at.seq);
  const int rows = s.n * G, row0 = at.row_tile * kAttnTileRows;
  if (row0 >= rows || !attn_serves(a, s)) return;
  const AttnSpan span = attn_span(a, s, row0, kAttnTileRows);
  if (at.split >= span.chunks) return;
  const int kbeg = span.lo + at.split * a.chunk, kend = min(span.hi, kbeg + a.chunk);

  const int row = row0 + 32 * wave + r32;
  const bool stored = row < rows;
  int lo = -0x7FFFFFFF, hi = 0x7FFFFFFF;  // past the last row: anything, not stored
  v8b q[J][2];
#pragma unroll
  for (int j = 0; j < J; ++j) q[j][0] = q[j][1] = v8b{};
  if (stored) {
    const int pos = s.start + row / G;
    hi = a.causal ? min(pos + 1, s.len) : s.len;
    if (a.window) lo = pos - a.window + 1;
    const uint16_t* qp = a.q + (int64_t)(s.first + row / G) * a.q_stride + (at.head * G + row % G) * D + 16 * h;
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        q[j][c] = __builtin_bit_cast(v8b, sign_queries(*reinterpret_cast<const uint4*>(qp + 32 * j + 8 * c), a.scale));
    }
  }
  // the wave's keys: none past the last of its rows' or before the first's
  const int wrow0 = row0 + 32 * wave, wrow1 = min(wrow0 + 32, rows) - 1;
  const bool idle = wrow0 >= rows;
  const int whi = idle ? 0 : (a.causal ? min(s.len, s.start + wrow1 / G + 1) : s.len);
  const int wlo = a.window ? s.start + wrow0 / G - a.window + 1 : 0;

  // the keys that every row of the workgroup sees
  const int row_last = min(row0 + kAttnTileRows, rows) - 1;
  const int all_hi = a.causal ? min(s.len, s.start + row0 / G + 1) : s.len;
  const int all_lo = a.window ? s.start + row_last / G - a.window + 1 : 0;

  v16f o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
  float m = kNoRef, l = 0.0f;
  bool huge = false;  // some row's reference passes kHuge
  int bref = kNoBias;

  // blocks and biases of a tile, scalars
  struct Blocks {
    int b[NB];
  };
  struct Biases {
    int k[NB], v[NB];
  };
  auto scalar = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  // granule g's entry
  auto pick = [](const int (&v)[NB], int g) {
    if constexpr (ONE) return v[0];
    else return g < 2 ? (g == 0 ? v[0] : v[1]) : (g == 2 ? v[2] : v[3]);
  };
  const int tiles = (kend - kbeg + kAttnTile - 1) / kAttnTile;
  auto fill = [&](int first) {  // the table for tiles [first, first + kStretch)
    if ((int)threadIdx.x < kStretch * NB) {
      const int pos = kbeg + first * kAttnTile + (int)threadIdx.x * (kAttnTile / NB);
      const int block = pos < kend ? kv_block(a.cache, a.batch, at.seq, pos >> a.block_shift) : -1;
      const int64_t c = (int64_t)max(block, 0) * H + at.head;
      table[0][threadIdx.x] = block;
      table[1][threadIdx.x] = a.cache.k_bias[c];
      table[2][threadIdx.x] = a.cache.v_bias[c];
    }
  };
  auto entry = [&](int (&to)[NB], int which, int t) {
    int v[NB];
#pragma unroll
    for (int g = 0; g < NB; ++g) v[g] = table[which][t * NB + g];
#pragma unroll
    for (int g = 0; g < NB; ++g) to[g] = scalar(v[g]);
  };
  const uint32_t ring0 = lds_addr(ring);
  // This wave's quarter of a tile's keys (values), D / 64 KB: KB i holds key rows
  // (dimensions) 4 i KBs past the first's, whose swizzle is the same -- but for
  // D = 256, where every other i is 16 rows on, in the other half of fk.
  const int kr = wave * (1024 / D) + lane / (D / 16), kc = (lane % (D / 16)) ^ fk<D>(kr);
  const int vd = wave * 16 + lane / 4, vc = (lane & 3) ^ ((vd >> 2) & 3);
  const uint32_t k_lane = kr * D + 16 * kc, v_lane = vd * BS + 16 * vc;
  auto issue_k = [&](int T, const Blocks& b, int buf) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint32_t to = ring0 + buf * 2 * kTileBytes + (wave + kWaves * i) * 1024;
      const int turn = D == 256 && (i & 1) ? 8 : 0;
      if constexpr (ONE) {
        const int64_t cell = (int64_t)max(b.b[0], 0) * H + at.head;
        dma16(a.cache.k + (cell * BS + (T & (BS - 1)) + 4096 / D * i) * D, k_lane ^ (16 * turn), to);
      } else {
        const int r = kr + 4096 / D * i;
        const int64_t cell = (int64_t)max(pick(b.b, r >> 4), 0) * H + at.head;
        dma16(a.cache.k + (cell * BS + ((T + r) & (BS - 1))) * D + 16 * (kc ^ turn), to);
      }
    }
  };
  auto issue_v = [&](int T, const Blocks& b, int buf) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint32_t to = ring0 + (2 * buf + 1) * kTileBytes + (wave + kWaves * i) * 1024;
      if constexpr (ONE) {
        const int64_t cell = (int64_t)max(b.b[0], 0) * H + at.head;
        dma16(a.cache.v + (cell * D + 64 * i) * BS + (T & (BS - 1)), v_lane, to);
      } else {
        const int64_t cell = (int64_t)max(pick(b.b, vc), 0) * H + at.head;
        dma16(a.cache.v + (cell * D + vd + 64 * i) * BS + ((T + 16 * vc) & (BS - 1)), to);
      }
    }
  };

  // Operand roles.  Row r32 of sub-tile `sub` (32 keys) of S^T's A operand is
  // key 16 ((r32 >> 2) & 1) + 4 (r32 >> 3) + (r32 & 3): S^T's result v of a
  // lane is then key 32 sub + 16 h + v.
  const int krow = 16 * ((r32 >> 2) & 1) + 4 * (r32 >> 3) + (r32 & 3);
  // chunk 2 j + h of its row, and chunk 2 sub + h: the swizzle is an XOR, so j
  // and sub are too
  const uint32_t kfrag = krow * D + ((h ^ fk<D>(krow)) << 4);
  const uint32_t vfrag = kTileBytes + r32 * 64 + ((h ^ ((r32 >> 2) & 3)) << 4);

  // No code of a slot that a row does not see may turn 0 * code into NaN.  So a
  // tile that some row of the workgroup does not see whole is searched for NaN
  // (and infinity) codes of values; if it holds any, the outputs of the rows
  // that do see them become NaN -- counted by a product of visibility with "is
  // bad" -- and then the codes become zeros, in LDS, for every wave.
  auto clean = [&](int T, uint32_t values, const Blocks& blocks) {
    uint32_t bad = 0;
    const uint32_t mine = values + threadIdx.x * (kTileBytes / (64 * kWaves));
#pragma unroll
    for (int i = 0; i < kTileBytes / (64 * kWaves); i += 16) {
      const v4i w = lds_read16(mine + i);
      bad |= bad_bytes<FMT>(w[0]) | bad_bytes<FMT>(w[1]) | bad_bytes<FMT>(w[2]) | bad_bytes<FMT>(w[3]);
    }
    const bool any = __any(bad != 0);
    if (lane == 0) found[wave] = any;
    __syncthreads();
    if (found[0] | found[1] | found[2] | found[3]) {
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const bool there = (h ? pick(blocks.b, 2 * sub + 1) : pick(blocks.b, 2 * sub)) >= 0;
        v8h see[2];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int key = T + 32 * sub + 16 * h + e;
          see[e >> 3][e & 7] = there && key >= lo && key < hi ? (_Float16)1.0f : (_Float16)0.0f;
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          __builtin_amdgcn_sched_barrier(0);
          const v4i w = lds_read16(((values - kTileBytes + vfrag) ^ (32 * sub)) + d * 32 * 64);
          v16f n;
#pragma unroll
          for (int e = 0; e < 16; ++e) n[e] = 0.0f;
          n = __builtin_amdgcn_mfma_f32_32x32x16_f16(ones_f16(bad_bytes<FMT>(w[0]), bad_bytes<FMT>(w[1])), see[0], n, 0,
                                                     0, 0);
          n = __builtin_amdgcn_mfma_f32_32x32x16_f16(ones_f16(bad_bytes<FMT>(w[2]), bad_bytes<FMT>(w[3])), see[1], n, 0,
                                                     0, 0);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[d][e] = n[e] > 0.0f ? NAN : o[d][e];
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kTileBytes / (64 * kWaves); i += 16) {
        v4i w = lds_read16(mine + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] &= ~bad_bytes<FMT>(w[e]);
        lds_write16(mine + i, w);
      }
    }
    __syncthreads();
  };

  // O and l times f, O at the value bias `low` (O is zero before the first one)
  auto rescale = [&](float f, int low) {
    l *= f;
    const float fo = f * pow2_scale(low - bref);
    bref = low;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] *= fo;
  };
  auto join = [](const v2h* p) {
    return v8h{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
  };

  // one tile for this wave's rows; masked: some row does not see all of it
  auto consume = [&](bool masked, int T, uint32_t tile, const Blocks& blocks, const Biases& bias) {
    auto seen = [&](int sub, int e) {
      const int key = T + 32 * sub + 16 * h + e;
      return (h ? pick(blocks.b, 2 * sub + 1) : pick(blocks.b, 2 * sub)) >= 0 && key >= lo && key < hi;
    };
    // LDS reads well ahead of their use: all keys before the first product, all
    // values before the probabilities (each wait on a read costs more than the
    // product it feeds)
    v4i kw[J][2], vw[2][DT];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) kw[j][sub] = lds_read16(((tile + kfrag) ^ (32 * j)) + sub * 32 * D);
    __builtin_amdgcn_sched_barrier(0);
    // the wave in a product goes first: its widening feeds the matrix core while
    // the SIMD's other wave forms probabilities (prompts 426 -> 406 us)
    __builtin_amdgcn_s_setprio(1);
    v16f sacc[2];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
      for (int e = 0; e < 16; ++e) sacc[sub][e] = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
          sacc[sub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_bf16<FMT>(kw[j][sub][2 * c], kw[j][sub][2 * c + 1]),
                                                              q[j][c], sacc[sub], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
      for (int d = 0; d < DT; ++d) vw[sub][d] = lds_read16(((tile + vfrag) ^ (32 * sub)) + d * 32 * 64);
    __builtin_amdgcn_sched_barrier(0);
    if (masked) {
      asm volatile("");  // a branch: as selects it would cost every tile
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int e = 0; e < 16; ++e) sacc[sub][e] = seen(sub, e) ? sacc[sub][e] : -INFINITY;
    }
    int low = bref;
#pragma unroll
    for (int g = 0; g < NB; ++g) low = blocks.b[g] < 0 ? low : min(low, bias.v[g]);
    if (low < bref) rescale(1.0f, low);
    float kscale[2], vscale[2];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      kscale[sub] = key_scale(a.scale_log2, h ? pick(bias.k, 2 * sub + 1) : pick(bias.k, 2 * sub));
      // (a missing granule's bias is block 0's: anything)
      vscale[sub] = pow2_scale(min(0, bref - (h ? pick(bias.v, 2 * sub + 1) : pick(bias.v, 2 * sub))) + kHead<FMT>);
    }
    // (as a branch of its own, and a rare one: rounding every product costs 5% of
    // the kernel, laying the branch out as an ordinary one 3% for heads of 256)
    auto round_logits = [&] {
      asm volatile("");
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
#pragma unroll
        for (int e = 0; e < 16; ++e) sacc[sub][e] = rounded(sacc[sub][e], kscale[sub]);
        kscale[sub] = 1.0f;
      }
    };
    if (__builtin_expect(huge, 0)) round_logits();
    // Probabilities against the reference as it is; their sum tells whether a
    // logit has outgrown it (it always has in a row's first tile), and only
    // then are the maxima taken and the tile done again.
    v2h p[2][8];
    float part;
    auto probabilities = [&] {
      part = 0.0f;
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v2f t;
#pragma unroll
          for (int c = 0; c < 2; ++c)
            t[c] = __builtin_amdgcn_exp2f(fmaf(sacc[sub][2 * e + c], kscale[sub], -m));
          p[sub][e] = __builtin_convertvector(t, v2h);
          part += t[0];  // of the fp32 values: the sum is held to fp32's precision
          part += t[1];
        }
    };
    probabilities();
    if (__any(!(part <= kMostPart))) {
      float top = -INFINITY;
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        float s = sacc[sub][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) s = raw_max(s, sacc[sub][e]);
        top = fmaxf(top, s * kscale[sub]);
      }
      top = swap32_max(top);
      const float up = reference_for(top), to = up > m ? up : m;
      const float f = __builtin_amdgcn_exp2f(m - to);
      m = to;
      rescale(f, bref);
      if (__any(fabsf(m) > kHuge && m != kNoRef)) {
        huge = true;
        round_logits();
      }
      probabilities();
    }
    l += part;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const v8h pc = join(p[sub] + 4 * c);
#pragma unroll
        for (int d = 0; d < DT; ++d)
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
              widen_f16<FMT>(vw[sub][d][2 * c], vw[sub][d][2 * c + 1], vscale[sub]), pc, o[d], 0, 0, 0);
      }
    __builtin_amdgcn_s_setprio(0);
  };

  static_assert(kStretch * 4 <= 64 * kWaves, "one table entry a lane");
  constexpr int kLoads = 2 * (D / 64);  // this wave's DMA loads a tile
  for (int first = 0; first < tiles; first += kStretch) {
    if (first) __syncthreads();  // every wave is done with the table and the ring
    fill(first);
    __syncthreads();
    const int n = min(kStretch, tiles - first), T0 = kbeg + first * kAttnTile;
    Blocks ahead;
    for (int t = 0; t < kRing - 1; ++t)
      if (t < n) {
        entry(ahead.b, 0, t);
        issue_k(T0 + t * kAttnTile, ahead, t);
        issue_v(T0 + t * kAttnTile, ahead, t);
      }
    for (int t = 0; t < n; ++t) {
      const int T = T0 + t * kAttnTile, buf = t & (kRing - 1);
      Blocks blocks;
      Biases bias;
      entry(blocks.b, 0, t);
      entry(bias.k, 1, t);
      entry(bias.v, 2, t);
      const bool more = t + kRing - 1 < n;
      if (more) entry(ahead.b, 0, t + kRing - 1);
      wait_stages<kLoads>(min(kRing - 2, n - 1 - t));
      bare_barrier();  // this tile is whole, and every wave is done with the one before
      if (more) {
        issue_k(T + (kRing - 1) * kAttnTile, ahead, (buf + kRing - 1) & (kRing - 1));
        issue_v(T + (kRing - 1) * kAttnTile, ahead, (buf + kRing - 1) & (kRing - 1));
      }
      const uint32_t tile = ring0 + buf * 2 * kTileBytes;
      bool there = true;
#pragma unroll
      for (int g = 0; g < NB; ++g) there = there && blocks.b[g] >= 0;
      if (!there || T + kAttnTile > all_hi || T < all_lo) clean(T, tile + kTileBytes, blocks);
      if (T >= whi || T + kAttnTile <= wlo) continue;  // nothing for this wave's rows
      const bool whole = there && T + kAttnTile <= hi && T >= lo;
      consume(!__all(whole), T, tile, blocks, bias);
    }
  }

  l = swap32_sum(l);
  if (!stored) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t cell = (int64_t)(s.first + row / G) * a.q_heads + at.head * G + row % G;
  const int64_t slot = (int64_t)at.split * a.batch.tokens * a.q_heads + cell;
  // result v of a lane is dimension 32 d + 8 (v / 4) + 4 h + v % 4
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = l == 0.0f ? 0.0f : __builtin_ldexpf(nan_if_infinite<FMT>(o[d][4 * u + e]) * inv, -(bref + kHead<FMT>));
      const int at_d = 32 * d + 8 * u + 4 * h;
      if (span.chunks == 1)
        *reinterpret_cast<uint2*>(a.out + cell * D + at_d) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      else
        *reinterpret_cast<v4f*>(a.part_o + slot * D + at_d) = v4f{v[0], v[1], v[2], v[3]};
    }
  if (h == 0) {
    if (span.chunks > 1) a.part_sum[slot] = make_float2(m, l);
    else if (a.lse) a.lse[cell] = row_lse(m, l);
  }
}

template <int D>
void run(const AttnArgs& a, uint32_t groups, hipStream_t stream) {
  const dim3 grid(groups), block(64 * kWaves);
  const bool one = a.cache.block_size >= kAttnTile;
  if (a.cache.fmt == FP8_E4M3) {
    if (one) hipLaunchKernelGGL((attn_tile_kernel<D, FP8_E4M3, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((attn_tile_kernel<D, FP8_E4M3, false>), grid, block, 0, stream, a);
  } else {
    if (one) hipLaunchKernelGGL((attn_tile_kernel<D, FP8_E5M2, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((attn_tile_kernel<D, FP8_E5M2, false>), grid, block, 0, stream, a);
  }
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs& a, uint32_t groups, hipStream_t stream) {
  if (a.cache.head_dim == 64) run<64>(a, groups, stream);
  else if (a.cache.head_dim == 128) run<128>(a, groups, stream);
  else run<256>(a, groups, stream);
  return hipGetLastError();
}

}  // namespace fp8lin
