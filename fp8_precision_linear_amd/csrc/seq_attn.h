// Attention over packed sequences, for training: what its forward and backward
// kernels share (include/fp8lin_train.h has the definitions).
//
//   s = scale q.k,  p = e^(s - lse),  out = sum_j p_j v_j
//   dp = dout.v,  delta = rowsum(dout * out),  ds = p (dp - delta)
//   dv_j = sum_q p dout,  dk_j = scale sum_q ds q,  dq = scale sum_j ds k_j
//
// Products run on the 32x32x16 bf16 MFMA (fp32 sums).  In its result a lane owns
// one column and, of every eight rows, the four of its half of the wave.  The
// first products put the axis that the second ones sum over on the rows, so
// that what a lane holds is the second product's B operand as it lies: slot e of
// step c of a lane of half h is row 16 c + 8 (e / 4) + 4 h + e % 4, and the
// other operand is read from LDS in the same order.
//
// Tiles lie in LDS as they do in memory, row by row, 16-byte chunks swizzled.
// The same tile is read by rows (16 bytes of a row a lane) and by columns (four
// rows of a column a lane, with the transposing LDS read), so that nothing is
// transposed on the way in or held twice.
#pragma once

#include "attn_common.h"
#include "lds_dma.h"
#include "quotient.h"

namespace fp8lin {

constexpr int kSeqRows = 128;  // query rows of a workgroup (forward, dq), and keys (dk, dv)

// A tile of kSeqRows keys, or rows: where its walk over the queries starts on the
// head's line of key tiles and its walk over the keys on that of row tiles; its
// sequence's first row and length, and its own first position.
struct SeqLine {
  int64_t start, start_q;
  int first, n, k0;
  int count;  // of the line's end: the tiles' number
};

struct SeqAttnArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* cu;
  int batch, tokens, max_len;
  int q_heads, heads, group;
  float scale, scale_log2;  // scale * log2(e)
  int causal, window;
  int tiles;       // most row (key) tiles of any sequence
  int rest;        // places of tiles past their sequences' first (ragged_places), or 0
  uint32_t first;  // this launch's first workgroup
  // forward: written; backward: read
  uint16_t* out;
  float* lse;
  // backward
  const uint16_t* dout;
  int64_t dout_stride, dq_stride, dk_stride, dv_stride;
  uint16_t *dq, *dk, *dv;
  float *lse2, *delta;  // [q_heads][tokens], lse * log2(e) and rowsum(dout * out)
  // sums of walks that are cut: [workgroups of that kind][2][kSeqRows][D]
  float *part_k, *part_v, *part_q;
  SeqLine *line, *line_end;  // tiles of a head; the lines' lengths, and the tiles' number
  int most_tiles;  // of `line`
  int shares, row_shares;  // of a head's line of key tiles, of row tiles; 0: a workgroup takes a tile
  uint32_t dkv_groups;  // workgroups of dk and dv, each
  uint32_t dq_first;    // workgroups of dq, where they come first, or 0
};

namespace {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef int v4i32 __attribute__((ext_vector_type(4)));

struct Seq {
  int first, n;
};
__device__ __forceinline__ Seq seq_of(const SeqAttnArgs& a, int i) {
  const int first = max(0, min(a.cu[i], a.tokens));
  const int end = max(first, min(a.cu[i + 1], a.tokens));
  return {__builtin_amdgcn_readfirstlane(first), __builtin_amdgcn_readfirstlane(min(end - first, a.max_len))};
}

// A workgroup for each tile that a sequence may have: were every sequence the
// longest, tiles * batch; of one long and many short ones, or with a loose bound,
// most of these have no rows, and each costs some 0.6 ns.  There are no more than
// tokens / 128 tiles beside the sequences' first ones, so where that leaves an
// eighth of the places a sequence's first tile has the place of its number, and the
// others are counted through in order.  4096 tokens and 1000 sequences of 64, 32
// heads of 128: forward 1222 -> 728 us, backward 4083 -> 2116; where it leaves a
// quarter (1024 tokens and 16 sequences of 100), 36 -> 38 and 93 -> 104.
inline int ragged_places(int tokens, int batch, int tiles) {
  const int64_t rest = tokens / kSeqRows;
  return 8 * (batch + rest) <= (int64_t)tiles * batch ? (int)rest : 0;
}

// A sequence's number and its tile's, or -1.
struct NthTile {
  int seq, tile;
};
// The r-th of the tiles that are not the first of their sequence.  Each wave looks
// at the lengths of 512 sequences at a time, eight a lane.
__device__ __forceinline__ NthTile nth_tile(const SeqAttnArgs& a, int r) {
  constexpr int kEach = 8;
  const int lane = threadIdx.x & 63;
  for (int i0 = 0; i0 < a.batch; i0 += 64 * kEach) {
    int end[kEach + 1], more[kEach], mine = 0;
#pragma unroll
    for (int e = 0; e <= kEach; ++e) end[e] = max(0, min(a.cu[min(i0 + lane * kEach + e, a.batch)], a.tokens));
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      more[e] = max(0, (min(end[e + 1] - end[e], a.max_len) - 1) / kSeqRows);  // (none past the last sequence)
      mine += more[e];
    }
    int upto = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(upto, off, 64);
      if (lane >= off) upto += o;
    }
    const uint64_t past = __ballot(upto > r);
    if (past != 0) {
      const int owner = __builtin_ctzll(past);
      int left = r - (upto - mine), e = 0;
#pragma unroll
      for (int c = 0; c + 1 < kEach; ++c)
        if (e == c && left >= more[c]) left -= more[c], ++e;
      return {__builtin_amdgcn_readlane(i0 + lane * kEach + e, owner), __builtin_amdgcn_readlane(left, owner) + 1};
    }
    r -= __builtin_amdgcn_readlane(upto, 63);
  }
  return {-1, 0};
}

// The swizzle of a tile of rows of D bf16: 16-byte chunk c of row r lies at
// c ^ swz(r).  Sixteen consecutive rows read at the same chunk, and four
// consecutive rows read at the same four chunks, each meet every bank once.
template <int D>
__device__ __forceinline__ int swz(int r) {
  if constexpr (D == 64) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  else return ((r & 3) << 2) | ((r >> 2) & 3);
}

__device__ __forceinline__ v8b lds_row(uint32_t at) {
  return *(__attribute__((address_space(3))) const v8b*)(uintptr_t)at;
}
__device__ __forceinline__ v4s lds_column(uint32_t at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(uintptr_t)at);
}

// A lane's place in a tile for reads by rows: row r32 of 32, 16-byte step j at
// (place ^ 32 j), the next 32 rows 64 D on.
template <int D>
__device__ __forceinline__ uint32_t row_place(int lane) {
  const int r = lane & 31;
  return r * 2 * D + (((lane >> 5) ^ swz<D>(r)) << 4);
}
// For reads by columns: column 32 d + r32, slots 0-3 of a step of 16 rows at
// (place ^ 64 d), 4-7 at (place ^ 64 d ^ 32) + 16 D, the next step 32 D on.
template <int D>
__device__ __forceinline__ uint32_t column_place(int lane) {
  const int r = 4 * (lane >> 5) + ((lane >> 2) & 3);
  return r * 2 * D + (((2 * ((lane >> 4) & 1) + ((lane >> 1) & 1)) ^ swz<D>(r)) << 4) + 8 * (lane & 1);
}
template <int D>
__device__ __forceinline__ v8b column_step(uint32_t place, int d) {
  const v4s a = lds_column(place ^ (64 * d)), b = lds_column((place ^ (64 * d) ^ 32) + 16 * D);
  return __builtin_bit_cast(v8b, v8s{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}

// DMA of ROWS rows of D bf16 by WAVES waves; rows past the last are the last one
// again (whoever reads them masks them).
template <int D, int ROWS, int WAVES = 4>
struct TileLoad {
  static constexpr int kBytes = ROWS * D * 2;
  static constexpr int kLoads = kBytes / (1024 * WAVES);  // of each wave
  static constexpr int kStep = 512 * WAVES / D;           // rows between a wave's loads
  // loads whose rows are swizzled differently (alike: sixteen rows apart)
  static constexpr int kKinds = kStep % 16 == 0 ? 1 : 16 / kStep;
  uint32_t offset[kKinds];
  static __device__ __forceinline__ uint32_t row_of(int lane, int wave) { return wave * (512 / D) + lane / (D / 8); }
  static __device__ __forceinline__ uint32_t chunk_of(int lane, uint32_t row) {
    return ((lane % (D / 8)) ^ swz<D>(row)) * 16;
  }
  __device__ __forceinline__ TileLoad(int lane, int wave, uint32_t stride_bytes) {
    const uint32_t row = row_of(lane, wave);
#pragma unroll
    for (int p = 0; p < kKinds; ++p) offset[p] = row * stride_bytes + chunk_of(lane, row + p * kStep);
  }
  // base: row 0 of the tile; left: rows there are (at least one)
  __device__ __forceinline__ void issue(const uint16_t* base, int64_t stride_bytes, int left, uint32_t lds,
                                        int wave) const {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(base);
    if (left >= ROWS) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        dma16(p + (int64_t)(i * kStep) * stride_bytes, offset[i % kKinds], lds + (wave + WAVES * i) * 1024);
    } else {
      const int lane = threadIdx.x & 63;
      const uint32_t row = row_of(lane, wave);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t r = min((int)row + i * kStep, left - 1);
        dma16(p, r * (uint32_t)stride_bytes + chunk_of(lane, row + (i % kKinds) * kStep), lds + (wave + WAVES * i) * 1024);
      }
    }
  }
};

__device__ __forceinline__ v16f zero16() {
  v16f r;
#pragma unroll
  for (int e = 0; e < 16; ++e) r[e] = 0.0f;
  return r;
}
__device__ __forceinline__ v16f mma(v8b a, v8b b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 0xFFFF in every half of w whose bf16 value is NaN or infinite.
__device__ __forceinline__ uint32_t bad_halves(uint32_t w) {
  return ((w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}
__device__ __forceinline__ v4i32 bad_of(v8b f) {
  v4i32 w = __builtin_bit_cast(v4i32, f);
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = (int)bad_halves((uint32_t)w[e]);
  return w;
}

// A tile that some column does not see whole is multiplied with zeros where it
// is not seen, and 0 * NaN must not reach a result.  So such tiles are searched
// for NaN and infinities (has_bad: whether any wave found one; the workgroup's
// waves call it together), and what is found is cleared in LDS (clear_bad) once
// those that do see it have it on record.
// GROUPS sets of WAVES waves have a tile each, the last ones perhaps none (`there`).
template <int BYTES, int GROUPS = 1, int WAVES = 4>
__device__ __forceinline__ bool has_bad(uint32_t tile, int* found, bool there = true) {
  uint32_t bad = 0;
  const uint32_t mine = tile + (threadIdx.x % (64 * WAVES)) * 16;
#pragma unroll
  for (int i = 0; i < BYTES; i += 1024 * WAVES) {
    const v4i32 w = bad_of(lds_row(mine + i));
    bad |= (uint32_t)(w[0] | w[1] | w[2] | w[3]);
  }
  const bool any = __any(bad != 0) && there;
  if ((threadIdx.x & 63) == 0) found[threadIdx.x >> 6] = any;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < WAVES * GROUPS; ++w) all |= found[w];
  return all != 0;
}
// rows: where given, set to 1 for each row of `row_bytes` that held one.
template <int BYTES, int WAVES = 4>
__device__ __forceinline__ void clear_bad(uint32_t tile, int row_bytes, int* rows) {
  __syncthreads();  // every wave is done with the tile as it was
  for (int i = (threadIdx.x % (64 * WAVES)) * 16; i < BYTES; i += 1024 * WAVES) {
    v4i32 w = __builtin_bit_cast(v4i32, lds_row(tile + i));
    const v4i32 bad = bad_of(__builtin_bit_cast(v8b, w));
    w &= ~bad;
    *(__attribute__((address_space(3))) v4i32*)(uintptr_t)(tile + i) = w;
    if (rows && (bad[0] | bad[1] | bad[2] | bad[3])) rows[i / row_bytes] = 1;
  }
  __syncthreads();
}

// Step c of a result's 16 values as the next product's operand, in bf16.
__device__ __forceinline__ v8b operand(const v16f& s, int c) {
  v2b r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = __builtin_convertvector((v2f{s[8 * c + 2 * e], s[8 * c + 2 * e + 1]}), v2b);
  return v8b{r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
}
// Row of a 32-row result that value e of a lane of half h is.
__device__ __forceinline__ int result_row(int e, int h) { return 8 * (e >> 2) + 4 * h + (e & 3); }

// NaN for an infinite value (include/fp8lin_train.h).
__device__ __forceinline__ float finite_or_nan(float v) { return v + (v - v); }

}  // namespace

struct SeqAttnShape {
  int batch, tokens, max_len, q_heads, heads, head_dim;
};
hipError_t launch_seq_attn_fwd(SeqAttnArgs a, int head_dim, hipStream_t stream);
int64_t seq_attn_bwd_workspace_bytes(const SeqAttnShape& s);
hipError_t launch_seq_attn_bwd(SeqAttnArgs a, int head_dim, void* ws, hipStream_t stream);

}  // namespace fp8lin
