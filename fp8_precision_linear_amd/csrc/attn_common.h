// What the attention kernels over the paged FP8 cache share.
//
//   t_j = scale * log2(e) * 2^-kb * (q . k8_j)          logits in base 2
//   p_j = 2^(t_j - m)          m: running reference of the row
//   l = sum p_j,  O = sum p_j v8_j 2^-vb,  out = O / l,  lse = ln 2 (m + log2 l)
//
// kb, vb: the key and value bias of token j's block and head.  Blocks hold a
// multiple of 16 tokens, so a "granule" of 16 aligned tokens has one block and
// one bias of each kind.
//
// Products.  S^T = K Q^T and O^T = V^T P^T, so that a lane owns one query row
// from the logits to the output: its row statistics need one or two cross-lane
// steps, and the probabilities it holds are already the B operand of the
// second product.  Which token a row of S^T's A operand stands for, and which
// dimension a slot of its contraction, is free as long as both operands agree:
// they are chosen so that every lane's A operand of either product is 16
// consecutive bytes of the cache (a token's 16 dimensions of K; a dimension's
// 16 tokens of V, which the cache holds transposed).  Nothing is shuffled or
// transposed on the way.
//
// Arithmetic.  Keys widen exactly to bf16, the queries' type; products and
// sums of the 16-bit MFMA are fp32.  Values widen to fp16, scaled by
// 2^(bref - vb + kHead) in the conversion itself, where bref is the smallest
// value bias met so far (O is rescaled when it drops): the largest values sit
// at the top of fp16's range, so a value loses only what lies 2^40 below them.
// Probabilities are fp16 scaled by 2^kShift relative to the reference: 11 bits
// down to 2^-22 of the largest, against bf16's 8 bits.  The reference follows
// the row maximum lazily: it moves only when a logit exceeds it by more than
// kLazy, so that most tiles rescale nothing and p, at most 2^15, stays in range.
//
// Where logits are huge, s * kscale is rounded before the reference is
// subtracted, as it was for the maximum that set the reference: fused into one
// operation its rounding error alone, 2^-24 of the logit, would drive the
// largest p out of fp16's range from 2^26 on.  The reference itself is a number
// of the logits' size, in steps of 16 from 2^27 on: logits are compared with it
// by their difference, which is exact, and it lies at most kShift below the
// maximum (reference_for).
#pragma once

#include <type_traits>

#include "kv_device.h"

namespace fp8lin {

struct AttnArgs {
  fp8_kv_cache_t cache;
  fp8_kv_batch_t batch;
  const uint16_t* q;
  int64_t q_stride;
  int q_heads;
  int group;        // query heads per key head
  int block_shift;  // log2 of the block size
  float scale;       // its sign, and zero
  float scale_log2;  // |scale| * log2(e), 1 for a scale of zero
  int causal, window;
  uint16_t* out;
  float* lse;
  float* part_o;    // [splits][tokens][q_heads][D], normalised
  float2* part_sum;  // [splits][tokens][q_heads], reference and sum
  int chunk;        // tile kernel: keys per split, a multiple of kAttnTile
  int splits;       // tile kernel: most chunks of any row tile
  int row_tiles;    // most row tiles of any sequence
  uint32_t first;   // this launch's first workgroup
  int least, most;  // rows of a key head that a sequence has to have to be served
  int shares;       // rows kernel: workgroups that share all keys evenly, or 0
  int2* segments;   // rows kernel, shares > 0: [batch][row_tiles][heads], the
                    // first and last workgroup of a segment
};

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

constexpr int kAttnWaves = 4;          // of a workgroup
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr int kAttnTile = 64;          // keys per step
constexpr float kShift = 8.0f;
constexpr float kLazy = 15.0f;         // rescale when t - m > kLazy (m includes the shift)
constexpr float kNoRef = -0x1.fffffep127f;  // reference of a row that has seen nothing
constexpr int kNoBias = 1 << 20;       // value bias before the first block
template <int FMT>
constexpr int kHead = FMT == FP8_E4M3 ? 7 : 0;  // 448 * 2^7 and 57344 both fit fp16

// A workgroup's place: workgroups that read the same keys differ by a multiple
// of the head count in their index, and the last row tiles (which see the most
// keys) come first.
struct AttnPlace {
  int head, split, seq, row_tile;
};
__device__ __forceinline__ AttnPlace attn_place(const AttnArgs& a) {
  AttnPlace p;
  uint32_t x = a.first + blockIdx.x;
  p.head = x % a.cache.heads;
  x /= a.cache.heads;
  p.split = x % a.splits;
  x /= a.splits;
  p.seq = x % a.batch.batch;
  p.row_tile = a.row_tiles - 1 - (int)(x / a.batch.batch);
  return p;
}

// Whether sequence s is this launch's (a mixed batch is two launches').
__device__ __forceinline__ bool attn_serves(const AttnArgs& a, const KVSeq& s) {
  const int rows = s.n * a.group;
  return rows >= a.least && rows <= a.most;
}

// The logits' factor scale * log2(e) is positive in the kernels: a negative
// scale negates the queries, a scale of zero clears them.
__device__ __forceinline__ uint4 sign_queries(uint4 v, float scale) {
  const uint32_t flip = scale < 0.0f ? 0x80008000u : 0u;
  return scale == 0.0f ? make_uint4(0, 0, 0, 0) : make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
}

// The keys a tile of rows [row0, row0 + count) of sequence s reads, and its
// chunks; rows run over (token, head of the group).
struct AttnSpan {
  int lo, hi, chunks;
};
__device__ __forceinline__ AttnSpan attn_span(const AttnArgs& a, const KVSeq& s, int row0, int count) {
  const int last = min(row0 + count, s.n * a.group) - 1;
  AttnSpan p;
  p.hi = a.causal ? min(s.len, s.start + last / a.group + 1) : s.len;
  p.lo = a.window ? max(0, s.start + row0 / a.group - a.window + 1) & ~(kAttnTile - 1) : 0;
  p.chunks = max(1, (p.hi - p.lo + a.chunk - 1) / a.chunk);
  return p;
}

// 2^e as a float for the conversions' scale operand, e clamped to normals.
__device__ __forceinline__ float pow2_scale(int e) {
  return __uint_as_float((uint32_t)(max(-126, min(127, e)) + 127) << 23);
}

// log2(e) * scale * 2^-kb, at least the smallest normal number: an invisible
// logit of -inf times it stays -inf.
__device__ __forceinline__ float key_scale(float scale_log2, int kb) {
  return fmaxf(scale_log2 * pow2_scale(-kb), 0x1p-126f);
}

// A product that is not fused with what follows.
__device__ __forceinline__ float rounded(float s, float kscale) {
#pragma clang fp contract(off)
  return s * kscale;
}

// The reference of a row whose largest logit is top: kShift below it, or top
// itself from 2^24 on, where rounding the difference could take it further down
// (and logits lie 2 and more apart).
__device__ __forceinline__ float reference_for(float top) { return fabsf(top) < 0x1p24f ? top - kShift : top; }

// 8 codes -> 8 bf16, exactly.
template <int FMT>
__device__ __forceinline__ v8b widen_bf16(uint32_t c0, uint32_t c1) {
  v2b r[4];
  if constexpr (FMT == FP8_E4M3) {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, 1.0f, false);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, 1.0f, true);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, 1.0f, false);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, 1.0f, true);
  } else {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c0, 1.0f, false);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c0, 1.0f, true);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c1, 1.0f, false);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c1, 1.0f, true);
  }
  return v8b{r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
}

// 8 codes -> 8 fp16 of value * scale (a power of two).
template <int FMT>
__device__ __forceinline__ v8h widen_f16(uint32_t c0, uint32_t c1, float scale) {
  v2h r[4];
  if constexpr (FMT == FP8_E4M3) {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c0, scale, false);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c0, scale, true);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c1, scale, false);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c1, scale, true);
  } else {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(c0, scale, false);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(c0, scale, true);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(c1, scale, false);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(c1, scale, true);
  }
  return v8h{r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
}

__device__ __forceinline__ v8h pack_f16(const float* p) {
  v2h r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = __builtin_convertvector((v2f{p[2 * e], p[2 * e + 1]}), v2h);
  return v8h{r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2b));
}

// 0xFF in every byte of w that holds a NaN (or, in E5M2, infinity) code.
template <int FMT>
__device__ __forceinline__ uint32_t bad_bytes(uint32_t w) {
  const uint32_t top = (((w & 0x7F7F7F7Fu) + (FMT == FP8_E4M3 ? 0x01010101u : 0x04040404u)) & 0x80808080u) >> 7;
  return top * 0xFFu;
}

// A finite sum of weighted values, or NaN.  An infinite sum means an infinity
// code (no sum of finite codes comes near fp32's range); its sign and whether it
// met a weight of zero would depend on where the keys were split and masked.
template <int FMT>
__device__ __forceinline__ float nan_if_infinite(float o) {
  if constexpr (FMT == FP8_E5M2) return o + (o - o);
  return o;
}

// 1.0 where the byte is set, as fp16.
__device__ __forceinline__ v8h ones_f16(uint32_t m0, uint32_t m1) {
  v8h r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    r[e] = (m0 >> (8 * e)) & 1u ? (_Float16)1.0f : (_Float16)0.0f;
    r[4 + e] = (m1 >> (8 * e)) & 1u ? (_Float16)1.0f : (_Float16)0.0f;
  }
  return r;
}

// The larger of two logits in one instruction (fmaxf first quiets what the
// compiler cannot prove quiet); a NaN loses to any number.
__device__ __forceinline__ float raw_max(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, INFINITY); }

// ln sum_j exp(s_j) of a row: m + log2(l) in base e.  In 64 bits until the last
// rounding: m carries kShift, which the logarithm takes off again (three keys with
// logits of zero: ln 3 = (log2 768 - 8) ln 2 came out 4 units in the last place
// off in fp32).  l = f 2^e with f in [2/3, 4/3): ln l = e ln 2 + 2 atanh(s),
// s = (f - 1) / (f + 1), |s| <= 1/5, by the series up to s^13 / 13 (the rest is
// below 2^-37).  The library's logarithm in its place cost 128 decoded sequences
// of 2000 tokens 92 us instead of 90.
__device__ __forceinline__ float row_lse(float m, float l) {
  if (!(l > 0.0f && l < INFINITY)) return l == 0.0f ? -INFINITY : l + m;  // NaN
  const int e = __builtin_amdgcn_frexp_expf(l * 0.75f);
  const double f = (double)__builtin_ldexpf(l, -e), up = f + 1.0;
  double r = (double)__builtin_amdgcn_rcpf((float)up);
  r = r * (2.0 - up * r);
  const double s = (f - 1.0) * r, s2 = s * s;
  double p = 2.0 / 13;
  p = fma(p, s2, 2.0 / 11);
  p = fma(p, s2, 2.0 / 9);
  p = fma(p, s2, 2.0 / 7);
  p = fma(p, s2, 2.0 / 5);
  p = fma(p, s2, 2.0 / 3);
  p = fma(p, s2, 2.0);
  return (float)fma((double)m + e, 0.693147180559945309417, p * s);
}

// Reductions over the lanes that share a query row: l ^ 32, and l ^ 16.
__device__ __forceinline__ float swap32_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float swap16_max(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float swap32_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap16_sum(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ int swap32_min(int v) {
  const auto r = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
  return min((int)r[0], (int)r[1]);
}
__device__ __forceinline__ int swap16_min(int v) {
  const auto r = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
  return min((int)r[0], (int)r[1]);
}

}  // namespace

// Launchers (attn_rows.hip, attn_tile.hip).  The rows kernel takes row tiles of
// 16 * row_blocks rows (1 or 2; 1 for head_dim 256), the tile kernel of 128.
constexpr int kAttnTileRows = 128;
hipError_t launch_attn_rows(const AttnArgs& a, int row_blocks, uint32_t groups, hipStream_t stream);
// Workgroups of the rows kernel that run at the same time on 256 CUs.
int attn_rows_resident(int head_dim, int row_blocks);
hipError_t launch_attn_tile(const AttnArgs& a, uint32_t groups, hipStream_t stream);

}  // namespace fp8lin
