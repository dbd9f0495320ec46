// Attention of a few query rows (single tokens, short drafts) over the paged
// FP8 cache: attn_common.h has the mathematics.
//
// HBM-bound: every cached byte of the (sequence, key head) is read once and
// serves the group's query rows, 16 per MFMA tile.  One workgroup of four
// waves per chunk of keys; the waves take the chunk's tiles of 64 keys in
// turn, each with its own running maximum, sum and O, and meet in LDS at the
// end.  Keys and values go from memory straight to registers: a load
// instruction covers whole 64-byte runs, and the next tile's keys are in
// flight during this tile's softmax, its values during the next one's logits.
#include "attn_common.h"

namespace fp8lin {
namespace {

constexpr int kWaves = 4;

template <int D, int FMT, int RB>
__global__ __launch_bounds__(64 * kWaves, D * RB >= 256 ? 1 : 2) void attn_rows_kernel(AttnArgs a) {
  constexpr int kRows = 16 * RB;
  constexpr int J = D / 64;   // 64-dimension steps of the logits
  constexpr int DT = D / 16;  // 16-dimension tiles of the output
  constexpr int kPitch = D + 4;
  __shared__ float so[kWaves][16][kPitch];
  __shared__ float sm[kWaves][kRows], sl[kWaves][kRows];
  __shared__ int sb[kWaves];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const AttnPlace at = attn_place(a);
  const int BS = a.cache.block_size, H = a.cache.heads, G = a.group;
  const KVSeq s = kv_seq(a.batch, BS, at.seq);
  const int rows = s.n * G, row0 = at.row_tile * kRows;
  if (row0 >= rows) return;
  const AttnSpan span = attn_span(a, s, row0, kRows);
  if (at.split >= span.chunks) return;
  const int kbeg = span.lo + at.split * a.chunk, kend = min(span.hi, kbeg + a.chunk);

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
      const uint16_t* qp = a.q + (int64_t)(s.first + row / G) * a.q_stride + (at.head * G + row % G) * D + 16 * g;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        q[rb][j][0] = *reinterpret_cast<const v8b*>(qp + 64 * j);
        q[rb][j][1] = *reinterpret_cast<const v8b*>(qp + 64 * j + 8);
      }
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

  // Operand roles.  Logits: row r16 of sub-tile `sub` is the key
  // 16 (r16 / 4) + 4 sub + r16 % 4 of the tile; then S^T's four results of
  // sub-tile `sub` in lane (r16, g) are the keys 16 g + 4 sub + 0..3.
  const int gk = r16 >> 2;
  auto block_of = [&](int pos) { return pos < kend ? kv_block(a.cache, a.batch, at.seq, pos / BS) : -1; };
  auto cell = [&](int block) { return (int64_t)max(block, 0) * H + at.head; };
  const uint32_t k_lane = (r16 & 3) * D + 16 * g, v_lane = r16 * BS;
  uint4 kreg[4][J], vreg[DT];
  auto load_k = [&](int T, int block) {
    const uint8_t* p = a.cache.k + cell(block) * BS * D + ((T + 16 * gk) & (BS - 1)) * D + k_lane;
#pragma unroll
    for (int sub = 0; sub < 4; ++sub)
#pragma unroll
      for (int j = 0; j < J; ++j) kreg[sub][j] = *reinterpret_cast<const uint4*>(p + 4 * sub * D + 64 * j);
  };
  auto load_v = [&](int T, int block) {
    const uint8_t* p = a.cache.v + cell(block) * BS * D + ((T + 16 * g) & (BS - 1)) + v_lane;
#pragma unroll
    for (int d = 0; d < DT; ++d) vreg[d] = *reinterpret_cast<const uint4*>(p + 16 * d * BS);
  };

  constexpr int kStep = kWaves * kAttnTile;
  int T = kbeg + wave * kAttnTile;
  int bk = -1, bv = -1, kb = 0, vb = 0;
  if (T < kend) {
    bk = block_of(T + 16 * gk);
    bv = block_of(T + 16 * g);
    load_k(T, bk);
    load_v(T, bv);
    kb = a.cache.k_bias[cell(bv)];
    vb = a.cache.v_bias[cell(bv)];
  }
  int nbk = block_of(T + kStep + 16 * gk), nbv = block_of(T + kStep + 16 * g);
  for (; T < kend; T += kStep) {
    // logits
    v4f sacc[RB][4];
#pragma unroll
    for (int sub = 0; sub < 4; ++sub) {
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
    const float kscale = a.scale_log2 * pow2_scale(-kb);
    const int vbias = block >= 0 ? vb : kNoBias;
    // the next tile's keys, and the block numbers of the one after
    const bool more = T + kStep < kend;
    if (more) {
      bk = nbk, bv = nbv;
      load_k(T + kStep, bk);
      kb = a.cache.k_bias[cell(bv)];
      vb = a.cache.v_bias[cell(bv)];
      nbk = block_of(T + 2 * kStep + 16 * gk);
      nbv = block_of(T + 2 * kStep + 16 * g);
    }

    bool inside = block >= 0;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) inside = inside && T + kAttnTile <= hi[rb] && T >= lo[rb];
    const bool masked = !__all(inside);
    v8h p[RB][2];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      float t[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) t[e] = sacc[rb][e >> 2][e & 3] * kscale;
      if (masked) {
        const int first = T + 16 * g;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (block < 0 || first + e < lo[rb] || first + e >= hi[rb]) t[e] = -INFINITY;
      }
      float top = t[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) top = fmaxf(top, t[e]);
      top = swap16_max(swap32_max(top));
      const bool move = top > m[rb] + kLazy;
      if (__any(move)) {
        const float to = move ? top - kShift : m[rb];
        const float f = __builtin_amdgcn_exp2f(m[rb] - to);
        m[rb] = to;
        l[rb] *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[rb][d] *= f;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        t[e] = __builtin_amdgcn_exp2f(t[e] - m[rb]);
        l[rb] += t[e];
      }
      p[rb][0] = pack_f16(t);
      p[rb][1] = pack_f16(t + 8);
    }

    // values, at the scale of the smallest bias so far
    const int low = __builtin_amdgcn_readfirstlane(swap16_min(swap32_min(vbias)));
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
    uint32_t bad = 0;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      uint4 w = vreg[d];
      if (masked) {  // no code of an invisible slot may turn 0 * code into NaN
        const uint4 b = make_uint4(bad_bytes<FMT>(w.x), bad_bytes<FMT>(w.y), bad_bytes<FMT>(w.z), bad_bytes<FMT>(w.w));
        bad |= b.x | b.y | b.z | b.w;
        w = make_uint4(w.x & ~b.x, w.y & ~b.y, w.z & ~b.z, w.w & ~b.w);
      }
      const v8h v0 = widen_f16<FMT>(w.x, w.y, vscale), v1 = widen_f16<FMT>(w.z, w.w, vscale);
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        o[rb][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p[rb][0], o[rb][d], 0, 0, 0);
        o[rb][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p[rb][1], o[rb][d], 0, 0, 0);
      }
    }
    if (masked && __any(bad != 0)) {
      // a NaN value reaches the rows that see its token: counted by a product
      // of visibility with "is bad"
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        v8h see[2];
        const int first = T + 16 * g;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          see[e >> 3][e & 7] =
              block < 0 || first + e < lo[rb] || first + e >= hi[rb] ? (_Float16)0.0f : (_Float16)1.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const uint4 w = vreg[d];
          v4f n{0, 0, 0, 0};
          n = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones_f16(bad_bytes<FMT>(w.x), bad_bytes<FMT>(w.y)), see[0], n, 0,
                                                     0, 0);
          n = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones_f16(bad_bytes<FMT>(w.z), bad_bytes<FMT>(w.w)), see[1], n, 0,
                                                     0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n[e] > 0.0f) o[rb][d][e] = NAN;
        }
      }
    }
    if (more) load_v(T + kStep, bv);
  }

  // the waves' results meet: row r of the workgroup, four waves in order
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
      for (int e = 0; e < 4; ++e) sum[e] = total == 0.0f ? 0.0f : __builtin_ldexpf(sum[e] * inv, -(low + kHead<FMT>));
      const float lse2 = total == 0.0f ? -INFINITY : top + log2f(total);
      const int64_t cell_at = (int64_t)(s.first + row / G) * a.q_heads + at.head * G + row % G;
      if (span.chunks == 1) {
        *reinterpret_cast<uint2*>(a.out + cell_at * D + d) =
            make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
        if (d == 0 && a.lse) a.lse[cell_at] = lse2 * 0.693147180559945309f;
      } else {
        const int64_t slot = (int64_t)at.split * a.batch.tokens * a.q_heads + cell_at;
        *reinterpret_cast<v4f*>(a.part_o + slot * D + d) = sum;
        if (d == 0) a.part_lse[slot] = lse2;
      }
    }
  }
}

template <int D, int RB>
void run(const AttnArgs& a, uint32_t groups, hipStream_t stream) {
  if (a.cache.fmt == FP8_E4M3)
    hipLaunchKernelGGL((attn_rows_kernel<D, FP8_E4M3, RB>), dim3(groups), dim3(64 * kWaves), 0, stream, a);
  else
    hipLaunchKernelGGL((attn_rows_kernel<D, FP8_E5M2, RB>), dim3(groups), dim3(64 * kWaves), 0, stream, a);
}

}  // namespace

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
