// Attention of many query rows (prompts, chunks of them) over the paged FP8
// cache: attn_common.h has the mathematics.
//
// MFMA- and VALU-bound.  A workgroup of four waves takes 128 rows (token, head
// of the group) of one sequence and key head; each wave owns 32 of them on the
// 32x32x16 MFMA and keeps its queries, logits and O in registers.  Tiles of 64
// keys and values go through LDS by DMA, as codes, in two buffers: the next
// tile lands while this one is consumed, one barrier a tile.  Each wave widens
// the codes it reads (half the LDS bytes that widened tiles would cost).
//
// LDS, 16-byte chunks swizzled so that the 16 lanes of a read address 16
// different bank groups (64 banks): keys [64][D], chunk c of row r at
// c ^ fk(r); values [D][64], chunk c of row d at c ^ ((d >> 2) & 3).  The DMA
// writes LDS linearly, so the swizzle sits in the lanes' source addresses.
#include "attn_common.h"
#include "lds_dma.h"

namespace fp8lin {
namespace {

constexpr int kWaves = 4;

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

template <int D, int FMT>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void attn_tile_kernel(AttnArgs a) {
  constexpr int J = D / 32;   // 32-dimension steps of the logits
  constexpr int DT = D / 32;  // 32-dimension tiles of the output
  constexpr int kTileBytes = kAttnTile * D;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[2][2][kTileBytes];  // [buffer][keys, values]

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  const AttnPlace at = attn_place(a);
  const int BS = a.cache.block_size, H = a.cache.heads, G = a.group;
  const KVSeq s = kv_seq_uniform(a.batch, BS, at.seq);
  const int rows = s.n * G, row0 = at.row_tile * kAttnTileRows;
  if (row0 >= rows) return;
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

  v16f o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
  float m = kNoRef, l = 0.0f;
  int bref = kNoBias;

  // blocks and biases of a tile's four granules of 16 keys, the same in every
  // lane; read a tile ahead, so that nothing waits for them before the tile's own
  // wait does
  struct Blocks {
    int b[4];
  };
  struct Biases {
    int k[4], v[4];
  };
  auto blocks_of = [&](int T) {
    Blocks r;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int pos = T + 16 * g;
      r.b[g] = pos < kend ? kv_block(a.cache, a.batch, at.seq, pos >> a.block_shift) : -1;
    }
    return r;
  };
  auto biases_of = [&](const Blocks& b) {
    Biases r;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int64_t c = (int64_t)max(b.b[g], 0) * H + at.head;
      r.k[g] = a.cache.k_bias[c];
      r.v[g] = b.b[g] < 0 ? kNoBias : a.cache.v_bias[c];
    }
    return r;
  };
  auto pick = [](const int (&v)[4], int g) { return g < 2 ? (g == 0 ? v[0] : v[1]) : (g == 2 ? v[2] : v[3]); };
  const uint32_t ring0 = lds_addr(ring);
  // this wave's quarter of a tile: D / 64 KB of keys and of values
  auto issue = [&](int T, const Blocks& b, int buf) {
    const uint32_t kdst = ring0 + buf * 2 * kTileBytes, vdst = kdst + kTileBytes;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int piece = wave + kWaves * i;
      {
        const int r = piece * (1024 / D) + lane / (D / 16), c = (lane % (D / 16)) ^ fk<D>(r);
        const int64_t cell = (int64_t)max(pick(b.b, r >> 4), 0) * H + at.head;
        dma16(a.cache.k + (cell * BS + ((T + r) & (BS - 1))) * D + 16 * c, kdst + piece * 1024);
      }
      {
        const int d = piece * 16 + lane / 4, c = (lane & 3) ^ ((d >> 2) & 3);
        const int64_t cell = (int64_t)max(pick(b.b, c), 0) * H + at.head;
        dma16(a.cache.v + (cell * D + d) * BS + ((T + 16 * c) & (BS - 1)), vdst + piece * 1024);
      }
    }
  };

  // Operand roles.  Row r32 of sub-tile `sub` (32 keys) of S^T's A operand is
  // key 16 ((r32 >> 2) & 1) + 4 (r32 >> 3) + (r32 & 3): S^T's result v of a
  // lane is then key 32 sub + 16 h + v.
  const int krow = 16 * ((r32 >> 2) & 1) + 4 * (r32 >> 3) + (r32 & 3);
  uint32_t kfrag[J], vfrag[2];
#pragma unroll
  for (int j = 0; j < J; ++j) kfrag[j] = krow * D + (((2 * j + h) ^ fk<D>(krow)) << 4);
#pragma unroll
  for (int sub = 0; sub < 2; ++sub) vfrag[sub] = kTileBytes + r32 * 64 + (((2 * sub + h) ^ ((r32 >> 2) & 3)) << 4);

  Blocks nb = blocks_of(kbeg);
  issue(kbeg, nb, 0);
  Biases nbias = biases_of(nb);
  Blocks cur = nb;
  nb = blocks_of(kbeg + kAttnTile);
  int buf = 0;
  for (int T = kbeg; T < kend; T += kAttnTile, buf ^= 1) {
    wait_all();
    bare_barrier();  // this tile is whole, and every wave is done with the other buffer
    Blocks blocks;
    Biases bias;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      blocks.b[g] = __builtin_amdgcn_readfirstlane(cur.b[g]);
      bias.k[g] = __builtin_amdgcn_readfirstlane(nbias.k[g]);
      bias.v[g] = __builtin_amdgcn_readfirstlane(nbias.v[g]);
    }
    if (T + kAttnTile < kend) {
      issue(T + kAttnTile, nb, buf ^ 1);
      nbias = biases_of(nb);
      cur = nb;
      nb = blocks_of(T + 2 * kAttnTile);
    }
    if (T >= whi || T + kAttnTile <= wlo) continue;  // nothing for this wave's rows
    const uint32_t tile = ring0 + buf * 2 * kTileBytes;

    v16f sacc[2];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
      for (int e = 0; e < 16; ++e) sacc[sub][e] = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const v4i w = lds_read16(tile + kfrag[j] + sub * 32 * D);
        sacc[sub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_bf16<FMT>(w[0], w[1]), q[j][0], sacc[sub], 0, 0, 0);
        sacc[sub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_bf16<FMT>(w[2], w[3]), q[j][1], sacc[sub], 0, 0, 0);
      }

    const bool missing = blocks.b[0] < 0 || blocks.b[1] < 0 || blocks.b[2] < 0 || blocks.b[3] < 0;
    const bool masked = missing || !__all(T + kAttnTile <= hi && T >= lo);
    float t[2][16];
    float top = -INFINITY;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const float kscale = a.scale_log2 * pow2_scale(-(h ? bias.k[2 * sub + 1] : bias.k[2 * sub]));
#pragma unroll
      for (int e = 0; e < 16; ++e) t[sub][e] = sacc[sub][e] * kscale;
      if (masked) {
        const int first = T + 32 * sub + 16 * h;
        const bool gone = (h ? blocks.b[2 * sub + 1] : blocks.b[2 * sub]) < 0;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (gone || first + e < lo || first + e >= hi) t[sub][e] = -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, t[sub][e]);
    }
    top = swap32_max(top);
    const bool move = top > m + kLazy;
    if (__any(move)) {
      const float to = move ? top - kShift : m;
      const float f = __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= f;
    }
    v8h p[2][2];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        t[sub][e] = __builtin_amdgcn_exp2f(t[sub][e] - m);
        l += t[sub][e];
      }
      p[sub][0] = pack_f16(t[sub]);
      p[sub][1] = pack_f16(t[sub] + 8);
    }

    const int low = min(min(bias.v[0], bias.v[1]), min(bias.v[2], bias.v[3]));
    if (low < bref) {
      if (bref != kNoBias) {
        const float f = pow2_scale(low - bref);
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= f;
      }
      bref = low;
    }
    uint32_t bad = 0;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const int vbias = h ? bias.v[2 * sub + 1] : bias.v[2 * sub];
      const float vscale = pow2_scale(min(bref, 1000) - min(vbias, 1000) + kHead<FMT>);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        v4i w = lds_read16(tile + vfrag[sub] + d * 32 * 64);
        if (masked) {  // no code of an invisible slot may turn 0 * code into NaN
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t b = bad_bytes<FMT>(w[e]);
            bad |= b;
            w[e] &= ~b;
          }
        }
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen_f16<FMT>(w[0], w[1], vscale), p[sub][0], o[d], 0, 0, 0);
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen_f16<FMT>(w[2], w[3], vscale), p[sub][1], o[d], 0, 0, 0);
      }
    }
    if (masked && __any(bad != 0)) {
      // a NaN value reaches the rows that see its token: counted by a product
      // of visibility with "is bad"
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const int first = T + 32 * sub + 16 * h;
        const bool gone = (h ? blocks.b[2 * sub + 1] : blocks.b[2 * sub]) < 0;
        v8h see[2];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          see[e >> 3][e & 7] = gone || first + e < lo || first + e >= hi ? (_Float16)0.0f : (_Float16)1.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const v4i w = lds_read16(tile + vfrag[sub] + d * 32 * 64);
          v16f n;
#pragma unroll
          for (int e = 0; e < 16; ++e) n[e] = 0.0f;
          n = __builtin_amdgcn_mfma_f32_32x32x16_f16(ones_f16(bad_bytes<FMT>(w[0]), bad_bytes<FMT>(w[1])), see[0], n, 0,
                                                     0, 0);
          n = __builtin_amdgcn_mfma_f32_32x32x16_f16(ones_f16(bad_bytes<FMT>(w[2]), bad_bytes<FMT>(w[3])), see[1], n, 0,
                                                     0, 0);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (n[e] > 0.0f) o[d][e] = NAN;
        }
      }
    }
  }
  wait_vmcnt<0>();

  l = swap32_sum(l);
  if (!stored) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const float lse2 = l == 0.0f ? -INFINITY : m + log2f(l);
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
        v[e] = l == 0.0f ? 0.0f : __builtin_ldexpf(o[d][4 * u + e] * inv, -(bref + kHead<FMT>));
      const int at_d = 32 * d + 8 * u + 4 * h;
      if (span.chunks == 1)
        *reinterpret_cast<uint2*>(a.out + cell * D + at_d) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      else
        *reinterpret_cast<v4f*>(a.part_o + slot * D + at_d) = v4f{v[0], v[1], v[2], v[3]};
    }
  if (h == 0) {
    if (span.chunks > 1) a.part_lse[slot] = lse2;
    else if (a.lse) a.lse[cell] = lse2 * 0.693147180559945309f;
  }
}

template <int D>
void run(const AttnArgs& a, uint32_t groups, hipStream_t stream) {
  if (a.cache.fmt == FP8_E4M3)
    hipLaunchKernelGGL((attn_tile_kernel<D, FP8_E4M3>), dim3(groups), dim3(64 * kWaves), 0, stream, a);
  else
    hipLaunchKernelGGL((attn_tile_kernel<D, FP8_E5M2>), dim3(groups), dim3(64 * kWaves), 0, stream, a);
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs& a, uint32_t groups, hipStream_t stream) {
  if (a.cache.head_dim == 64) run<64>(a, groups, stream);
  else if (a.cache.head_dim == 128) run<128>(a, groups, stream);
  else run<256>(a, groups, stream);
  return hipGetLastError();
}

}  // namespace fp8lin
