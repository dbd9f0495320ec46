// Attention over packed sequences, forward: seq_attn.h has the mathematics.
//
// A workgroup takes 128 query rows of one head, a wave 32 of them, its queries,
// logits and output in registers.  Tiles of 64 keys and values (32 with heads of
// 256) go through LDS by DMA, the next one on its way while one is consumed.  Logits
// against a reference that follows the row maximum lazily: it moves when a tile's
// probabilities outgrow it, so most tiles rescale nothing.
//
// Where the workgroups would leave CUs without work they have more waves than rows
// need: two sets of four with every other tile of the keys, or four sets of two
// waves with 64 rows (two with heads of 256); the sets are joined in LDS at the end.
//
// Large calls: two sequences of 4096, 32 heads of 128, everything seen, MFMA busy 46%
// of the SIMDs' cycles and the other vector instructions 39%, with little overlap, at
// 1.6-1.7 GHz (the power limit), no bank conflicts; four causal ones 610-640 us, 860-900
// TFLOP/s.  Heads of 256 hold one wave a SIMD (its output alone takes 128 registers):
// three causal sequences of 2000, 16 heads on 4, 263 us, 370 TFLOP/s.  Small calls
// are latency: 2 x 1024, 12 heads of 64, 14-16 us.
#include <algorithm>

#include "seq_attn.h"

namespace fp8lin {
namespace {

// Keys of a tile: the sets' buffers, two of keys and values each, fit the LDS.
template <int D, int SETS>
constexpr int kKeysOf = D * SETS >= 256 && !(D == 128 && SETS == 2) ? 32 : 64;
// A lane's 32 probabilities of a tile may add up to this before its row's
// reference moves.
constexpr float kMostPart = 0x1p16f;
// References from here on have their logits rounded before they are subtracted
// (attn_common.h).
constexpr float kHuge = 0x1p22f;

// SETS of WAVES waves, each with 32 rows.
template <int D, int WAVES, int SETS>
__global__ __launch_bounds__(64 * WAVES * SETS, D == 256 ? 1 : 2) void seq_attn_fwd_kernel(SeqAttnArgs a) {
  constexpr int J = D / 16, DT = D / 32, kKeys = kKeysOf<D, SETS>, SUB = kKeys / 32, kRows = 32 * WAVES;
  using Load = TileLoad<D, kKeys, WAVES>;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[SETS][2][2][Load::kBytes];  // [set][buffer][keys, values]
  __shared__ int found[WAVES * SETS];

  const int lane = threadIdx.x & 63, all_waves = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wave = all_waves % WAVES, set = all_waves / WAVES;
  const int r32 = lane & 31, h = lane >> 5;
  uint32_t x = a.first + blockIdx.x;
  const int kv_head = x % a.heads;
  x /= a.heads;
  const int head = kv_head * a.group + x % a.group;
  x /= a.group;
  // late rows see most: first
  NthTile tile = {(int)(x % a.batch), a.tiles - 1 - (int)(x / a.batch)};
  if (a.rest > 0) {
    tile = {(int)x - a.rest, 0};
    if ((int)x < a.rest) tile = nth_tile(a, a.rest - 1 - (int)x);
    if (tile.seq < 0) return;
  }
  const Seq s = seq_of(a, tile.seq);
  const int row0 = tile.tile * kRows;
  if (row0 >= s.n) return;
  const int khi = a.causal ? min(s.n, row0 + kRows) : s.n;
  const int klo = a.window ? max(0, row0 - a.window + 1) & ~(kKeys - 1) : 0;

  const uint32_t ring0 = lds_addr(ring[set]);
  const int64_t ks = a.k_stride * 2, vs = a.v_stride * 2;
  const Load load_k(lane, wave, (uint32_t)ks), load_v(lane, wave, (uint32_t)vs);
  const uint16_t* kp = a.k + (int64_t)(s.first + klo) * a.k_stride + kv_head * D;
  const uint16_t* vp = a.v + (int64_t)(s.first + klo) * a.v_stride + kv_head * D;
  auto issue = [&](int T, int buf) {
    load_k.issue(kp + (int64_t)(T - klo) * a.k_stride, ks, s.n - T, ring0 + buf * 2 * Load::kBytes, wave);
    load_v.issue(vp + (int64_t)(T - klo) * a.v_stride, vs, s.n - T, ring0 + (2 * buf + 1) * Load::kBytes, wave);
  };
  const int first_key = klo + set * kKeys;
  if (first_key < khi) issue(first_key, 0);

  const int wrow = row0 + 32 * wave, row = wrow + r32;
  v8b q[J];
#pragma unroll
  for (int j = 0; j < J; ++j) q[j] = v8b{};
  if (row < s.n) {
    const uint16_t* p = a.q + (int64_t)(s.first + row) * a.q_stride + head * D + 8 * h;
#pragma unroll
    for (int j = 0; j < J; ++j) q[j] = *reinterpret_cast<const v8b*>(p + 16 * j);
    // (all on their way before the first is used: 1000 sequences of 64 tokens, 32 heads
    // of 128, one after the other 616 us, so 464)
    if (__builtin_expect(a.scale == 0.0f, 0)) {
      asm volatile("");  // a branch
#pragma unroll
      for (int j = 0; j < J; ++j) q[j] = __builtin_bit_cast(v8b, bad_of(q[j]) & 0x7FC07FC0);  // 0 * NaN, 0 * inf
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) q[j] = __builtin_bit_cast(v8b, sign_queries(__builtin_bit_cast(uint4, q[j]), a.scale));
    }
  }
  const float c_log2 = a.scale == 0.0f ? 1.0f : fabsf(a.scale_log2);
  // the keys of the lane's row, and of any of the wave's
  const int hi = a.causal ? min(row + 1, s.n) : s.n, lo = a.window ? row - a.window + 1 : 0;
  const int whi = wrow >= s.n ? 0 : (a.causal ? min(wrow + 32, s.n) : s.n);
  const int wlo = a.window ? wrow - a.window + 1 : 0;
  // the keys that every row of the workgroup sees
  const int all_hi = a.causal ? min(s.n, row0 + 1) : s.n;
  const int all_lo = a.window ? min(row0 + kRows, s.n) - a.window : 0;

  v16f o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = zero16();
  float m = kNoRef, l = 0.0f;
  bool huge = false;  // the row's reference passes kHuge

  const uint32_t krow = row_place<D>(lane), vcol = column_place<D>(lane);

  auto consume = [&](bool masked, int T, uint32_t tile) {
    auto seen = [&](int sub, int e) {
      const int key = T + 32 * sub + result_row(e, h);
      return key >= lo && key < hi;
    };
    v16f t[SUB];
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub) t[sub] = zero16();
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub) t[sub] = mma(lds_row(((tile + krow) ^ (32 * j)) + sub * 64 * D), q[j], t[sub]);
      if (D > 64 && j % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // LDS reads do not run further ahead: registers
    }
    __builtin_amdgcn_s_setprio(0);
    if (masked) {
      asm volatile("");  // a branch: as selects it would cost every tile
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
        for (int e = 0; e < 16; ++e) t[sub][e] = seen(sub, e) ? t[sub][e] : -INFINITY;
    }
    float scale = c_log2;
    // of the rows whose reference is huge; what a row's bits are depends on no other row
    auto round_logits = [&](bool now) {
      asm volatile("");  // a branch of its own, and a rare one
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
        for (int e = 0; e < 16; ++e) t[sub][e] = now ? rounded(t[sub][e], scale) : t[sub][e];
      scale = now ? 1.0f : scale;
    };
    if (__builtin_expect(__any(huge), 0)) round_logits(huge);
    v8b p[SUB][2];
    float part;
    auto probabilities = [&] {
      part = 0.0f;
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub) {
        v16f w;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          w[e] = __builtin_amdgcn_exp2f(fmaf(t[sub][e], scale, -m));
          part += w[e];  // of the fp32 values
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) p[sub][c] = operand(w, c);
      }
    };
    probabilities();
    const bool over = !(part <= kMostPart);
    if (__any(over)) {
      float top = -INFINITY;
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = raw_max(top, t[sub][e]);
      top = swap32_max(top * scale);
      const bool move = swap32_max(over ? 1.0f : 0.0f) > 0.0f;  // this row's, in either half
      const float to = move && top > m ? top : m;
      const float f = __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= f;
      const bool now = !huge && fabsf(m) > kHuge && m != kNoRef;
      if (__any(now)) {
        round_logits(now);
        huge = huge || now;
      }
      probabilities();
    }
    l += part;
    if (D > 64) __builtin_amdgcn_sched_barrier(0);
    const uint32_t v = tile + Load::kBytes + vcol;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int c = 0; c < 2 * SUB; ++c) {
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] = mma(column_step<D>(v + c * 32 * D, d), p[c >> 1][c & 1], o[d]);
      if (D > 64 && (c & 1)) __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
  };

  // Values of a tile that are NaN or infinite: the outputs of the rows that see
  // them become NaN -- counted by a product of "is bad" with what is seen --
  // before they are cleared.
  auto record = [&](int T, uint32_t values) {
    v8b see[2 * SUB];
#pragma unroll
    for (int c = 0; c < 2 * SUB; ++c) {
      v8s w;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int key = T + 32 * (c >> 1) + result_row(8 * (c & 1) + e, h);
        w[e] = key >= lo && key < hi ? 0x3F80 : 0;  // 1.0
      }
      see[c] = __builtin_bit_cast(v8b, w);
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      v16f n = zero16();
#pragma unroll
      for (int c = 0; c < 2 * SUB; ++c) {
        __builtin_amdgcn_sched_barrier(0);
        v4i32 bad = bad_of(column_step<D>(values + vcol + c * 32 * D, d));
        bad &= 0x3F803F80;
        n = mma(__builtin_bit_cast(v8b, bad), see[c], n);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = n[e] > 0.0f ? NAN : o[d][e];
    }
  };

  int buf = 0;
  for (int all = klo; all < khi; all += SETS * kKeys, buf ^= 1) {
    const int T = all + set * kKeys;
    wait_vmcnt<0>();
    bare_barrier();  // this tile is whole, and every wave is done with the one before
    if (T + SETS * kKeys < khi) issue(T + SETS * kKeys, buf ^ 1);
    const uint32_t tile = ring0 + buf * 2 * Load::kBytes;
    if (all + SETS * kKeys > all_hi || all < all_lo) {
      const uint32_t values = tile + Load::kBytes;
      if (has_bad<Load::kBytes, SETS, WAVES>(values, found, T < khi)) {
        if (T < khi) record(T, values);
        clear_bad<Load::kBytes, WAVES>(values, 2 * D, nullptr);
      }
    }
    if (T >= min(whi, khi) || T + kKeys <= wlo) continue;
    // (rows past the sequence's end see what its last row sees: not stored)
    const bool whole = T + kKeys <= min(s.n, a.causal ? wrow + 1 : s.n) && (!a.window || T > wrow + 31 - a.window);
    consume(!whole, T, tile);
  }

  if constexpr (SETS > 1) {
    // the other sets' rows to LDS, lane by lane; the first set's waves add them
    constexpr int kState = 64 * (16 * DT + 2);
    static_assert(sizeof(ring) >= (SETS - 1) * WAVES * kState * 4, "the sets' state fits the ring");
    float* state = reinterpret_cast<float*>(&ring[0][0][0][0]) + (all_waves - WAVES) * kState + lane;
    __syncthreads();
    if (set > 0) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) state[64 * (16 * d + e)] = o[d][e];
      state[64 * 16 * DT] = m;
      state[64 * (16 * DT + 1)] = l;
    }
    __syncthreads();
    if (set > 0) return;
#pragma unroll 1
    for (int other = 1; other < SETS; ++other) {
      state += WAVES * kState;
      const float m1 = state[64 * 16 * DT], to = m1 > m ? m1 : m;
      const float f0 = __builtin_amdgcn_exp2f(m - to), f1 = __builtin_amdgcn_exp2f(m1 - to);
      m = to;
      l = l * f0 + state[64 * (16 * DT + 1)] * f1;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = o[d][e] * f0 + state[64 * (16 * d + e)] * f1;
    }
  }

  l = swap32_sum(l);
  if (row >= s.n) return;
  const float inv = 1.0f / l;
  const int64_t cell = (int64_t)(s.first + row) * a.q_heads + head;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = finite_or_nan(o[d][4 * u + e]) * inv;
      *reinterpret_cast<uint2*>(a.out + cell * D + 32 * d + 8 * u + 4 * h) =
          make_uint2(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]));
    }
  if (h == 0) a.lse[cell] = row_lse(m, l);
}

}  // namespace

hipError_t launch_seq_attn_fwd(SeqAttnArgs a, int head_dim, hipStream_t stream) {
  a.tiles = (a.max_len + kSeqRows - 1) / kSeqRows;
  a.rest = ragged_places(a.tokens, a.batch, a.tiles);
  int64_t groups = (a.rest > 0 ? (int64_t)a.rest + a.batch : (int64_t)a.tiles * a.batch) * a.q_heads;
  // tiles of 128 rows that there may be, of all heads; and whether the last rows of
  // a sequence walk on when the others are done
  const int64_t busy = std::min(groups, ((int64_t)a.tokens / kSeqRows + a.batch) * a.q_heads);
  const bool uneven = a.causal && a.window == 0, long_rows = a.max_len >= 2048;
  // 64 rows a workgroup where each has a CU to itself (256 CUs); of uneven walks
  // also where two share one, with heads of 128 only the long ones' (the sets' tiles
  // are half as large there, and half as many fit a CU).  us with 128 and with 64
  // rows: causal, 2 x 1024 tokens of 12 heads of 64 17.1 and 13.9, 4000 of 2 of 128
  // 69 and 48, 4000 of 2 of 256 267 and 161, 2048 of 16 on 4 of 256 146 and 104, 8192
  // of 4 of 128 139 and 110; but 1024 of 32 of 128 26.6 and 28.1, 8192 of 8 of 64 98
  // and 100; everything seen, 2048 of 16 on 4 of 256 147 and 176.
  const int64_t most = !uneven ? 128 : head_dim == 64 ? (long_rows ? 400 : 256) : head_dim == 256 || long_rows ? 256 : 128;
  const bool half = busy <= most && a.max_len > 64 && a.rest == 0;
  // 128 rows, two sets: where a workgroup has a CU to itself, and where the last rows
  // of a long causal sequence would go on alone: us with one set and with two, one of
  // 8192 tokens, 8 heads of 64, 123 and 98, 2048 of 32 heads of 128 59 and 54.
  // Elsewhere the sets' joining costs more: two sequences of 1000 tokens, 32 heads of
  // 64, 21.5 and 23.1, of 1500 and 300, 40 heads of 128, 47 and 60.
  const bool two = (busy <= 256 || (uneven && long_rows && busy <= 600)) && a.max_len > 64;
  if (half) {
    a.tiles = (a.max_len + 63) / 64;
    groups = (int64_t)a.tiles * a.batch * a.q_heads;
  }
  auto launch = [&](auto kernel, int threads) {
    in_stretches(groups, threads, [&](uint32_t first, uint32_t count) {
      a.first = first;
      hipLaunchKernelGGL(kernel, dim3(count), dim3(threads), 0, stream, a);
    });
  };
  if (head_dim == 64) {
    if (half) launch(seq_attn_fwd_kernel<64, 2, 4>, 512);
    else two ? launch(seq_attn_fwd_kernel<64, 4, 2>, 512) : launch(seq_attn_fwd_kernel<64, 4, 1>, 256);
  } else if (head_dim == 128) {
    if (half) launch(seq_attn_fwd_kernel<128, 2, 4>, 512);
    else two ? launch(seq_attn_fwd_kernel<128, 4, 2>, 512) : launch(seq_attn_fwd_kernel<128, 4, 1>, 256);
  } else {
    half ? launch(seq_attn_fwd_kernel<256, 2, 2>, 256) : launch(seq_attn_fwd_kernel<256, 4, 1>, 256);
  }
  return hipGetLastError();
}

}  // namespace fp8lin
