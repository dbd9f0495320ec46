// The paged FP8 cache of keys and values: written as tokens arrive, and read
// back (include/fp8lin_block.h has the definitions).
//
// Append.  One workgroup per (sequence, touched block, head) holds that block's
// new keys and values in registers between their largest magnitude and the
// codes, so they are read once; the rotation is applied on the way.  Values
// change their order (tokens by dimensions -> dimensions by tokens) four by four
// codes in registers, then through LDS.  Further workgroups of the same launch
// rotate the queries.  Single tokens are bound by three loads that wait for one
// another (lengths, block number, tokens: the last two overlap); prompts by the
// same chain under load, since a workgroup has only 64 KB to fetch: 3.7 TB/s
// for keys and values, 5.1 for the queries; 617 MB of four prompts of 700 to
// 4000 tokens, 32 heads of 128, in 152-154 us.
//
// Read.  HBM-bound: 629 MB of eight sequences of 9000 to 16384 tokens, 8 heads
// of 128, in 116-117 us, 5.4 TB/s.
#include <type_traits>

#include "fp8_code.h"
#include "internal.h"
#include "kv_device.h"
#include "rope.h"

namespace fp8lin {
namespace {

// Largest finite magnitude bits.
__device__ __forceinline__ uint32_t finite_mag(float v) {
  const uint32_t m = __float_as_uint(v) & 0x7FFFFFFFu;
  return m < 0x7F800000u ? m : 0u;
}

template <int FMT>
__device__ __forceinline__ float code_value(uint32_t c) {
  if constexpr (FMT == FP8_E4M3)
    return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
  else
    return __builtin_amdgcn_cvt_f32_bf8((int)c, 0);
}

// The 4 x 4 bytes of r[0..3] (row i, byte j) transposed: r[j], byte i.
__device__ __forceinline__ void transpose4(uint32_t (&r)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u);  // bytes 0 0 1 1 of rows 0 1
  const uint32_t b = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);  // bytes 2 2 3 3
  const uint32_t c = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
  r[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  r[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  r[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  r[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

struct AppendArgs {
  fp8_kv_cache_t cache;
  fp8_kv_batch_t batch;
  const void* k;
  const void* v;
  const void* q;
  int64_t k_stride, v_stride, q_stride;
  int q_heads;
  uint16_t* q_out;
  Rope rope;
  int blocks_per_seq;   // most blocks a sequence's new tokens touch
  int64_t kv_groups;    // workgroups of the keys and values; the others are the queries'
  uint32_t first;       // this launch's first workgroup
  int q_tokens;         // tokens of one of the queries' workgroups
  int q_groups;         // of them per sequence
};

constexpr int kUnits = 4;  // units a lane holds

template <int DT, int FMT, int D, int ROPE>
__global__ __launch_bounds__(1024) void kv_append_kernel(AppendArgs a) {
  constexpr int kUpt = D / 8;       // units of a token and head
  extern __shared__ uint8_t lds[];  // values' codes, [D][block_size + 4]
  __shared__ uint32_t part[2][16];
  const int nt = blockDim.x, t = threadIdx.x;
  const int BS = a.cache.block_size, H = a.cache.heads;

  uint32_t g = a.first + blockIdx.x;
  if ((int64_t)g >= a.kv_groups) {  // some tokens' queries
    g -= (uint32_t)a.kv_groups;
    const int i = g / a.q_groups, nth = (g % a.q_groups) * a.q_tokens;
    const KVSeq s = kv_seq_uniform(a.batch, BS, i);
    const int count = min(a.q_tokens, s.n - nth);
    if (count <= 0) return;
    const int units = a.q_heads * kUpt;  // of a token
    for (int tok = 0; tok < count; ++tok) {
      const int64_t row = s.first + nth + tok;
      for (int x0 = t; x0 < units; x0 += kUnits * nt) {
        float v[kUnits][8], angle[8];
        // x % kUpt is the same for every q: nt is a multiple of kUpt
        load_angles<D, ROPE>(angle, x0 % kUpt, s.start + nth + tok, a.rope);
#pragma unroll
        for (int q = 0; q < kUnits; ++q) {
          const int x = x0 + q * nt, head = x / kUpt, u = x % kUpt;
          if (x < units) {
            load4<DT>(a.q, row * a.q_stride + head * D + unit_lo<D>(u), v[q]);
            load4<DT>(a.q, row * a.q_stride + head * D + unit_hi<D>(u), v[q] + 4);
          }
        }
#pragma unroll
        for (int q = 0; q < kUnits; ++q) {
          const int x = x0 + q * nt, head = x / kUpt, u = x % kUpt;
          if (x < units) {
            rotate<ROPE>(v[q], angle);
            uint16_t* o = a.q_out + (row * a.q_heads + head) * D;
            *reinterpret_cast<uint2*>(o + unit_lo<D>(u)) = bf16x4(v[q]);
            *reinterpret_cast<uint2*>(o + unit_hi<D>(u)) = bf16x4(v[q] + 4);
          }
        }
      }
    }
    return;
  }

  const int head = g % H;
  g /= H;
  const int nth_block = g % a.blocks_per_seq, i = g / a.blocks_per_seq;
  const KVSeq s = kv_seq_uniform(a.batch, BS, i);
  if (s.n == 0) return;
  const int block_at = (s.start >> __builtin_ctz(BS)) + nth_block;  // of the sequence
  const int p0 = max(s.start, block_at * BS);                       // first new position in the block
  const int p1 = min(s.start + s.n, block_at * BS + BS);            // one past the last
  if (p0 >= p1) return;
  const int block_number = kv_block(a.cache, a.batch, i, block_at);  // needed after the tokens are in
  const int slot0 = p0 - block_at * BS, slot1 = p1 - block_at * BS;

  // This lane's units: keys, unit t + q * nt of the new tokens in order;
  // values, dimensions u of the four tokens of an aligned quad of slots, which
  // makes four codes of one dimension a word.
  const int64_t row0 = s.first - s.start + (int64_t)block_at * BS;  // of slot 0
  const int u = t % kUpt;                                           // nt is a multiple of kUpt
  auto key_slot = [&](int q) { return slot0 + (t + q * nt) / kUpt; };
  const int quad = 4 * ((slot0 >> 2) + t / kUpt);
  float kv[kUnits][8], vv[kUnits][8], angle[kUnits][8];
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
#pragma unroll
    for (int e = 0; e < 8; ++e) kv[q][e] = vv[q][e] = angle[q][e] = 0.0f;
    if (key_slot(q) < slot1) {
      const int64_t at = (row0 + key_slot(q)) * a.k_stride + head * D;
      load4<DT>(a.k, at + unit_lo<D>(u), kv[q]);
      load4<DT>(a.k, at + unit_hi<D>(u), kv[q] + 4);
      load_angles<D, ROPE>(angle[q], u, block_at * BS + key_slot(q), a.rope);
    }
  }
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    if (quad + q >= slot0 && quad + q < slot1) {
      const int64_t at = (row0 + quad + q) * a.v_stride + head * D;
      load4<DT>(a.v, at + unit_lo<D>(u), vv[q]);
      load4<DT>(a.v, at + unit_hi<D>(u), vv[q] + 4);
    }
  }
  const int block = __builtin_amdgcn_readfirstlane(block_number);
  if (block < 0) return;
  const int64_t cell = (int64_t)block * H + head;
  const int32_t old_k = a.cache.k_bias[cell], old_v = a.cache.v_bias[cell];
  uint32_t mk = 0, mv = 0;
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    rotate<ROPE>(kv[q], angle[q]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mk = max(mk, finite_mag(kv[q][e]));
      mv = max(mv, finite_mag(vv[q][e]));
    }
  }
  for (int off = 32; off > 0; off >>= 1) {
    mk = max(mk, (uint32_t)__shfl_xor((int)mk, off, 64));
    mv = max(mv, (uint32_t)__shfl_xor((int)mv, off, 64));
  }
  if ((t & 63) == 0) {
    part[0][t >> 6] = mk;
    part[1][t >> 6] = mv;
  }
  __syncthreads();  // (and every lane has read the old biases)
  for (int w = 0; w < nt / 64; ++w) {
    mk = max(mk, part[0][w]);
    mv = max(mv, part[1][w]);
  }

  // a block's bias; where it falls, the tokens that were there are coded again
  uint8_t* k_codes = a.cache.k + cell * BS * D;
  uint8_t* v_codes = a.cache.v + cell * BS * D;
  auto settle = [&](uint32_t m, int32_t old, int32_t* bias, uint8_t* codes, bool values) {
    int32_t b = m == 0 ? FP8_KV_MAX_BIAS : min(FP8_KV_MAX_BIAS, bias_from_amax_bits(m, FMT, 0));
    if (slot0 > 0) {
      b = min(b, old);
      if (b < old) {
        const int32_t step = b < old - 300 ? -300 : b - old;
        for (int x = t; x < slot0 * D; x += nt) {
          uint8_t* c = codes + (values ? (x / slot0) * BS + x % slot0 : x);
          const uint32_t old_code = *c;
          if ((old_code & 0x7Fu) < (FMT == FP8_E4M3 ? 0x7Fu : 0x7Cu))  // NaN and infinity stay
            *c = (uint8_t)fp8_code<FMT>(__float_as_uint(code_value<FMT>(old_code)), step);
        }
      }
    }
    if (t == 0) *bias = b;
    return b;
  };
  const Coder<FMT> k_coder(settle(mk, old_k, a.cache.k_bias + cell, k_codes, false));
  const Coder<FMT> v_coder(settle(mv, old_v, a.cache.v_bias + cell, v_codes, true));

#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    if (key_slot(q) < slot1) {
      uint8_t* o = k_codes + key_slot(q) * D;
      *reinterpret_cast<uint32_t*>(o + unit_lo<D>(u)) = k_coder.four(*reinterpret_cast<const float(*)[4]>(kv[q]));
      *reinterpret_cast<uint32_t*>(o + unit_hi<D>(u)) = k_coder.four(*reinterpret_cast<const float(*)[4]>(kv[q] + 4));
    }
  }

  uint32_t code[kUnits][2];
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    code[q][0] = v_coder.four(*reinterpret_cast<const float(*)[4]>(vv[q]));
    code[q][1] = v_coder.four(*reinterpret_cast<const float(*)[4]>(vv[q] + 4));
  }
  if (slot1 - slot0 == 1) {  // one token: its codes go out byte by byte
#pragma unroll
    for (int q = 0; q < kUnits; ++q)
      if (quad + q == slot0)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v_codes[((e < 4 ? unit_lo<D>(u) : unit_hi<D>(u) - 4) + e) * BS + slot0] =
              (uint8_t)(code[q][e >> 2] >> (8 * (e & 3)));
    return;
  }
  const int pitch = BS + 4;
  if (quad < slot1) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t r[4] = {code[0][half], code[1][half], code[2][half], code[3][half]};
      transpose4(r);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<uint32_t*>(lds + ((half ? unit_hi<D>(u) : unit_lo<D>(u)) + e) * pitch + quad) = r[e];
    }
  }
  __syncthreads();
  const int words = BS / 4, shift = __builtin_ctz(words);  // of a dimension's row
  for (int x = t; x < D * words; x += nt) {
    const int d = x >> shift, c = 4 * (x & (words - 1));
    if (c >= slot0 && c + 4 <= slot1) {
      *reinterpret_cast<uint32_t*>(v_codes + d * BS + c) = *reinterpret_cast<const uint32_t*>(lds + d * pitch + c);
    } else {
      for (int e = 0; e < 4; ++e)
        if (c + e >= slot0 && c + e < slot1) v_codes[d * BS + c + e] = lds[d * pitch + c + e];
    }
  }
}

// ---------------------------------------------------------------- read
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

struct ReadArgs {
  fp8_kv_cache_t cache;
  fp8_kv_batch_t batch;
  void* k;
  void* v;
  int blocks_per_seq;
  uint32_t first;  // this launch's first workgroup
};

// 8 codes (two words) times 2^-b -> out_dtype at o, each rounded once: by the
// conversion itself where 2^-b and every result are normal numbers.
template <int OT, int FMT>
__device__ __forceinline__ void write8(void* p, int64_t i, uint32_t c0, uint32_t c1, int32_t b, float scale, bool hw) {
  if constexpr (OT == FP8_IN_FP32) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __builtin_ldexpf(code_value<FMT>((c0 >> (8 * e)) & 0xFFu), -b);
      v[4 + e] = __builtin_ldexpf(code_value<FMT>((c1 >> (8 * e)) & 0xFFu), -b);
    }
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint4 o;
    if (hw) {
      hw_v2bf r[4];
      if constexpr (FMT == FP8_E4M3) {
        r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, scale, false);
        r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, scale, true);
        r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, scale, false);
        r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, scale, true);
      } else {
        r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c0, scale, false);
        r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c0, scale, true);
        r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c1, scale, false);
        r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c1, scale, true);
      }
      o = make_uint4(__builtin_bit_cast(uint32_t, r[0]), __builtin_bit_cast(uint32_t, r[1]),
                     __builtin_bit_cast(uint32_t, r[2]), __builtin_bit_cast(uint32_t, r[3]));
    } else {
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = __builtin_ldexpf(code_value<FMT>((c0 >> (8 * e)) & 0xFFu), -b);
        v[4 + e] = __builtin_ldexpf(code_value<FMT>((c1 >> (8 * e)) & 0xFFu), -b);
      }
      const uint2 lo = bf16x4(v), hi = bf16x4(v + 4);
      o = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    // streaming: 117 us over 8 x 16384 tokens of 8 heads, 126 through the caches
    __builtin_nontemporal_store(u32x4{o.x, o.y, o.z, o.w}, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i));
  }
}

// One workgroup per (sequence, block, head, keys | values).  A lane writes
// eight dimensions of a token at a time; values come through LDS, words of four
// tokens of a dimension, eight of which it transposes in registers.
template <int OT, int FMT, int D>
__global__ __launch_bounds__(256) void kv_read_kernel(ReadArgs a) {
  constexpr int kUpt = D / 8;
  extern __shared__ uint8_t lds[];
  const int t = threadIdx.x;
  const int BS = a.cache.block_size, H = a.cache.heads;
  uint32_t g = a.first + blockIdx.x;
  const bool values = g & 1;
  g >>= 1;
  const int head = g % H;
  g /= H;
  const int nth_block = g % a.blocks_per_seq, i = g / a.blocks_per_seq;
  void* out = values ? a.v : a.k;
  if (!out) return;
  const KVSeq s = kv_seq_uniform(a.batch, BS, i);
  if (s.n == 0) return;
  const int block_at = (s.start >> __builtin_ctz(BS)) + nth_block;
  const int p0 = max(s.start, block_at * BS), p1 = min(s.start + s.n, block_at * BS + BS);
  if (p0 >= p1) return;
  const int block = __builtin_amdgcn_readfirstlane(kv_block(a.cache, a.batch, i, block_at));
  const int slot0 = p0 - block_at * BS, slot1 = p1 - block_at * BS;
  const int64_t row0 = s.first - s.start + (int64_t)block_at * BS;  // of slot 0
  const int64_t cell = (int64_t)max(block, 0) * H + head;
  const uint8_t* codes = (values ? a.cache.v : a.cache.k) + cell * BS * D;
  int32_t b = 0;
  if (block >= 0) b = (values ? a.cache.v_bias : a.cache.k_bias)[cell];
  const bool hw = b >= -100 && b <= 100;
  const float scale = __builtin_ldexpf(1.0f, hw ? -b : 0);
  auto at = [&](int slot, int u) { return ((row0 + slot) * H + head) * D + 8 * u; };
  if (!values || block < 0) {
    for (int x = t; x < (slot1 - slot0) * kUpt; x += 256) {
      const int slot = slot0 + x / kUpt, u = x % kUpt;
      uint2 w = make_uint2(0, 0);
      if (block >= 0) w = *reinterpret_cast<const uint2*>(codes + slot * D + 8 * u);
      write8<OT, FMT>(out, at(slot, u), w.x, w.y, b, scale, hw);
    }
    return;
  }
  const int pitch = BS + 4;
  const int shift = __builtin_ctz(BS) - 4;  // 16-byte pieces of a dimension's row
  for (int x = t; x < D << shift; x += 256) {
    const int d = x >> shift, c = 16 * (x & ((1 << shift) - 1));
    const uint4 w = *reinterpret_cast<const uint4*>(codes + d * BS + c);
    uint32_t* o = reinterpret_cast<uint32_t*>(lds + d * pitch + c);
    o[0] = w.x, o[1] = w.y, o[2] = w.z, o[3] = w.w;
  }
  __syncthreads();
  for (int x = t; x < BS / 4 * kUpt; x += 256) {
    const int quad = x / kUpt, u = x % kUpt;
    if (4 * quad + 4 <= slot0 || 4 * quad >= slot1) continue;
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = *reinterpret_cast<const uint32_t*>(lds + (8 * u + e) * pitch + 4 * quad);
      hi[e] = *reinterpret_cast<const uint32_t*>(lds + (8 * u + 4 + e) * pitch + 4 * quad);
    }
    transpose4(lo);
    transpose4(hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int slot = 4 * quad + e;
      if (slot >= slot0 && slot < slot1) write8<OT, FMT>(out, at(slot, u), lo[e], hi[e], b, scale, hw);
    }
  }
}

int lds_bytes(const fp8_kv_cache_t& c) { return c.head_dim * (c.block_size + 4); }

}  // namespace

int64_t kv_append_groups(const fp8_kv_cache_t& c, const fp8_kv_batch_t& b, bool queries) {
  if (b.max_new == 0) return 0;
  const int64_t per = (b.max_new - 1) / c.block_size + 2;
  const int64_t kv = (int64_t)b.batch * c.heads * 2;  // below 2^63: both are 32-bit
  if (kv > ((int64_t)1 << 31) / per) return (int64_t)1 << 31;
  return kv * per + (queries ? (int64_t)b.batch * b.max_new : 0);
}

hipError_t launch_kv_append(const fp8_kv_cache_t& c, const fp8_kv_batch_t& batch, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, int dtype, const void* q, int64_t q_stride, int q_heads,
                            uint16_t* q_out, const float* cos, const float* sin, int rope_rows, int rope_pairs,
                            hipStream_t stream) {
  AppendArgs a{};
  a.cache = c;
  a.batch = batch;
  a.k = k, a.v = v, a.q = q;
  a.k_stride = k_stride, a.v_stride = v_stride, a.q_stride = q_stride;
  a.q_heads = q_heads;
  a.q_out = q_out;
  a.rope = {cos, sin, rope_rows};
  // one new token touches one block; n tokens at most (n - 1) / block_size + 2
  a.blocks_per_seq = batch.max_new == 1 ? 1 : (batch.max_new - 1) / c.block_size + 2;
  a.kv_groups = (int64_t)batch.batch * a.blocks_per_seq * c.heads;
  // queries: about 16384 elements a workgroup
  int64_t groups = a.kv_groups;
  if (q) {
    const int64_t want = 16384 / ((int64_t)q_heads * c.head_dim);
    a.q_tokens = (int)(want < 1 ? 1 : want < batch.max_new ? want : batch.max_new);
    a.q_groups = (batch.max_new + a.q_tokens - 1) / a.q_tokens;
    groups += (int64_t)batch.batch * a.q_groups;
  }
  // lanes: a block's new tokens in kUnits units each (values: its quads of
  // slots), a multiple of a token's units
  const int upt = c.head_dim / 8;
  const int quads = batch.max_new < c.block_size ? (batch.max_new + 2) / 4 + 1 : c.block_size / 4;
  int threads = (quads < c.block_size / 4 ? quads : c.block_size / 4) * upt;
  threads = (threads + 63) / 64 * 64;
  if (q && threads < 256) threads = 256;
  using std::integral_constant;
  auto run = [&](auto dt, auto fmt, auto d, auto rope) {
    in_stretches(groups, threads, [&](uint32_t first, uint32_t count) {
      a.first = first;
      hipLaunchKernelGGL((kv_append_kernel<dt.value, fmt.value, d.value, rope.value>), dim3(count), dim3(threads),
                         lds_bytes(c), stream, a);
    });
  };
  auto with_rope = [&](auto dt, auto fmt, auto d) {
    if (!cos) run(dt, fmt, d, integral_constant<int, kRopeNone>{});
    else if (rope_pairs) run(dt, fmt, d, integral_constant<int, kRopePairs>{});
    else run(dt, fmt, d, integral_constant<int, kRopeHalves>{});
  };
  auto with_dim = [&](auto dt, auto fmt) {
    if (c.head_dim == 64) with_rope(dt, fmt, integral_constant<int, 64>{});
    else if (c.head_dim == 128) with_rope(dt, fmt, integral_constant<int, 128>{});
    else with_rope(dt, fmt, integral_constant<int, 256>{});
  };
  auto with_fmt = [&](auto dt) {
    if (c.fmt == FP8_E4M3) with_dim(dt, integral_constant<int, FP8_E4M3>{});
    else with_dim(dt, integral_constant<int, FP8_E5M2>{});
  };
  if (dtype == FP8_IN_FP32) with_fmt(integral_constant<int, FP8_IN_FP32>{});
  else with_fmt(integral_constant<int, FP8_IN_BF16>{});
  return hipGetLastError();
}

hipError_t launch_kv_read(const fp8_kv_cache_t& c, const fp8_kv_batch_t& batch, int out_dtype, void* k, void* v,
                          hipStream_t stream) {
  ReadArgs a{c, batch, k, v, (batch.max_new - 1) / c.block_size + 2, 0};
  const int64_t groups = (int64_t)batch.batch * a.blocks_per_seq * c.heads * 2;
  using std::integral_constant;
  auto run = [&](auto dt, auto fmt, auto d) {
    in_stretches(groups, 256, [&](uint32_t first, uint32_t count) {
      a.first = first;
      hipLaunchKernelGGL((kv_read_kernel<dt.value, fmt.value, d.value>), dim3(count), dim3(256), lds_bytes(c), stream,
                         a);
    });
  };
  auto with_dim = [&](auto dt, auto fmt) {
    if (c.head_dim == 64) run(dt, fmt, integral_constant<int, 64>{});
    else if (c.head_dim == 128) run(dt, fmt, integral_constant<int, 128>{});
    else run(dt, fmt, integral_constant<int, 256>{});
  };
  auto with_fmt = [&](auto dt) {
    if (c.fmt == FP8_E4M3) with_dim(dt, integral_constant<int, FP8_E4M3>{});
    else with_dim(dt, integral_constant<int, FP8_E5M2>{});
  };
  if (out_dtype == FP8_IN_FP32) with_fmt(integral_constant<int, FP8_IN_FP32>{});
  else with_fmt(integral_constant<int, FP8_IN_BF16>{});
  return hipGetLastError();
}

}  // namespace fp8lin
