// The paged FP8 cache of keys and values: written as tokens arrive, and read
// back (include/fp8lin_block.h has the definitions).
//
// Append.  One workgroup per (sequence, touched block, head, keys | values)
// holds that block's new tokens in registers between their largest magnitude
// and the codes, so they are read once; the rotation is applied on the way.
// Values change their order (tokens by dimensions -> dimensions by tokens)
// through LDS bytes.  Further workgroups of the same launch rotate the
// queries, one token each.  HBM-bound for prompts; for single tokens the
// launch is most of the time.
#include <type_traits>

#include "fp8_code.h"
#include "internal.h"
#include "kv_device.h"

namespace fp8lin {
namespace {

// 8 elements at p (16-byte aligned) as fp32.
template <int DT>
__device__ __forceinline__ void load4(const void* p, int64_t i, float* v) {
  if constexpr (DT == FP8_IN_FP32) {
    const float4 t = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
  } else {
    const uint2 t = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    v[0] = __uint_as_float(t.x << 16);
    v[1] = __uint_as_float(t.x & 0xFFFF0000u);
    v[2] = __uint_as_float(t.y << 16);
    v[3] = __uint_as_float(t.y & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint2 bf16x4(const float* v) { return make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3])); }

struct Rope {
  const float* cos;  // null: no rotation
  const float* sin;
  int rows;
  int pairs;
};

// A unit of a head's dimensions: two groups of four.  Rotated halves: [4u, +4)
// and [D/2 + 4u, +4); otherwise [8u, +8).
__device__ __forceinline__ int unit_lo(int u, bool halves) { return halves ? 4 * u : 8 * u; }
__device__ __forceinline__ int unit_hi(int u, bool halves, int D) { return halves ? D / 2 + 4 * u : 8 * u + 4; }

// Rotates one unit of the token at `pos` in place.  Products and sums are
// rounded separately, as the definition has them.
__device__ __forceinline__ void rotate(float (&v)[8], int u, int pos, int D, const Rope& r) {
#pragma clang fp contract(off)
  const int64_t row = (int64_t)min(pos, r.rows - 1) * (D / 2);
  float c[4], s[4];
  load4<FP8_IN_FP32>(r.cos, row + 4 * u, c);
  load4<FP8_IN_FP32>(r.sin, row + 4 * u, s);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float& x = r.pairs ? v[2 * e] : v[e];
    float& y = r.pairs ? v[2 * e + 1] : v[4 + e];
    const float a = x, b = y;
    const float ac = a * c[e], bs = b * s[e], bc = b * c[e], as = a * s[e];
    x = ac - bs;
    y = bc + as;
  }
}

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
};

constexpr int kUnits = 4;  // units a lane holds

template <int DT, int FMT>
__global__ __launch_bounds__(1024) void kv_append_kernel(AppendArgs a) {
  extern __shared__ uint8_t lds[];  // values' codes, [D][block_size + 4]
  __shared__ uint32_t part[16];
  const int nt = blockDim.x, t = threadIdx.x;
  const int D = a.cache.head_dim, BS = a.cache.block_size, H = a.cache.heads;

  if ((int64_t)blockIdx.x >= a.kv_groups) {  // one token's queries
    const int64_t g = (int64_t)blockIdx.x - a.kv_groups;
    const int i = (int)(g / a.batch.max_new), nth = (int)(g % a.batch.max_new);
    const KVSeq s = kv_seq_uniform(a.batch, BS, i);
    if (nth >= s.n) return;
    const bool halves = a.rope.cos && !a.rope.pairs;
    const int64_t row = s.first + nth;
    const int units = a.q_heads * (D / 8);
    for (int x = t; x < units; x += nt) {
      const int head = x / (D / 8), u = x % (D / 8);
      const int lo = unit_lo(u, halves), hi = unit_hi(u, halves, D);
      float v[8];
      load4<DT>(a.q, row * a.q_stride + head * D + lo, v);
      load4<DT>(a.q, row * a.q_stride + head * D + hi, v + 4);
      if (a.rope.cos) rotate(v, u, s.start + nth, D, a.rope);
      uint16_t* o = a.q_out + (row * a.q_heads + head) * D;
      *reinterpret_cast<uint2*>(o + lo) = bf16x4(v);
      *reinterpret_cast<uint2*>(o + hi) = bf16x4(v + 4);
    }
    return;
  }

  int64_t g = blockIdx.x;
  const bool values = g & 1;
  g >>= 1;
  const int head = (int)(g % H);
  g /= H;
  const int nth_block = (int)(g % a.blocks_per_seq), i = (int)(g / a.blocks_per_seq);
  const KVSeq s = kv_seq_uniform(a.batch, BS, i);
  if (s.n == 0) return;
  const int block_at = s.start / BS + nth_block;          // of the sequence
  const int p0 = max(s.start, block_at * BS);             // first new position in the block
  const int p1 = min(s.start + s.n, block_at * BS + BS);  // one past the last
  if (p0 >= p1) return;
  const int block = kv_block(a.cache, a.batch, i, block_at);
  if (block < 0) return;
  const int slot0 = p0 - block_at * BS, count = p1 - p0;

  const bool rot = a.rope.cos && !values;
  const bool halves = rot && !a.rope.pairs;
  const void* src = values ? a.v : a.k;
  const int64_t stride = values ? a.v_stride : a.k_stride;
  const int64_t row0 = s.first + (p0 - s.start);
  const int upt = D / 8, units = count * upt;
  float v[kUnits][8];
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    const int x = q * nt + t;
    if (x < units) {
      const int tok = x / upt, u = x % upt;
      const int64_t at = (row0 + tok) * stride + head * D;
      load4<DT>(src, at + unit_lo(u, halves), v[q]);
      load4<DT>(src, at + unit_hi(u, halves, D), v[q] + 4);
    }
  }
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    const int x = q * nt + t;
    if (x < units) {
      if (rot) rotate(v[q], x % upt, p0 + x / upt, D, a.rope);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, finite_mag(v[q][e]));
    }
  }
  for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  if ((t & 63) == 0) part[t >> 6] = m;
  __syncthreads();
  for (int w = 0; w < nt / 64; ++w) m = max(m, part[w]);

  int32_t* bias = (values ? a.cache.v_bias : a.cache.k_bias) + (int64_t)block * H + head;
  uint8_t* codes = (values ? a.cache.v : a.cache.k) + ((int64_t)block * H + head) * BS * D;
  int32_t b = m == 0 ? FP8_KV_MAX_BIAS : min(FP8_KV_MAX_BIAS, bias_from_amax_bits(m, FMT, 0));
  if (slot0 > 0) {
    const int32_t old = *bias;
    b = min(b, old);
    if (b < old) {  // the tokens that were there, at the new scale
      const int32_t step = b < old - 300 ? -300 : b - old;
      for (int x = t; x < slot0 * D; x += nt) {
        uint8_t* c = codes + (values ? (x / slot0) * BS + x % slot0 : x);
        const uint32_t old_code = *c;
        if ((old_code & 0x7Fu) < (FMT == FP8_E4M3 ? 0x7Fu : 0x7Cu))  // NaN and infinity stay
          *c = (uint8_t)fp8_code<FMT>(__float_as_uint(code_value<FMT>(old_code)), step);
      }
    }
    __syncthreads();  // every lane has read the old bias
  }
  if (t == 0) *bias = b;

  if (!values) {
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
      const int x = q * nt + t;
      if (x < units) {
        const int tok = x / upt, u = x % upt;
        const float(&lo)[4] = *reinterpret_cast<const float(*)[4]>(v[q]);
        const float(&hi)[4] = *reinterpret_cast<const float(*)[4]>(v[q] + 4);
        uint8_t* o = codes + (slot0 + tok) * D;
        *reinterpret_cast<uint32_t*>(o + unit_lo(u, halves)) = codes4_f32<FMT>(lo, b);
        *reinterpret_cast<uint32_t*>(o + unit_hi(u, halves, D)) = codes4_f32<FMT>(hi, b);
      }
    }
    return;
  }
  const int pitch = BS + 4;
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    const int x = q * nt + t;
    if (x < units) {
      const int tok = x / upt, u = x % upt;
      const float(&lo)[4] = *reinterpret_cast<const float(*)[4]>(v[q]);
      const float(&hi)[4] = *reinterpret_cast<const float(*)[4]>(v[q] + 4);
      const uint32_t c0 = codes4_f32<FMT>(lo, b), c1 = codes4_f32<FMT>(hi, b);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lds[(8 * u + e) * pitch + slot0 + tok] = (uint8_t)(c0 >> (8 * e));
        lds[(8 * u + 4 + e) * pitch + slot0 + tok] = (uint8_t)(c1 >> (8 * e));
      }
    }
  }
  __syncthreads();
  const int slot1 = slot0 + count;
  if (count == 1) {
    for (int d = t; d < D; d += nt) codes[d * BS + slot0] = lds[d * pitch + slot0];
    return;
  }
  for (int x = t; x < D * (BS / 4); x += nt) {
    const int d = x / (BS / 4), c = 4 * (x % (BS / 4));
    if (c >= slot0 && c + 4 <= slot1) {
      *reinterpret_cast<uint32_t*>(codes + d * BS + c) = *reinterpret_cast<const uint32_t*>(lds + d * pitch + c);
    } else {
      for (int e = 0; e < 4; ++e)
        if (c + e >= slot0 && c + e < slot1) codes[d * BS + c + e] = lds[d * pitch + c + e];
    }
  }
}

// ---------------------------------------------------------------- read
struct ReadArgs {
  fp8_kv_cache_t cache;
  fp8_kv_batch_t batch;
  void* k;
  void* v;
  int blocks_per_seq;
};

// 8 codes (two dwords) at bias b -> out_dtype at o.
template <int OT, int FMT>
__device__ __forceinline__ void write8(void* p, int64_t i, uint32_t c0, uint32_t c1, int32_t b) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = __builtin_ldexpf(code_value<FMT>((c0 >> (8 * e)) & 0xFFu), -b);
    v[4 + e] = __builtin_ldexpf(code_value<FMT>((c1 >> (8 * e)) & 0xFFu), -b);
  }
  if constexpr (OT == FP8_IN_FP32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    const uint2 lo = bf16x4(v), hi = bf16x4(v + 4);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
}

template <int OT, int FMT>
__global__ __launch_bounds__(256) void kv_read_kernel(ReadArgs a) {
  extern __shared__ uint8_t lds[];
  const int t = threadIdx.x;
  const int D = a.cache.head_dim, BS = a.cache.block_size, H = a.cache.heads;
  int64_t g = blockIdx.x;
  const bool values = g & 1;
  g >>= 1;
  const int head = (int)(g % H);
  g /= H;
  const int nth_block = (int)(g % a.blocks_per_seq), i = (int)(g / a.blocks_per_seq);
  void* out = values ? a.v : a.k;
  if (!out) return;
  const KVSeq s = kv_seq_uniform(a.batch, BS, i);
  if (s.n == 0) return;
  const int block_at = s.start / BS + nth_block;
  const int p0 = max(s.start, block_at * BS), p1 = min(s.start + s.n, block_at * BS + BS);
  if (p0 >= p1) return;
  const int block = kv_block(a.cache, a.batch, i, block_at);
  const int slot0 = p0 - block_at * BS, count = p1 - p0;
  const int64_t row0 = s.first + (p0 - s.start);
  const int upt = D / 8, units = count * upt;
  const int64_t cell = (int64_t)max(block, 0) * H + head;
  const uint8_t* codes = (values ? a.cache.v : a.cache.k) + cell * BS * D;
  int32_t b = 0;
  if (block >= 0) b = (values ? a.cache.v_bias : a.cache.k_bias)[cell];
  const int pitch = BS + 4;
  if (values && block >= 0) {
    for (int x = t; x < D * (BS / 16); x += 256) {
      const int d = x / (BS / 16), c = 16 * (x % (BS / 16));
      const uint4 w = *reinterpret_cast<const uint4*>(codes + d * BS + c);
      uint32_t* o = reinterpret_cast<uint32_t*>(lds + d * pitch + c);
      o[0] = w.x, o[1] = w.y, o[2] = w.z, o[3] = w.w;
    }
    __syncthreads();
  }
  for (int x = t; x < units; x += 256) {
    const int tok = x / upt, u = x % upt;
    uint32_t c0 = 0, c1 = 0;
    if (block >= 0) {
      if (values) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c0 |= (uint32_t)lds[(8 * u + e) * pitch + slot0 + tok] << (8 * e);
          c1 |= (uint32_t)lds[(8 * u + 4 + e) * pitch + slot0 + tok] << (8 * e);
        }
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(codes + (slot0 + tok) * D + 8 * u);
        c0 = w.x, c1 = w.y;
      }
    }
    write8<OT, FMT>(out, ((row0 + tok) * H + head) * D + 8 * u, c0, c1, b);
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
  AppendArgs a{c, batch, k, v, q, k_stride, v_stride, q_stride, q_heads, q_out, {cos, sin, rope_rows, rope_pairs}, 0, 0};
  // one new token touches one block; n tokens at most (n - 1) / block_size + 2
  a.blocks_per_seq = batch.max_new == 1 ? 1 : (batch.max_new - 1) / c.block_size + 2;
  a.kv_groups = (int64_t)batch.batch * a.blocks_per_seq * c.heads * 2;
  const int64_t groups = a.kv_groups + (q ? (int64_t)batch.batch * batch.max_new : 0);
  // lanes: a block's new tokens in kUnits units each
  const int units = (batch.max_new < c.block_size ? batch.max_new : c.block_size) * (c.head_dim / 8);
  int threads = (units + kUnits - 1) / kUnits;
  threads = threads < 256 ? (q ? 256 : (threads + 63) / 64 * 64) : (threads + 63) / 64 * 64;
  auto run = [&](auto dt, auto fmt) {
    hipLaunchKernelGGL((kv_append_kernel<dt.value, fmt.value>), dim3((uint32_t)groups), dim3(threads), lds_bytes(c),
                       stream, a);
  };
  using std::integral_constant;
  if (dtype == FP8_IN_FP32) {
    if (c.fmt == FP8_E4M3) run(integral_constant<int, FP8_IN_FP32>{}, integral_constant<int, FP8_E4M3>{});
    else run(integral_constant<int, FP8_IN_FP32>{}, integral_constant<int, FP8_E5M2>{});
  } else {
    if (c.fmt == FP8_E4M3) run(integral_constant<int, FP8_IN_BF16>{}, integral_constant<int, FP8_E4M3>{});
    else run(integral_constant<int, FP8_IN_BF16>{}, integral_constant<int, FP8_E5M2>{});
  }
  return hipGetLastError();
}

hipError_t launch_kv_read(const fp8_kv_cache_t& c, const fp8_kv_batch_t& batch, int out_dtype, void* k, void* v,
                          hipStream_t stream) {
  ReadArgs a{c, batch, k, v, (batch.max_new - 1) / c.block_size + 2};
  const int64_t groups = (int64_t)batch.batch * a.blocks_per_seq * c.heads * 2;
  auto run = [&](auto dt, auto fmt) {
    hipLaunchKernelGGL((kv_read_kernel<dt.value, fmt.value>), dim3((uint32_t)groups), dim3(256), lds_bytes(c), stream,
                       a);
  };
  using std::integral_constant;
  if (out_dtype == FP8_IN_FP32) {
    if (c.fmt == FP8_E4M3) run(integral_constant<int, FP8_IN_FP32>{}, integral_constant<int, FP8_E4M3>{});
    else run(integral_constant<int, FP8_IN_FP32>{}, integral_constant<int, FP8_E5M2>{});
  } else {
    if (c.fmt == FP8_E4M3) run(integral_constant<int, FP8_IN_BF16>{}, integral_constant<int, FP8_E4M3>{});
    else run(integral_constant<int, FP8_IN_BF16>{}, integral_constant<int, FP8_E5M2>{});
  }
  return hipGetLastError();
}

}  // namespace fp8lin
