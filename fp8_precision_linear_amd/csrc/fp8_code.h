// FP8 codes and scaling biases on gfx950: the bias of an amax, the rounding of
// one fp32 value to a code, and the hardware conversion of four of them.
// Shared by every kernel that writes codes.
#pragma once

#include "internal.h"

namespace fp8lin {
namespace {

// ---------------------------------------------------------------- bias
// floor(log2(fmt_max / A)) - margin with fmt_max = t * 2^emax, t = 1.75 for
// E4M3 (448) and E5M2 (57344), 1.875 for E3M4 (30).  Writing A = (1 + f) * 2^e
// with f in [0, 1): fmt_max / A = t / (1 + f) * 2^(emax - e) and t / (1 + f)
// lies in (t / 2, t], so its floor(log2) is 0 when 1 + f <= t (fraction field
// <= 0x600000, resp. 0x700000) and -1 otherwise.
__device__ __forceinline__ int32_t bias_from_amax_bits(uint32_t a, int fmt, int32_t margin) {
  if (a == 0u || a >= 0x7F800000u) return 0;  // zero, inf, NaN (or a negative input)
  int e;
  uint32_t frac;
  if ((a >> 23) == 0u) {  // subnormal: normalise on the leading one
    const int p = 31 - __clz(a);
    e = p - 149;
    frac = (a << (23 - p)) & 0x7FFFFFu;
  } else {
    e = (int)(a >> 23) - 127;
    frac = a & 0x7FFFFFu;
  }
  const int emax = fmt == FP8_E4M3 ? 8 : (fmt == FP8_E5M2 ? 15 : 4);
  const uint32_t tfrac = fmt == FP8_E3M4 ? 0x700000u : 0x600000u;
  return emax - e - (frac > tfrac ? 1 : 0) - margin;
}

// ---------------------------------------------------------------- cast
// x * 2^b is formed exactly with ldexp: fp32 denormals are kept (the kernels
// run with denormal mode "preserve"), results at or above 2^-126 are exact,
// smaller ones cast to a signed zero in both formats anyway, and results past
// the fp32 range become inf, which saturates like any value above fmt_max.
// The magnitude bits a of the scaled value are then rounded to the format:
//   normal range    round-to-nearest-even on the dropped fraction bits, the
//                   exponent re-biased by one constant (a carry moves into the
//                   next binade on its own);
//   subnormal range adding 2^(23 + emin - mbits) -- the power of two whose
//                   fp32 ulp is the format's smallest subnormal -- lets the
//                   fp32 adder round to that quantum; the integer difference
//                   of the bit patterns is the code;
// then saturation at the largest finite code and NaN -> 0x7F, sign copied.
template <int FMT>
__device__ __forceinline__ uint32_t fp8_code(uint32_t xbits, int32_t b) {
  const uint32_t vb = __float_as_uint(__builtin_ldexpf(__uint_as_float(xbits), b));
  const uint32_t a = vb & 0x7FFFFFFFu;
  uint32_t code;
  if constexpr (FMT == FP8_E4M3) {
    // normal: code = (fp32 exponent - 120) * 8 + top 3 fraction bits, rounded
    const uint32_t nrm = (a + (0x7FFFFu - 0x3C000000u) + ((a >> 20) & 1u)) >> 20;
    // subnormal (|v| < 2^-6): the ulp of 2^14 in fp32 is 2^-9
    const uint32_t sub = __float_as_uint(__uint_as_float(a) + 16384.0f) - 0x46800000u;
    code = a < 0x3C800000u ? sub : nrm;
    code = min(code, 0x7Eu);
  } else if constexpr (FMT == FP8_E5M2) {
    // normal: code = (fp32 exponent - 112) * 4 + top 2 fraction bits, rounded
    const uint32_t nrm = (a + (0xFFFFFu - 0x38000000u) + ((a >> 21) & 1u)) >> 21;
    // subnormal (|v| < 2^-14): the ulp of 2^7 in fp32 is 2^-16
    const uint32_t sub = __float_as_uint(__uint_as_float(a) + 128.0f) - 0x43000000u;
    code = a < 0x38800000u ? sub : nrm;
    code = min(code, 0x7Bu);
  } else {
    static_assert(FMT == FP8_E3M4, "unknown format");
    // normal: code = (fp32 exponent - 124) * 16 + top 4 fraction bits, rounded
    const uint32_t nrm = (a + (0x3FFFFu - 0x3E000000u) + ((a >> 19) & 1u)) >> 19;
    // subnormal (|v| < 2^-2): the ulp of 2^17 in fp32 is 2^-6
    const uint32_t sub = __float_as_uint(__uint_as_float(a) + 131072.0f) - 0x48000000u;
    code = a < 0x3E800000u ? sub : nrm;
    code = min(code, 0x7Eu);  // 30; the code above it is NaN
  }
  code = a > 0x7F800000u ? 0x7Fu : code;
  return code | ((vb >> 24) & 0x80u);
}

template <int FMT>
__device__ __forceinline__ uint32_t pack4_f32(uint4 v, int32_t b) {
  return fp8_code<FMT>(v.x, b) | (fp8_code<FMT>(v.y, b) << 8) | (fp8_code<FMT>(v.z, b) << 16) |
         (fp8_code<FMT>(v.w, b) << 24);
}

// ---------------------------------------------------------------- cast, hardware conversion
// gfx950's v_cvt_scalef32_pk_{fp8,bf8}_bf16 converts two bf16 values x to the
// FP8 codes of x / scale with round-to-nearest-even.  Measured against the
// rounding defined above on every bf16 pattern and every scale 2^k,
// k = -126..127: bit-identical for every finite input whose scaled value does
// not exceed the format's largest finite value; beyond it the instruction
// returns NaN / inf codes instead of saturating, and its NaN and inf codes
// differ from the ones defined here.  So, with scale = 2^-b (a normal float
// for b in [-127, 126]):
//  * finite inputs are first clamped in magnitude to fmt_max * 2^-b (a packed
//    16-bit integer min on the magnitude bits: for non-negative IEEE values
//    integer order is value order), which turns overflow into exactly the
//    saturation the rounding above performs (every value at or beyond
//    fmt_max rounds to the largest finite code);
//  * a unit holding any inf or NaN is redone with fp8_code.
// E3M4 has no such conversion and always takes fp8_code.
constexpr int kHwBiasMin = -127, kHwBiasMax = 126;
template <int FMT>
constexpr bool kHwConvert = FMT == FP8_E4M3 || FMT == FP8_E5M2;

typedef short hw_v2s __attribute__((ext_vector_type(2)));
typedef __bf16 hw_v2bf __attribute__((ext_vector_type(2)));

// fp32 magnitude bits of min(fmt_max * 2^-b, largest finite fp32); fmt_max =
// 1.75 * 2^emax has fp32 fraction bits 0x600000.
template <int FMT>
__device__ __forceinline__ uint32_t hw_bound_f32(int32_t b) {
  static_assert(kHwConvert<FMT>, "no hardware conversion for this format");
  const int efield = (FMT == FP8_E4M3 ? 8 : 15) + 127 - b;
  return efield >= 255 ? 0x7F7FFFFFu : (((uint32_t)efield << 23) | 0x600000u);
}

// Four fp32 values -> four codes with v_cvt_scalef32_pk_{fp8,bf8}_f32, the
// magnitudes clamped to fmt_max * 2^-b first (as for bf16 inputs); mx keeps
// the largest magnitude seen, for the non-finite check.
template <int FMT>
__device__ __forceinline__ uint32_t pack4_f32_hw(uint4 v, uint32_t bound, float scale, uint32_t& mx) {
  const uint32_t m0 = v.x & 0x7FFFFFFFu, m1 = v.y & 0x7FFFFFFFu;
  const uint32_t m2 = v.z & 0x7FFFFFFFu, m3 = v.w & 0x7FFFFFFFu;
  mx = max(mx, max(max(m0, m1), max(m2, m3)));
  const float c0 = __uint_as_float((v.x & 0x80000000u) | min(m0, bound));
  const float c1 = __uint_as_float((v.y & 0x80000000u) | min(m1, bound));
  const float c2 = __uint_as_float((v.z & 0x80000000u) | min(m2, bound));
  const float c3 = __uint_as_float((v.w & 0x80000000u) | min(m3, bound));
  hw_v2s r = {0, 0};
  if constexpr (FMT == FP8_E4M3) {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c0, c1, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c2, c3, scale, true);
  } else {
    r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, c0, c1, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, c2, c3, scale, true);
  }
  return __builtin_bit_cast(uint32_t, r);
}

// Four fp32 values -> four codes at bias b: the hardware conversion where hw
// (b in [kHwBiasMin, kHwBiasMax]), groups with an inf or NaN by fp8_code.
template <int FMT>
__device__ __forceinline__ uint32_t cast4_f32(uint4 v, bool hw, int32_t b, uint32_t bound, float scale) {
  if constexpr (kHwConvert<FMT>) {
    if (hw) {
      uint32_t mx = 0;
      const uint32_t o = pack4_f32_hw<FMT>(v, bound, scale, mx);
      if (mx < 0x7F800000u) return o;
    }
  }
  return pack4_f32<FMT>(v, b);
}


// Two fp32 values -> two bf16 words, rounded to nearest even (v_cvt_pk_bf16_f32;
// NaN stays NaN).
typedef float hw_v2f __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((hw_v2f{a, b}), hw_v2bf));
}

// Four fp32 values -> the four codes of v * 2^b, as fp8_code gives them, for a
// bias known beforehand.  The values are clamped to fmt_max * 2^-b, which is
// the saturation (infinities too), and converted at the scale 2^-b; where that
// or the bound is no normal number they are scaled first, exactly.  A NaN, which the clamp
// would lose, shows in the sum of the four (as may infinities of both signs):
// such a group takes fp8_code.
template <int FMT>
struct Coder {
  static_assert(kHwConvert<FMT>, "no hardware conversion for this format");
  int32_t b;
  bool first;  // scale first
  float bound, scale;
  __device__ __forceinline__ explicit Coder(int32_t bias) : b(bias) {
    first = b < (FMT == FP8_E4M3 ? -119 : -112) || b > kHwBiasMax;
    bound = __uint_as_float(hw_bound_f32<FMT>(first ? 0 : b));
    scale = __builtin_ldexpf(1.0f, first ? 0 : -b);
  }
  __device__ __forceinline__ uint32_t four(const float (&v)[4]) const {
    float c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = v[e];
      if (first) c[e] = __builtin_ldexpf(c[e], b);
      c[e] = __builtin_amdgcn_fmed3f(c[e], -bound, bound);
    }
    hw_v2s r = {0, 0};
    if constexpr (FMT == FP8_E4M3) {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c[0], c[1], scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c[2], c[3], scale, true);
    } else {
      r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, c[0], c[1], scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, c[2], c[3], scale, true);
    }
    uint32_t o = __builtin_bit_cast(uint32_t, r);
    const float sum = (v[0] + v[1]) + (v[2] + v[3]);
    if (__builtin_expect(sum != sum, 0)) {
      o = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) o |= fp8_code<FMT>(__float_as_uint(v[e]), b) << (8 * e);
    }
    return o;
  }
};

}  // namespace
}  // namespace fp8lin
