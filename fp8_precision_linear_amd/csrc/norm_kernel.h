// RMS norm with the residual's addition in front of an FP8 product, forward
// (output in FP8 codes or bf16) and backward.
//
//   h = round(x + r)          rounded to r's type; h = x without a residual
//   rstd = (mean_j h_j^2 + eps)^(-1/2)
//   y_j = (h_j * rstd) * w_j  -> codes of y * 2^bias, or bf16
//   backward, g = dy * w, xhat = h * rstd, c = mean_j g_j xhat_j:
//   dx_j = rstd * (g_j - xhat_j * c) + dh_j       dw_j = sum_rows dy_j * xhat_j
//
// h is rounded before the statistics so that the backward, which has only the
// stored h, differentiates exactly the function the forward computed.  Sums,
// rstd and y are fp32.
//
// HBM-bound: a row (d <= 32768; 16384 where d is not a multiple of 4) stays in
// registers between the sum of squares and the output, so every input is read
// once and every output written once.  One, four, eight or sixteen waves take a
// row, in units of four elements (16 bytes of fp32), two to eight of them in
// flight per lane; sums go through wave shuffles and LDS.
#pragma once

#include <type_traits>

#include "fp8_code.h"
#include "internal.h"

namespace fp8lin {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kNone = -1;  // "no residual" as a type

// A unit is four consecutive elements.  WHOLE: d is a multiple of 4, so every
// row starts on 16-byte boundaries (8 of bf16, 4 of codes) and has whole units
// only.  Otherwise a unit lies at any element -- still one load or store, which
// the hardware takes at any address (8000 x 4099 in 76 us, element by element
// 144; 4000 x 3001 backward in 43, element by element 70) -- and a row's last one may hold fewer: `left`
// elements of the row lie at and after a unit's first.
typedef f32x4 f32x4_loose __attribute__((aligned(4)));
typedef u32x2 u32x2_loose __attribute__((aligned(2)));
typedef uint32_t u32_loose __attribute__((aligned(1)));

// A unit of type DT (FP8_IN_BF16 or FP8_IN_FP32) as it lies in memory, loaded
// past the caches if STREAM (each input is read once), and as fp32.  Elements
// past the row are zeros.
template <int DT>
using Raw = std::conditional_t<DT == FP8_IN_FP32, f32x4, u32x2>;
template <int DT, bool WHOLE, bool STREAM>
__device__ __forceinline__ Raw<DT> load_raw(const void* p, int64_t i, int left) {
  using E = std::conditional_t<DT == FP8_IN_FP32, float, uint16_t>;
  using Loose = std::conditional_t<DT == FP8_IN_FP32, f32x4_loose, u32x2_loose>;
  using At = std::conditional_t<WHOLE, Raw<DT>, Loose>;
  const E* q = static_cast<const E*>(p) + i;
  if (WHOLE || left >= 4) {
    if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const At*>(q));
    else return *reinterpret_cast<const At*>(q);
  }
  Raw<DT> r{};
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    if (e < left) {
      if constexpr (DT == FP8_IN_FP32) r[e] = q[e];
      else r[e >> 1] |= (uint32_t)q[e] << (16 * (e & 1));
    }
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void unpack(const Raw<DT>& r, float (&v)[4]) {
  if constexpr (DT == FP8_IN_FP32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = r[e];
  } else {
    v[0] = __uint_as_float(r[0] << 16);
    v[1] = __uint_as_float(r[0] & 0xFFFF0000u);
    v[2] = __uint_as_float(r[1] << 16);
    v[3] = __uint_as_float(r[1] & 0xFFFF0000u);
  }
}
template <int DT, bool WHOLE>
__device__ __forceinline__ void load_stream(const void* p, int64_t i, int left, float (&v)[4]) {
  unpack<DT>(load_raw<DT, WHOLE, true>(p, i, left), v);
}

// The weight, its type chosen at run time; it comes from a cache.
template <bool WHOLE>
__device__ __forceinline__ void load_weight(const void* p, int dt, int64_t i, int left, float (&v)[4]) {
  if (dt == FP8_IN_FP32) unpack<FP8_IN_FP32>(load_raw<FP8_IN_FP32, WHOLE, false>(p, i, left), v);
  else unpack<FP8_IN_BF16>(load_raw<FP8_IN_BF16, WHOLE, false>(p, i, left), v);
}

template <int DT, bool WHOLE>
__device__ __forceinline__ void store_as(void* p, int64_t i, int left, const float (&v)[4]) {
  using E = std::conditional_t<DT == FP8_IN_FP32, float, uint16_t>;
  using Loose = std::conditional_t<DT == FP8_IN_FP32, f32x4_loose, u32x2_loose>;
  using At = std::conditional_t<WHOLE, Raw<DT>, Loose>;
  E* q = static_cast<E*>(p) + i;
  Raw<DT> r;
  if constexpr (DT == FP8_IN_FP32) r = f32x4{v[0], v[1], v[2], v[3]};
  else r = u32x2{bf16x2(v[0], v[1]), bf16x2(v[2], v[3])};
  if (WHOLE || left >= 4) {
    *reinterpret_cast<At*>(q) = r;
    return;
  }
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    if (e < left) {
      if constexpr (DT == FP8_IN_FP32) q[e] = r[e];
      else q[e] = (uint16_t)(r[e >> 1] >> (16 * (e & 1)));
    }
  }
}

// Rounds v to type DT in place.
template <int DT>
__device__ __forceinline__ void round_to(float (&v)[4]) {
  if constexpr (DT == FP8_IN_BF16) unpack<FP8_IN_BF16>(u32x2{bf16x2(v[0], v[1]), bf16x2(v[2], v[3])}, v);
}

// The largest magnitude (fp32 bits) of m and a unit's elements.
template <bool WHOLE>
__device__ __forceinline__ uint32_t unit_max(uint32_t m, int left, const float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (WHOLE || e < left) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  return m;
}

// The codes of v * 2^b (E4M3 or E5M2).
struct Codes {
  int fmt;
  Coder<FP8_E4M3> e4;
  Coder<FP8_E5M2> e5;
  __device__ __forceinline__ Codes(int fmt_, int32_t b) : fmt(fmt_), e4(b), e5(b) {}
  template <bool WHOLE>
  __device__ __forceinline__ void store(uint8_t* y, int64_t i, int left, const float (&v)[4]) const {
    const uint32_t c = fmt == FP8_E4M3 ? e4.four(v) : e5.four(v);
    if (WHOLE || left >= 4) {
      *reinterpret_cast<std::conditional_t<WHOLE, uint32_t, u32_loose>*>(y + i) = c;
      return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < left) y[i + e] = (uint8_t)(c >> (8 * e));
  }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  return v;
}

// Sum (maximum) over the W waves that share a row, in a fixed order.  `part`:
// W words of LDS that no other reduction in flight uses; one barrier.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = wave_sum(v);
  if constexpr (W == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = part[0];
#pragma unroll
  for (int w = 1; w < W; ++w) s += part[w];
  return s;
}
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part) {
  v = wave_max(v);
  if constexpr (W == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t s = part[0];
#pragma unroll
  for (int w = 1; w < W; ++w) s = max(s, part[w]);
  return s;
}

// Threads of a workgroup whose rows take W waves each: four rows of one wave,
// or one row.
template <int W>
constexpr int kBlock = W == 1 ? 256 : 64 * W;

// The wave's largest magnitude (fp32 bits) into *amax.
__device__ __forceinline__ void fold_amax_wave(uint32_t m, uint32_t* amax) {
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0 && m > __hip_atomic_load(amax, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
    atomicMax(amax, m);
}

__global__ void clear_kernel(uint32_t* p) { *p = 0u; }

// The shapes a row length runs in: whole units or not, U units per lane, W
// waves per row.  Fewer units a lane and more waves a row are faster as long as
// the row's sum does not dominate: rows of 1028 to 2048 on four waves instead of
// one, 28 us against 33 over 8000 x 2048 forward and 25 against 27 over 4095 x
// 2048 backward; rows of 4100 to 8192 on eight instead of four, 94 against 100
// over 8192 x 8192 and 53 against 56 over 4095 x 5120.
template <typename F>
void for_shape(int d, F&& f) {
  using std::bool_constant;
  using std::integral_constant;
  auto units = [&](auto whole) {
    auto go = [&](auto u, auto w) { f(whole, u, w); };
    if (d <= 1024) go(integral_constant<int, 4>{}, integral_constant<int, 1>{});
    else if (d <= 2048) go(integral_constant<int, 2>{}, integral_constant<int, 4>{});
    else if (d <= 4096) go(integral_constant<int, 4>{}, integral_constant<int, 4>{});
    else if (d <= 8192) go(integral_constant<int, 4>{}, integral_constant<int, 8>{});
    else if (d <= 16384) go(integral_constant<int, 4>{}, integral_constant<int, 16>{});
    else if constexpr (decltype(whole)::value) go(integral_constant<int, 8>{}, integral_constant<int, 16>{});
  };
  if (d % 4 == 0) units(bool_constant<true>{});
  else units(bool_constant<false>{});
}

template <typename F>
void for_dtype(int dt, F&& f) {
  using std::integral_constant;
  if (dt == FP8_IN_BF16) f(integral_constant<int, FP8_IN_BF16>{});
  else if (dt == FP8_IN_FP32) f(integral_constant<int, FP8_IN_FP32>{});
  else f(integral_constant<int, kNone>{});
}

}  // namespace
}  // namespace fp8lin
