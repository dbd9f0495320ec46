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
// HBM-bound: a row (d <= 32768; 16384 where d is not a multiple of 4) stays in registers between the sum of squares
// and the output, so every input is read once and every output written once.
// One wave, four or sixteen take a row, 16 bytes per fp32 load and 4 or 8
// units in flight per lane; sums go through wave shuffles and LDS.
#pragma once

#include <type_traits>

#include "fp8_code.h"
#include "internal.h"

namespace fp8lin {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kNone = -1;  // "no residual" as a type

// V consecutive elements of type DT (FP8_IN_BF16 or FP8_IN_FP32) as they lie in
// memory, loaded past the caches (each input is read once), and as fp32.
template <int DT, int V>
using Raw = std::conditional_t<DT == FP8_IN_FP32, std::conditional_t<V == 4, f32x4, float>,
                               std::conditional_t<V == 4, u32x2, uint16_t>>;
template <int DT, int V>
__device__ __forceinline__ Raw<DT, V> load_raw(const void* p, int64_t i) {
  using E = std::conditional_t<DT == FP8_IN_FP32, float, uint16_t>;
  return __builtin_nontemporal_load(reinterpret_cast<const Raw<DT, V>*>(static_cast<const E*>(p) + i));
}
template <int DT, int V>
__device__ __forceinline__ void unpack(const Raw<DT, V>& r, float (&v)[V]) {
  if constexpr (DT == FP8_IN_FP32 && V == 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = r[e];
  } else if constexpr (DT == FP8_IN_FP32) {
    v[0] = r;
  } else if constexpr (V == 4) {
    v[0] = __uint_as_float(r[0] << 16);
    v[1] = __uint_as_float(r[0] & 0xFFFF0000u);
    v[2] = __uint_as_float(r[1] << 16);
    v[3] = __uint_as_float(r[1] & 0xFFFF0000u);
  } else {
    v[0] = __uint_as_float((uint32_t)r << 16);
  }
}
template <int DT, int V>
__device__ __forceinline__ void load_stream(const void* p, int64_t i, float (&v)[V]) {
  unpack<DT, V>(load_raw<DT, V>(p, i), v);
}

// Ordinary loads, the type chosen at run time (the weight, and h on its second
// reading: both come from a cache).
template <int V>
__device__ __forceinline__ void load_cached(const void* p, int dt, int64_t i, float (&v)[V]) {
  if (dt == FP8_IN_FP32) {
    const float* q = static_cast<const float*>(p) + i;
    if constexpr (V == 4) {
      const float4 t = *reinterpret_cast<const float4*>(q);
      v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else {
      v[0] = *q;
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if constexpr (V == 4) {
      const uint2 t = *reinterpret_cast<const uint2*>(q);
      v[0] = __uint_as_float(t.x << 16);
      v[1] = __uint_as_float(t.x & 0xFFFF0000u);
      v[2] = __uint_as_float(t.y << 16);
      v[3] = __uint_as_float(t.y & 0xFFFF0000u);
    } else {
      v[0] = __uint_as_float((uint32_t)*q << 16);
    }
  }
}

template <int DT, int V>
__device__ __forceinline__ void store_as(void* p, int64_t i, const float (&v)[V]) {
  if constexpr (DT == FP8_IN_FP32) {
    float* q = static_cast<float*>(p) + i;
    if constexpr (V == 4)
      *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *q = v[0];
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(q) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
    else
      *q = (uint16_t)bf16x2(v[0], 0.0f);
  }
}

// Rounds v to type DT in place.
template <int DT, int V>
__device__ __forceinline__ void round_to(float (&v)[V]) {
  if constexpr (DT == FP8_IN_BF16) {
    if constexpr (V == 4) {
      const uint32_t a = bf16x2(v[0], v[1]), b = bf16x2(v[2], v[3]);
      v[0] = __uint_as_float(a << 16);
      v[1] = __uint_as_float(a & 0xFFFF0000u);
      v[2] = __uint_as_float(b << 16);
      v[3] = __uint_as_float(b & 0xFFFF0000u);
    } else {
      v[0] = __uint_as_float(bf16x2(v[0], 0.0f) << 16);
    }
  }
}

// The codes of v * 2^b (E4M3 or E5M2).
struct Codes {
  int fmt;
  int32_t b;
  Coder<FP8_E4M3> e4;
  Coder<FP8_E5M2> e5;
  __device__ __forceinline__ Codes(int fmt_, int32_t b_) : fmt(fmt_), b(b_), e4(b_), e5(b_) {}
  template <int V>
  __device__ __forceinline__ void store(uint8_t* y, int64_t i, const float (&v)[V]) const {
    if constexpr (V == 4) {
      *reinterpret_cast<uint32_t*>(y + i) = fmt == FP8_E4M3 ? e4.four(v) : e5.four(v);
    } else {
      const uint32_t u = __float_as_uint(v[0]);
      y[i] = (uint8_t)(fmt == FP8_E4M3 ? fp8_code<FP8_E4M3>(u, b) : fp8_code<FP8_E5M2>(u, b));
    }
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

// The shapes a row length runs in: V elements per unit (4 where rows start on
// 16-byte boundaries whatever their type), W waves per row, U units per lane.
// Fewer units a lane and more waves a row are faster as long as the row's sum
// does not dominate: rows of 1028 to 2048 on four waves instead of one, 28 us
// against 33 over 8000 x 2048 forward and 25 against 27 over 4095 x 2048
// backward; rows of 4100 to 8192 on eight instead of four, 94 against 100 over
// 8192 x 8192 and 53 against 56 over 4095 x 5120.
template <typename F>
void for_shape(int d, F&& f) {
  using std::integral_constant;
#define FP8LIN_SHAPE(V, U, W) \
  f(integral_constant<int, V>{}, integral_constant<int, U>{}, integral_constant<int, W>{})
  if (d % 4 == 0) {
    if (d <= 1024) FP8LIN_SHAPE(4, 4, 1);
    else if (d <= 2048) FP8LIN_SHAPE(4, 2, 4);
    else if (d <= 4096) FP8LIN_SHAPE(4, 4, 4);
    else if (d <= 8192) FP8LIN_SHAPE(4, 4, 8);
    else if (d <= 16384) FP8LIN_SHAPE(4, 4, 16);
    else FP8LIN_SHAPE(4, 8, 16);
  } else {
    if (d <= 2048) FP8LIN_SHAPE(1, 8, 4);
    else FP8LIN_SHAPE(1, 16, 16);
  }
#undef FP8LIN_SHAPE
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
