// Heads of queries and keys taken apart for the rotary positions: loads, the
// pairing of dimensions, and the rotation itself (kv_cache.hip, qk_norm.hip).
#pragma once

#include "fp8_code.h"
#include "internal.h"

namespace fp8lin {
namespace {

// 4 elements at p + i as fp32.
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

// How keys and queries are rotated.
constexpr int kRopeNone = 0, kRopeHalves = 1, kRopePairs = 2;

// A unit of a head's dimensions: [4u, +4) and [D/2 + 4u, +4), which the halves'
// rotation pairs; the lanes of a load read consecutive bytes.
template <int D>
__device__ __forceinline__ int unit_lo(int u) { return 4 * u; }
template <int D>
__device__ __forceinline__ int unit_hi(int u) { return D / 2 + 4 * u; }

struct Rope {
  const float* cos;
  const float* sin;
  int rows;
};

// The cosines (angle[0..3]) and sines (angle[4..7]) of a unit of the token at
// `pos`: loaded with the token itself.
template <int D, int ROPE>
__device__ __forceinline__ void load_angles(float (&angle)[8], int u, int pos, const Rope& r) {
  if constexpr (ROPE == kRopeNone) return;
  const int64_t row = (int64_t)min(pos, r.rows - 1) * (D / 2);
  if constexpr (ROPE == kRopeHalves) {
    load4<FP8_IN_FP32>(r.cos, row + 4 * u, angle);
    load4<FP8_IN_FP32>(r.sin, row + 4 * u, angle + 4);
  } else {
    const float2 c0 = *reinterpret_cast<const float2*>(r.cos + row + 2 * u);
    const float2 c1 = *reinterpret_cast<const float2*>(r.cos + row + D / 4 + 2 * u);
    const float2 s0 = *reinterpret_cast<const float2*>(r.sin + row + 2 * u);
    const float2 s1 = *reinterpret_cast<const float2*>(r.sin + row + D / 4 + 2 * u);
    angle[0] = c0.x, angle[1] = c0.y, angle[2] = c1.x, angle[3] = c1.y;
    angle[4] = s0.x, angle[5] = s0.y, angle[6] = s1.x, angle[7] = s1.y;
  }
}

// Rotates one unit in place.  Products and sums are rounded separately, as the
// definition has them.
template <int ROPE>
__device__ __forceinline__ void rotate(float (&v)[8], const float (&angle)[8]) {
#pragma clang fp contract(off)
  if constexpr (ROPE == kRopeNone) return;
  const float* c = angle;
  const float* s = angle + 4;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float& x = ROPE == kRopePairs ? v[2 * e] : v[e];
    float& y = ROPE == kRopePairs ? v[2 * e + 1] : v[4 + e];
    const float a = x, b = y;
    const float ac = a * c[e], bs = b * s[e], bc = b * c[e], as = a * s[e];
    x = ac - bs;
    y = bc + as;
  }
}

}  // namespace
}  // namespace fp8lin
