// Division of 64-bit counts that nearly always fit 32 bits.
#pragma once

#include "internal.h"

namespace fp8lin {
namespace {

// a / b, both at least 0 and b not 0.  A 64-bit division takes some hundred
// instructions, a 32-bit one some twenty.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((uint64_t)(a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

}  // namespace
}  // namespace fp8lin
