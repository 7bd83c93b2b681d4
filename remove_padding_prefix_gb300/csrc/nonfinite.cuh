// Helpers for elements that are not finite, for the two decoder attentions.
//
// A weight of the softmax is above 0 for every score but -inf, however far below the largest, so a value
// that is not finite makes every output that sees it what the sum of such values is, whatever the
// weights.  The products do not get there by themselves: 0 * inf is NaN where the arithmetic made the weight 0
// (or a part of it, or the factor of a maximum that moved).  An infinity that came out is right,
// so both kernels look for NaN at the end of their sums, once, and only then at the values again.
#pragma once
#include <type_traits>

#include "common.cuh"

namespace rpp {

// bits 15 and 31 set where the low / high 16-bit float of the word is not finite (its exponent all
// ones, so one more carries out of it); other bits arbitrary
template <typename T>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
  constexpr uint32_t one = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
  return (w & e) + one;
}

// the low / high 16-bit float of a word
template <typename T>
__device__ __forceinline__ float half_of(uint32_t w, int high) {
  const unsigned short h = static_cast<unsigned short>(high ? w >> 16 : w);
  return to_f32(*reinterpret_cast<const T*>(&h));
}

// the largest of three, NaN where one of them is
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// whether a lane's part of a row of D elements, D / 32 at p, holds one that is not finite
template <typename T, int D>
__device__ __forceinline__ bool part_nonfinite(const T* p) {
  uint32_t f;
  if constexpr (D == 64) {
    f = nonfinite2<T>(*reinterpret_cast<const uint32_t*>(p));
  } else {
    static_assert(D == 128, "rows of 64 or 128");
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    f = nonfinite2<T>(w.x) | nonfinite2<T>(w.y);
  }
  return (f & 0x80008000u) != 0;
}

}  // namespace rpp
