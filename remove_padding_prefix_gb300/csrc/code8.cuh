// 8-bit codes of the quantised key-value cache and their scales.
//
// A block of tokens of one head shares a scale byte b: a code c stands for c * 2^(b - 127), b = 255 for NaN.  Powers of
// two, because a block takes its tokens one at a time: each time a larger one raises the scale, the codes it has are
// rounded again, at twice the step or more, so all roundings of a value together stay within one last step
// (1/2 + 1/4 + ...), where scales that creep up would add half a step each time.  The products with them
// are exact, so the values are the same to the bit wherever they are computed; int8 gives up to one of its bits
// for it, e4m3 nothing.
#pragma once
#include "common.cuh"

namespace rpp {

// the largest code, and what is half a step past it
template <bool kI8> struct Code8 {
  static constexpr float kTop = kI8 ? 127.f : 448.f;
  static constexpr float kPast = kI8 ? 127.5f : 464.f;
  static constexpr int kLog = kI8 ? 6 : 8;      // 2^kLog <= kTop < 2^(kLog + 1)
};

// 2^(b - 127), NaN of 255
__device__ __forceinline__ float scale_of(int b) {
  return b == 255 ? __int_as_float(0x7fffffff) : __int_as_float(b > 0 ? b << 23 : 1 << 22);
}
// 2^(127 - b) of a byte below 255
__device__ __forceinline__ float inverse_of(int b) { return __int_as_float(b < 254 ? (254 - b) << 23 : 1 << 22); }
// 2^-n, 0 from n = 127 on (n >= 0)
__device__ __forceinline__ float pow2_neg(int n) { return n < 127 ? __int_as_float((127 - n) << 23) : 0.f; }

// The scale byte of values up to `most` >= 0: the smallest at which most / scale is no more than kPast.
template <bool kI8>
__device__ __forceinline__ int scale_byte(float most) {
  const int field = __float_as_int(most) >> 23;
  if (field == 255) return 255;
  const int b = max(field - Code8<kI8>::kLog, 0);
  return b + (most * inverse_of(b) > Code8<kI8>::kPast ? 1 : 0);
}

// four values in steps -> four codes, rounded half to even, saturated
template <bool kI8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (kI8) {
    // 1.5 * 2^23 added: the sum's last bits are the rounded integer
    constexpr float kMagic = 12582912.f, kTop = Code8<true>::kTop;
    const uint32_t x = __float_as_uint(fminf(fmaxf(a, -kTop), kTop) + kMagic);
    const uint32_t y = __float_as_uint(fminf(fmaxf(b, -kTop), kTop) + kMagic);
    const uint32_t z = __float_as_uint(fminf(fmaxf(c, -kTop), kTop) + kMagic);
    const uint32_t w = __float_as_uint(fminf(fmaxf(d, -kTop), kTop) + kMagic);
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  } else {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
  }
}

// The codes of a word as two f16 pairs (exact): bytes 0, 1 and bytes 2, 3.  int8: the byte plus 128 as the last bits of a
// half of 1024 to 2047, less 1152.
template <bool kI8>
__device__ __forceinline__ uint2 decode4(uint32_t w) {
  uint2 r;
  if constexpr (kI8) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __floats2half2_rn(1152.f, 1152.f);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), off);
    r.x = *reinterpret_cast<const uint32_t*>(&a);
    r.y = *reinterpret_cast<const uint32_t*>(&b);
  } else {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(w));
  }
  return r;
}
// and as four floats
template <bool kI8>
__device__ __forceinline__ float4 decode4f(uint32_t w) {
  const uint2 r = decode4<kI8>(w);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

}  // namespace rpp
