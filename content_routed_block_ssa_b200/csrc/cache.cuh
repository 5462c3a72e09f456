// Codes and scales of the paged 8-bit cache.  A page's values of one kv-head
// are e4m3 codes times one power of two 2^e: with a power of two the division
// is exact, and a page whose scale grows keeps its stored mantissas.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace ssa {

constexpr int kExpMin = -40, kExpMax = 120;   // 448 * 2^120 exceeds every float

// The least e with amax <= 448 * 2^e (448 = 1.75 * 2^8), clamped.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kExpMin), kExpMax);   // zero and subnormals fall below the clamp
}

__device__ __forceinline__ float pow2(int e) {   // e in -126 .. 127, 0 below
  return e < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ int exponent_of(float scale) {
  return static_cast<int>((__float_as_uint(scale) >> 23) & 0xFFu) - 127;
}

// Two floats to two codes (low byte first), nearest even, +-448 at most.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Two codes (the low 16 bits) to two halfs; every code is exact in float16.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(codes));
  return h;
}

// Four codes to two pairs of halfs (the low codes in `lo`).
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

}  // namespace ssa
