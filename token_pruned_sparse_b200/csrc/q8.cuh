// e4m3 conversions shared by the kernels of the 8-bit key/value cache.
#pragma once

#include "tps_internal.cuh"

namespace tps {

constexpr int kScaleBlock = 128;   // tokens that share a scale (per head and tensor)

// Two fp32 values -> packed e4m3x2 (lo in bits 0-7), round to nearest even;
// beyond 448 saturates, NaN becomes the e4m3 NaN.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four fp32 values -> one word of e4m3 codes.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}
// Two fp32 values -> packed f16x2 (lo in bits 0-15), round to nearest even.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes (bits 0-15 of w) -> packed f16x2; exact (e4m3 is a subset of f16).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f2(uint32_t w) {
  float2 f;
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.f32.f16 %0, lo;\ncvt.f32.f16 %1, hi;\n}\n"
      : "=f"(f.x), "=f"(f.y)
      : "r"(w));
  return f;
}

// The smallest 2^e (as fp32) with amax <= 448 * 2^e, e kept in [-100, 100]; 0 for
// amax = 0. 448 = 1.75 * 2^8, so with amax = 1.f * 2^E, e = E - 8 if 1.f <= 1.75
// and E - 7 otherwise: exponent and mantissa bits decide, nothing is rounded.
template <int kLeast = -100, int kMost = 100>
__device__ __forceinline__ float scale_of_amax(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const uint32_t b = __float_as_uint(amax);
  int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < kLeast ? kLeast : (e > kMost ? kMost : e);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// The power of two of a row of Q: as above over all of bf16 (the largest needs 2^120; rows below 448 * 2^-126
// keep fewer bits), and 1 for a row of zeros.
__device__ __forceinline__ float scale_of_row(float amax) { return amax > 0.f ? scale_of_amax<-126, 120>(amax) : 1.f; }

}  // namespace tps
