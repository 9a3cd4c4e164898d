// The cache of keys and values in 8 bits: E4M3 codes in pages, one power-of-two scale (an E8M0 byte,
// exponent + 127) for each page and head.  Conversions shared by kv_e4m3.cu and attn_e4m3.cu.
#pragma once

#include "elem16.cuh"

namespace wq {

// Exponents that kv_e4m3.cu gives a scale: enough for 448 * 2^64, and narrow enough that sums of
// 2^-e over a sequence stay far inside float32 (attn_e4m3.cu).
constexpr int kScaleLow = -64, kScaleHigh = 64, kScaleBias = 127;

// Two E4M3 codes (the low byte first) as two fp16 values, exact.  NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(codes));
  return d;
}
// The low and the high two codes of a word.
__device__ __forceinline__ uint32_t e4m3_low(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w)); }
__device__ __forceinline__ uint32_t e4m3_high(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16)); }

// Two floats -> two codes (lo in the low byte): nearest, ties to even, saturating at +-448; NaN -> NaN.
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// 2^e of a scale byte: as a float for 1 .. 254.
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }

}  // namespace wq
