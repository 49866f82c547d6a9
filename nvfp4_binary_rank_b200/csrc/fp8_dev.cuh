// FP8 block format on the device: E4M3 codes with one FP32 scale per 128 elements
// (of a row for activations, of a 128 x 128 tile for weights).
//
//   a = max(|v| over the block, 2^-100),  scale = RN(a / 448),  code = E4M3(RN(v * RN(448 / a)))
//
// with E4M3 rounding to nearest-even and saturating at 448.  The lower limit keeps
// 448 / a finite, so an all-zero block needs no branch: its codes are zero.  A NaN in
// a block makes its scale and codes NaN; an infinity makes the scale infinite (its
// own code is NaN and every other product of the block 0 * inf), so neither is
// silently turned into a finite value.
#pragma once

#include <cstdint>

namespace biloco {

constexpr int kFp8Block = 128;
constexpr float kE4m3Max = 448.0f;
constexpr float kFp8TinyAmax = 0x1p-100f;

struct Fp8Scale {
  float scale, inv;
};

// `bits`: the largest |v| of the block as FP32 bits.  Non-negative floats order like
// their bits, with every NaN above infinity, so an integer maximum keeps NaNs.
__device__ __forceinline__ Fp8Scale fp8_block_scale(uint32_t bits) {
  float a = __uint_as_float(bits);
  if (a < kFp8TinyAmax) a = kFp8TinyAmax;     // false for NaN
  Fp8Scale s;
  s.scale = __fdiv_rn(a, kE4m3Max);
  s.inv = __fdiv_rn(kE4m3Max, a);
  return s;
}

// Two FP32 values -> two E4M3 codes, `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_from_f32(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4_from_f32(float a, float b, float c, float d) {
  return e4m3x2_from_f32(a, b) | (e4m3x2_from_f32(c, d) << 16);
}

// Two BF16 values packed in a word -> FP32.
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// FP32 -> BF16 pair, nearest-even, `lo` in the low half.
__device__ __forceinline__ uint32_t bf16x2_from_f32(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace biloco
