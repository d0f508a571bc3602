// Device helpers of the block-scaled 8-bit floating point layer: a block's scale and its E4M3 codes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8.hpp"

namespace svdq {

constexpr int64_t kFp8Block = 128;  // values to a scale, along K; weights also 128 channels
constexpr int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }
// The scales of a block of K: one row of M values, padded so that every row is 16-byte aligned.
constexpr int64_t fp8_pad(int64_t M) { return (M + 3) / 4 * 4; }

// A block's scale s = a / 448 and the factor r = 448 / a of its codes (both IEEE quotients: the first by a product and one
// correction with the exact residual, which gives the correctly rounded one for every a), from the bits of its largest
// magnitude; a is floored at 2^-96 (zeros get zero codes, r stays finite).  A block that holds a NaN or an infinity gets a
// NaN scale and r = 0, so that its codes are 0 and the row's outputs NaN.
__device__ __forceinline__ void block_scale(uint32_t abits, float& s, float& r) {
  const bool bad = abits >= 0x7F800000u;
  const float a = __uint_as_float(umax(abits, 0x0F800000u));  // 2^-96
  const float q = a * (1.0f / 448.0f);
  s = bad ? __uint_as_float(0x7FC00000u) : fmaf(fmaf(-448.0f, q, a), 1.0f / 448.0f, q);
  r = bad ? 0.0f : 448.0f / a;
}

// Four codes E4M3(v r) as the bytes of a word, to nearest, ties to the even code: the hardware's conversion.
// |v r| <= 448 (1 + 2^-22) rounds to at most 448, so nothing saturates.  A bad block (r = 0, which no other has) gets
// zeros whatever it holds.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float r) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * r, b * r, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * r, d * r, w, true);
  return r == 0.0f ? 0u : (uint32_t)w;
}

}  // namespace svdq
