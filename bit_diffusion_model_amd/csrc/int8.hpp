// Device helpers of the 8-bit layer: loads of bf16 or fp32 rows as fp32 values, the
// largest magnitude of a row, and the 8-bit codes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "int8_host.hpp"

namespace svdq {

// Eight consecutive values k .. k+7 of a row as fp32; values at or past K are 0.  VEC: the
// row is 16-byte aligned at k (two 16-byte loads for fp32, one for bf16).
template <typename T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load1<uint16_t>(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

__device__ __forceinline__ void load8_vec(const uint16_t* p, float v[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  v[0] = bf16_lo_to_f32(w.x), v[1] = bf16_hi_to_f32(w.x), v[2] = bf16_lo_to_f32(w.y), v[3] = bf16_hi_to_f32(w.y);
  v[4] = bf16_lo_to_f32(w.z), v[5] = bf16_hi_to_f32(w.z), v[6] = bf16_lo_to_f32(w.w), v[7] = bf16_hi_to_f32(w.w);
}
__device__ __forceinline__ void load8_vec(const float* p, float v[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int64_t k, int64_t K, float v[8]) {
  if (VEC && k + 8 <= K) {
    load8_vec(row + k, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = k + e < K ? load1(row + k + e) : 0.0f;
  }
}

// Magnitudes are compared as unsigned bit patterns: their order is the order of the values,
// and a NaN or an infinity (0x7F800000 and above) is larger than every finite value.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = umax(v, (uint32_t)__shfl_xor((int)v, m, 64));
  return v;
}

// A row's scale s = a / 127 and the factor r = 127 / a of its codes (both IEEE quotients), from
// the bits of its largest magnitude; a is floored at 2^-96, below which r would pass the
// fp32 range (a row of zeros gets zero codes).  A row that holds a NaN or an infinity
// gets a NaN scale and r = 0, so that its codes are 0 and its outputs NaN.
__device__ __forceinline__ void row_scale(uint32_t abits, float& s, float& r) {
  const bool bad = abits >= 0x7F800000u;
  const float a = __uint_as_float(umax(abits, 0x0F800000u));  // 2^-96
  s = bad ? __uint_as_float(0x7FC00000u) : a / 127.0f;
  r = bad ? 0.0f : 127.0f / a;
}

// Four codes round_half_even(v r) in [-127, 127] as the bytes of a word.  Adding 1.5 * 2^23
// rounds to a whole number (ties to even) whose two's complement is in the low bits;
// |v r| <= 127 (1 + 2^-22), so no clamp is needed.  A NaN product (r = 0) has a zero low byte.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float r) {
  const float m = 12582912.0f;
  const uint32_t x = __float_as_uint(a * r + m), y = __float_as_uint(b * r + m);
  const uint32_t z = __float_as_uint(c * r + m), w = __float_as_uint(d * r + m);
  const uint32_t lo = __builtin_amdgcn_perm(y, x, 0x0C0C0400u), hi = __builtin_amdgcn_perm(w, z, 0x04000C0Cu);
  return lo | hi;
}

}  // namespace svdq
