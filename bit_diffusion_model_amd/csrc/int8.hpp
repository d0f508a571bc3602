// Device helpers of the 8-bit layer: loads of bf16 or fp32 rows as fp32 values, the
// largest magnitude of a row, and the 8-bit codes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "int8_host.hpp"

namespace svdq {

// Row reads without branches, so that all of a row's loads can be issued before the first is
// waited for.  A Row covers K values from p; load(k) starts the read of values k .. k+7 and
// value() turns it into fp32; what lies at or past K reads as 0 (the buffer's range).
// VEC: p is 4-byte aligned (16-byte loads need no more).  A bf16 row that may begin in the middle
// of a word is read from the word's start, 20 bytes for 8 values, and shifted.  Only whole aligned
// words are read: the first and the last may hold a neighbour's value, never an unmapped byte, and
// value() drops the last one's second half where that is not the row's.
template <typename T, bool VEC>
struct Row;

template <bool VEC>
struct Row<float, VEC> {
  typedef struct { uint4 a, b; } Raw;
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Row(const float* p, int K) : r(make_rsrc(p, (uint32_t)K * 4)) {}
  __device__ __forceinline__ Raw load(int k) const {
    return Raw{buf_load16(r, (uint32_t)k * 4), buf_load16(r, (uint32_t)k * 4 + 16)};
  }
  __device__ __forceinline__ void value(const Raw& w, int, float v[8]) const {
    v[0] = __uint_as_float(w.a.x), v[1] = __uint_as_float(w.a.y), v[2] = __uint_as_float(w.a.z), v[3] = __uint_as_float(w.a.w);
    v[4] = __uint_as_float(w.b.x), v[5] = __uint_as_float(w.b.y), v[6] = __uint_as_float(w.b.z), v[7] = __uint_as_float(w.b.w);
  }
};

template <>
struct Row<uint16_t, true> {
  typedef uint4 Raw;
  __amdgpu_buffer_rsrc_t r;
  int odd_end;  // K if K is odd, else past every k
  __device__ __forceinline__ Row(const uint16_t* p, int K)
      : r(make_rsrc(p, ((uint32_t)K + 1) / 2 * 4)), odd_end(K & 1 ? K : 0x7FFFFFFF) {}
  __device__ __forceinline__ Raw load(int k) const { return buf_load16(r, (uint32_t)k * 2); }
  __device__ __forceinline__ void value(const Raw& w, int k, float v[8]) const {
    v[0] = bf16_lo_to_f32(w.x), v[1] = bf16_hi_to_f32(w.x), v[2] = bf16_lo_to_f32(w.y), v[3] = bf16_hi_to_f32(w.y);
    v[4] = bf16_lo_to_f32(w.z), v[5] = bf16_hi_to_f32(w.z), v[6] = bf16_lo_to_f32(w.w), v[7] = bf16_hi_to_f32(w.w);
    if (odd_end != 0x7FFFFFFF) {
#pragma unroll
      for (int e = 1; e < 8; e += 2)
        if (k + e == odd_end) v[e] = 0.0f;
    }
  }
};

template <>
struct Row<uint16_t, false> {
  typedef struct { uint4 a; uint32_t b; } Raw;
  __amdgpu_buffer_rsrc_t r;
  uint32_t shift;  // 16 where the row begins in the middle of a word, else 0
  int end;         // K where a neighbour's value follows the last one in its word, else past every k
  __device__ __forceinline__ Row(const uint16_t* p, int K) : shift((uint32_t)(reinterpret_cast<uintptr_t>(p) & 2) * 8) {
    const uint32_t halves = (uint32_t)K + shift / 16;
    r = make_rsrc(p - shift / 16, K > 0 ? (halves + 1) / 2 * 4 : 0);
    end = halves & 1 ? K : 0x7FFFFFFF;
  }
  __device__ __forceinline__ Raw load(int k) const {
    return Raw{buf_load16(r, (uint32_t)k * 2), buf_load4(r, (uint32_t)k * 2 + 16)};
  }
  __device__ __forceinline__ void value(const Raw& w, int k, float v[8]) const {
    const uint32_t x[5] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t d = __builtin_amdgcn_alignbit(x[i + 1], x[i], shift);
      v[2 * i] = bf16_lo_to_f32(d), v[2 * i + 1] = bf16_hi_to_f32(d);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e == end) v[e] = 0.0f;
  }
};

// GELU x Phi(x) for outputs that are rounded to bf16: Phi(-|x|) = t 2^(P(t) - x^2 / (2 ln 2)), t = 1 /
// (1 + |x| / 5), P the polynomial of degree 5 that fits log2(Phi(-a) / t) + a^2 / (2 ln 2) over 0 <= a <= 14
// best in the largest error (8.5e-6 of Phi).  With fp32 rounding GELU's relative error stays below 2e-5 (a bf16
// rounding: 2e-3), in the tail too.  Four terms fewer than gelu_erf: the product 4608x3072x9216
// with GELU 144 -> 140 us.
__device__ __forceinline__ float gelu5(float x) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.2f, fabsf(x), 1.0f));
  float p = -0.843770526f;
  p = fmaf(p, t, 1.98156184f);
  p = fmaf(p, t, -1.07346919f);
  p = fmaf(p, t, 1.25041619f);
  p = fmaf(p, t, 1.32332888f);
  p = fmaf(p, t, -3.63807946f);
  const float h = t * __builtin_amdgcn_exp2f(fmaf(x * x, -0.721347520f, p));
  return x * (x >= 0.0f ? 1.0f - h : h);
}

// Magnitudes are compared as unsigned bit patterns: their order is the order of the values,
// and a NaN or an infinity (0x7F800000 and above) is larger than every finite value.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// A reduction over groups of L lanes (4, 8, 16, 32 or 64) by lane moves in the vector unit (no LDS
// round trips): two quad permutations, for 8 lanes a mirror, for more two rotations of a row of
// 16, then the row and half swaps.  Every lane gets its group's result.
template <int L, typename F>
__device__ __forceinline__ uint32_t lane_reduce(uint32_t v, F f) {
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));   // quad [1 0 3 2]
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));   // quad [2 3 0 1]
  if constexpr (L == 8) v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));  // halves of a row mirrored
  if constexpr (L >= 16) {
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, true));  // row rotated by 4
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, true));  // row rotated by 8
  }
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = f(r[0], r[1]);
  }
  if constexpr (L >= 64) {
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = f(h[0], h[1]);
  }
  return v;
}
template <int L = 64>
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  return lane_reduce<L>(v, [](uint32_t a, uint32_t b) { return umax(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(lane_reduce<64>(
      __float_as_uint(v), [](uint32_t a, uint32_t b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); }));
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
// |v r| <= 127 (1 + 2^-22), so no clamp is needed.  A bad row (r = 0, which no other row has) may hold NaNs, whose
// payload comes through product and sum: there the bytes are taken from no word at all (selector 0x0C: zero), which
// costs nothing a value, the two selectors being the row's.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float r) {
  const float m = 12582912.0f;
  const uint32_t x = __float_as_uint(a * r + m), y = __float_as_uint(b * r + m);
  const uint32_t z = __float_as_uint(c * r + m), w = __float_as_uint(d * r + m);
  const bool bad = r == 0.0f;
  const uint32_t lo = __builtin_amdgcn_perm(y, x, bad ? 0x0C0C0C0Cu : 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm(w, z, bad ? 0x0C0C0C0Cu : 0x04000C0Cu);
  return lo | hi;
}

}  // namespace svdq
