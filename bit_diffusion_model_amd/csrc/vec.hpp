// Vectors of V consecutive values of fp32 or bf16 rows, as the norms load and store them.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace svdq {

// ---- vectors of V channels, at any value's address: the memory takes wide loads and stores at every alignment

typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2a __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32a __attribute__((aligned(2)));

template <typename T, int V>
struct Vec {  // V values as loaded
  static constexpr int W = V * (int)sizeof(T) / 4;
  uint32_t w[W < 1 ? 1 : W];
};

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> loadv(const T* p) {
  Vec<T, V> r;
  constexpr int W = Vec<T, V>::W;
  if constexpr (W >= 4) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const u32x4a q = reinterpret_cast<const u32x4a*>(p)[i];
      r.w[4 * i] = q.x, r.w[4 * i + 1] = q.y, r.w[4 * i + 2] = q.z, r.w[4 * i + 3] = q.w;
    }
  } else if constexpr (W == 2) {
    const u32x2a q = *reinterpret_cast<const u32x2a*>(p);
    r.w[0] = q.x, r.w[1] = q.y;
  } else if constexpr (W == 1) {
    r.w[0] = *reinterpret_cast<const u32a*>(p);
  } else {
    r.w[0] = *p;
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void valuev(const Vec<T, V>& r, float v[V]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = __uint_as_float(r.w[e]);
  } else if constexpr (V == 1) {
    v[0] = __uint_as_float(r.w[0] << 16);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = e & 1 ? bf16_hi_to_f32(r.w[e / 2]) : bf16_lo_to_f32(r.w[e / 2]);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

template <bool NT, typename P, typename W>
__device__ __forceinline__ void put(P* p, W w) {
  if constexpr (NT) __builtin_nontemporal_store(w, p);
  else *p = w;
}

// NT: past the caches, for outputs that nothing reads before they are evicted (where x and y together
// pass the 256 MB cache: 262144x256 fp32 172 -> 156 us, 1048576x128 bf16 163 -> 135; below, the next
// operator finds y in the cache)
template <typename TY, int V, bool NT = false>
__device__ __forceinline__ void storev(TY* p, const float v[V]) {
  constexpr int W = V * (int)sizeof(TY) / 4;
  uint32_t w[W < 1 ? 1 : W];
  if constexpr (sizeof(TY) == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = __float_as_uint(v[e]);
  } else if constexpr (V > 1) {
#pragma unroll
    for (int e = 0; e < V; e += 2) w[e / 2] = pack_bf16(v[e], v[e + 1]);
  }
  if constexpr (W >= 4) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i)
      put<NT>(reinterpret_cast<u32x4a*>(p) + i, u32x4a{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]});
  } else if constexpr (W == 2) {
    *reinterpret_cast<u32x2a*>(p) = u32x2a{w[0], w[1]};
  } else if constexpr (W == 1) {
    *reinterpret_cast<u32a*>(p) = w[0];
  } else {
    *reinterpret_cast<__bf16*>(p) = (__bf16)v[0];
  }
}

// Values k .. k + 7 of a row of K values from p; what lies at or past K reads as 0.  At a row's end every value comes from
// an address of the row, so that the eight loads go out together (a branch each: one after the other's wait).
template <typename T>
__device__ __forceinline__ Vec<T, 8> load8(const T* p, int k, int K) {
  Vec<T, 8> r = {};
  if (k + 8 <= K) {
    r = loadv<T, 8>(p + k);
  } else if (k < K) {
    T t[7];
#pragma unroll
    for (int e = 0; e < 7; ++e) t[e] = p[k + e < K ? k + e : K - 1];
#pragma unroll
    for (int e = 0; e < 7; ++e) {
      if constexpr (sizeof(T) == 4) r.w[e] = k + e < K ? __float_as_uint(t[e]) : 0u;
      else r.w[e / 2] |= k + e < K ? (uint32_t)t[e] << (16 * (e & 1)) : 0u;
    }
  }
  return r;
}

}  // namespace svdq
