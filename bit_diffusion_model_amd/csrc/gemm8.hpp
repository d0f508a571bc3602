// What the two 8-bit products (integers, and floating point with a scale for each block) share: loads into LDS and
// their waits, the outputs' epilogue stores, the numbering of tiles.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8.hpp"
#include "vec.hpp"

namespace svdq {

__device__ __forceinline__ int swz8(int row) { return (row ^ (row >> 3)) & 7; }

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, soff, 0, 0);
}

// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_vm_lgkm0() {
  static_assert(N >= 0 && N < 64, "counter range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

struct Out {
  const float *sX, *sW, *bias;
  void* Y;
  int64_t ldy, M, N;
  int ydtype;
};

constexpr float kNoBias = -0.0f;  // y + -0 is y, whatever y's sign

// One output, its type asked at run time
__device__ __forceinline__ void store1(const Out& o, int64_t m, int64_t n, float y) {
  if (o.ydtype == 0) static_cast<float*>(o.Y)[m * o.ldy + n] = y;
  else static_cast<__bf16*>(o.Y)[m * o.ldy + n] = (__bf16)(o.ydtype == 2 ? gelu5(y) : y);
}

// Eight outputs n .. n + 7 (n a multiple of 8) of row m, by stores of sixteen bytes at any output's address (rows of an odd
// length included: 4141x1408x4274 fp32 95 us by single outputs, 50 so).  WHOLE: all of them lie within Y; else
// channels may lie past N.  OUT: 0 fp32, 1 bf16, 2 bf16 of GELU.
template <int OUT, bool WHOLE>
__device__ __forceinline__ void store8(const Out& o, int64_t m, int64_t n, const float y[8]) {
  const bool whole = WHOLE || n + 8 <= o.N;
  if constexpr (OUT == 0) {
    float* p = static_cast<float*>(o.Y) + m * o.ldy + n;
    if (whole) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4a w = {__float_as_uint(y[4 * h]), __float_as_uint(y[4 * h + 1]), __float_as_uint(y[4 * h + 2]),
                          __float_as_uint(y[4 * h + 3])};
        reinterpret_cast<u32x4a*>(p)[h] = w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < o.N) p[e] = y[e];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(o.Y) + m * o.ldy + n;
    u32x4a w;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = OUT == 2 ? pack_bf16(gelu5(y[2 * e]), gelu5(y[2 * e + 1])) : pack_bf16(y[2 * e], y[2 * e + 1]);
    if (whole) {
      *reinterpret_cast<u32x4a*>(p) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < o.N) p[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
    }
  }
}

__device__ __forceinline__ void load_channels(const Out& o, int64_t n, float sw[8], float bb[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    sw[e] = n + e < o.N ? o.sW[n + e] : 0.0f;
    bb[e] = o.bias && n + e < o.N ? o.bias[n + e] : kNoBias;
  }
}

// One of the four arrays, by values: chosen by reference they would be fetched from scratch memory
__device__ __forceinline__ uint8_t* one_of(int i, uint8_t* a, uint8_t* b, uint8_t* c, uint8_t* d) {
  return i == 0 ? a : i == 1 ? b : i == 2 ? c : d;
}

// Tile t of tiles_m x tiles_n in strips of 8 tile rows
__device__ __forceinline__ void tile_at(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, uint32_t& m, uint32_t& n) {
  constexpr uint32_t GM = 8;
  const uint32_t grp = t / (GM * tiles_n), fm = grp * GM, gs = tiles_m - fm < GM ? tiles_m - fm : GM;
  const uint32_t in = t - grp * GM * tiles_n;
  m = fm + in % gs;
  n = in / gs;
}

// Compute units of the current device, asked once per thread and device.
inline int device_cus() {
  static thread_local int dev_of = -1, cus = 0;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  if (dev != dev_of) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1) n = 256;
    cus = n;
    dev_of = dev;
  }
  return cus;
}

}  // namespace svdq
