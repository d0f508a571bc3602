// Kernel 6: the W8A8 product, 8-bit codes with one scale per token and one per channel.
//
// Mathematics: I[m][n] = sum_k qX[m][k] qW[n][k], exact in 32-bit integers (K <= 131072:
// 127^2 K < 2^31); y = ((float)I s_X[m]) s_W[n] + bias[n], in fp32, then optionally GELU,
// rounded once to the output type.
//
// Design (gfx950): v_mfma_i32_32x32x32_i8; a block of 4 waves owns a 64 x 64 tile of Y
// (one 32 x 32 accumulator per wave) and walks K in stages of 128 bytes; both operands
// go global -> LDS by LDS-destination buffer loads, one stage ahead, into two buffers, the
// 16-byte slots of a row XOR-swizzled so that the operand reads of 16 consecutive rows
// fall in distinct bank groups.  Rows past M and channels past N lie beyond the buffers'
// ranges: they read as zeros and are not stored.
#include "int8.hpp"
#include "kernels.hpp"

namespace svdq {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

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

// TI x TJ accumulators of 32 x 32 per wave, WM x WN waves
template <int WM, int WN, int TI, int TJ>
__global__ __launch_bounds__(64 * WM * WN) void k6_gemm(const int8_t* __restrict__ qX, int64_t ld, int64_t M,
                                                        const int8_t* __restrict__ qW, int64_t N,
                                                        const float* __restrict__ sX, const float* __restrict__ sW,
                                                        const float* __restrict__ bias, void* __restrict__ Y,
                                                        int64_t ldy, int ydtype, uint32_t tiles_n) {
  constexpr int BM = 32 * TI * WM, BN = 32 * TJ * WN, NW = WM * WN;
  constexpr int AB = BM * 128, BB = BN * 128;
  static_assert(AB % (1024 * NW) == 0 && BB % (1024 * NW) == 0, "whole 1 KB loads per wave");
  constexpr int NA = AB / 1024 / NW, NB = BB / 1024 / NW;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * (AB + BB)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, kh = lane >> 5;
  const int wr = (wave / WN) * 32 * TI, wc = (wave % WN) * 32 * TJ;
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * BM, n0 = (int64_t)(blockIdx.x % tiles_n) * BN;
  const uint32_t rows = (uint32_t)(M - m0 < BM ? M - m0 : BM), cols = (uint32_t)(N - n0 < BN ? N - n0 : BN);
  const int nst = (int)(ld / 128);
  const __amdgpu_buffer_rsrc_t rA = make_rsrc(qX + m0 * ld, rows * (uint32_t)ld);
  const __amdgpu_buffer_rsrc_t rB = make_rsrc(qW + n0 * ld, cols * (uint32_t)ld);
  uint32_t va[NA], vb[NB];
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int row = (wave + NW * q) * 8 + (lane >> 3);
    va[q] = (uint32_t)row * (uint32_t)ld + (uint32_t)(((lane & 7) ^ swz8(row)) * 16);
  }
#pragma unroll
  for (int q = 0; q < NB; ++q) {
    const int row = (wave + NW * q) * 8 + (lane >> 3);
    vb[q] = (uint32_t)row * (uint32_t)ld + (uint32_t)(((lane & 7) ^ swz8(row)) * 16);
  }
  auto issue = [&](int k, uint8_t* buf) {
#pragma unroll
    for (int q = 0; q < NA; ++q) dma16(rA, buf + (wave + NW * q) * 1024, va[q], (uint32_t)k * 128);
#pragma unroll
    for (int q = 0; q < NB; ++q) dma16(rB, buf + AB + (wave + NW * q) * 1024, vb[q], (uint32_t)k * 128);
  };

  v16i acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v16i{};

  issue(0, lds);
  for (int k = 0; k < nst; ++k) {
    uint8_t* cur = lds + (k & 1) * (AB + BB);
    // stage k has arrived; every wave is done with the other buffer
    wait_vm_lgkm0<0>();
    __syncthreads();
    if (k + 1 < nst) issue(k + 1, lds + ((k + 1) & 1) * (AB + BB));
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v4i A[TI], B[TJ];
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int r = wr + 32 * i + l32;
        A[i] = *reinterpret_cast<const v4i*>(cur + r * 128 + (((2 * s + kh) ^ swz8(r)) * 16));
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int c = wc + 32 * j + l32;
        B[j] = *reinterpret_cast<const v4i*>(cur + AB + c * 128 + (((2 * s + kh) ^ swz8(c)) * 16));
      }
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(A[i], B[j], acc[i][j], 0, 0, 0);
    }
  }

#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int64_t n = n0 + wc + 32 * j + l32;
    if (n >= N) continue;
    const float sw = sW[n], b = bias ? bias[n] : 0.0f;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
#pragma unroll
      for (int a = 0; a < 16; ++a) {
        const int64_t m = m0 + wr + 32 * i + 8 * (a >> 2) + 4 * kh + (a & 3);
        if (m >= M) continue;
        float y = (float)acc[i][j][a] * sX[m] * sw;
        if (bias) y += b;
        if (ydtype == 0) static_cast<float*>(Y)[m * ldy + n] = y;
        else static_cast<__bf16*>(Y)[m * ldy + n] = (__bf16)(ydtype == 2 ? gelu_erf(y) : y);
      }
    }
  }
}

}  // namespace

hipError_t launch_w8a8(int64_t M, int64_t K, int64_t N, const int8_t* qX, const float* sX, const int8_t* qW,
                       const float* sW, const float* bias, void* Y, int64_t ldy, int ydtype, hipStream_t st) {
  const uint32_t tiles_m = (uint32_t)((M + 63) / 64), tiles_n = (uint32_t)((N + 63) / 64);
  hipLaunchKernelGGL((k6_gemm<2, 2, 1, 1>), dim3(tiles_m * tiles_n), dim3(256), 0, st, qX, i8_ld(K), M, qW, N, sX, sW,
                     bias, Y, ldy, ydtype, tiles_n);
  return hipGetLastError();
}

}  // namespace svdq
