// Kernel 5: 8-bit activation codes with one scale per token.
//
// Mathematics (per token row, all in fp32, one rounding per operation): v_k = x_k inv_s_k;
// a = max(max_k |v_k|, 2^-96); s = a / 127; r = 127 / a; q_k = round_half_even(v_k r).
//
// Design (gfx950): bound by HBM (x read once, a byte per value written).  A row stays in
// registers between the maximum and the codes, so x is read once: one wave per row up to
// 4096 values (8 per lane and 16-byte load, up to 8 loads in flight), four waves per row
// up to 16384; longer rows are read twice (the second time from L2).
#include "int8.hpp"
#include "kernels.hpp"

namespace svdq {
namespace {

constexpr int Q_NT = 256;

// WPR waves per row, NC chunks of 8 values per lane (NC = 0: any length, read twice)
template <typename T, bool VEC, int WPR, int NC>
__global__ __launch_bounds__(Q_NT) void k5_quant(const T* __restrict__ X, int64_t ldx, int64_t M, int64_t K,
                                                 const float* __restrict__ inv_s, int8_t* __restrict__ qX, int64_t ldq,
                                                 float* __restrict__ sX) {
  __shared__ uint32_t part[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = (int64_t)blockIdx.x * (4 / WPR) + wave / WPR;
  if (WPR == 1 && row >= M) return;  // WPR == 4: one row per block, the grid has M blocks
  const T* x = X + row * ldx;
  int8_t* q = qX + row * ldq;
  const int li = (wave % WPR) * 64 + lane;
  constexpr int STEP = 8 * 64 * WPR;

  auto smoothed = [&](int64_t k, float v[8]) {
    load8<T, VEC>(x, k, K, v);
    if (inv_s) {
      float f[8];
      load8<float, true>(inv_s, k, K, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= f[e];
    }
  };
  auto amax8 = [](const float v[8], uint32_t a) {
#pragma unroll
    for (int e = 0; e < 8; ++e) a = umax(a, abs_bits(v[e]));
    return a;
  };
  auto row_max = [&](uint32_t a) {
    a = wave_umax(a);
    if (WPR > 1) {
      if (lane == 0) part[wave] = a;
      __syncthreads();
      a = umax(umax(part[0], part[1]), umax(part[2], part[3]));
    }
    return a;
  };
  auto store8 = [&](int64_t k, const float v[8], float r) {
    if (k < ldq)
      *reinterpret_cast<uint2*>(q + k) = make_uint2(codes4(v[0], v[1], v[2], v[3], r), codes4(v[4], v[5], v[6], v[7], r));
  };

  uint32_t a = 0;
  float s, r;
  if constexpr (NC > 0) {
    float v[NC][8];
#pragma unroll
    for (int j = 0; j < NC; ++j) smoothed(8 * li + j * STEP, v[j]);
#pragma unroll
    for (int j = 0; j < NC; ++j) a = amax8(v[j], a);
    row_scale(row_max(a), s, r);
#pragma unroll
    for (int j = 0; j < NC; ++j) store8(8 * li + j * STEP, v[j], r);
  } else {
    for (int64_t k = 8 * li; k < K; k += STEP) {
      float v[8];
      smoothed(k, v);
      a = amax8(v, a);
    }
    row_scale(row_max(a), s, r);
    for (int64_t k = 8 * li; k < ldq; k += STEP) {
      float v[8];
      smoothed(k, v);
      store8(k, v, r);
    }
  }
  if (li == 0) sX[row] = s;
}

template <typename T, bool VEC>
void launch(int64_t M, int64_t K, const T* X, int64_t ldx, const float* inv_s, int8_t* qX, float* sX, hipStream_t st) {
  const int64_t ldq = i8_ld(K);
  const dim3 g4((uint32_t)((M + 3) / 4)), g1((uint32_t)M), b(Q_NT);
  if (ldq <= 512) hipLaunchKernelGGL((k5_quant<T, VEC, 1, 1>), g4, b, 0, st, X, ldx, M, K, inv_s, qX, ldq, sX);
  else if (ldq <= 1024) hipLaunchKernelGGL((k5_quant<T, VEC, 1, 2>), g4, b, 0, st, X, ldx, M, K, inv_s, qX, ldq, sX);
  else if (ldq <= 2048) hipLaunchKernelGGL((k5_quant<T, VEC, 1, 4>), g4, b, 0, st, X, ldx, M, K, inv_s, qX, ldq, sX);
  else if (ldq <= 4096) hipLaunchKernelGGL((k5_quant<T, VEC, 1, 8>), g4, b, 0, st, X, ldx, M, K, inv_s, qX, ldq, sX);
  else if (ldq <= 8192) hipLaunchKernelGGL((k5_quant<T, VEC, 4, 4>), g1, b, 0, st, X, ldx, M, K, inv_s, qX, ldq, sX);
  else if (ldq <= 16384) hipLaunchKernelGGL((k5_quant<T, VEC, 4, 8>), g1, b, 0, st, X, ldx, M, K, inv_s, qX, ldq, sX);
  else hipLaunchKernelGGL((k5_quant<T, VEC, 4, 0>), g1, b, 0, st, X, ldx, M, K, inv_s, qX, ldq, sX);
}

}  // namespace

hipError_t launch_quant_i8(int64_t M, int64_t K, const void* X, int xdtype, int64_t ldx, const float* inv_s, int8_t* qX,
                           float* sX, hipStream_t st) {
  // 16-byte loads need every row 16-byte aligned; other rows are loaded value by value
  const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % (xdtype == 0 ? 4 : 8) == 0;
  if (xdtype == 0) {
    const float* x = static_cast<const float*>(X);
    vec ? launch<float, true>(M, K, x, ldx, inv_s, qX, sX, st) : launch<float, false>(M, K, x, ldx, inv_s, qX, sX, st);
  } else {
    const uint16_t* x = static_cast<const uint16_t*>(X);
    vec ? launch<uint16_t, true>(M, K, x, ldx, inv_s, qX, sX, st)
        : launch<uint16_t, false>(M, K, x, ldx, inv_s, qX, sX, st);
  }
  return hipGetLastError();
}

}  // namespace svdq
