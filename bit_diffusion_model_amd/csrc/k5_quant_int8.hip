// Kernel 5: 8-bit activation codes with one scale per token.
//
// Mathematics (per token row, all in fp32, one rounding per operation): v_k = x_k inv_s_k;
// a = max(max_k |v_k|, 2^-96); s = a / 127; r = 127 / a; q_k = round_half_even(v_k r).
//
// Design (gfx950): bound by HBM (x read once, a byte per value written).  A row stays in
// registers between the maximum and the codes, so x is read once, all of its loads in
// flight together: one wave per row up to 1024 values (8 per lane and load), four waves per row
// up to 16384; longer rows are read twice (the second time from L2).  One wave a row against
// four (us): 16384 rows of 512 5.2 (10.1), of 1024 8.9 (12.7), of 2048 15.8 (16.8), of 4096 30.5 (29.3:
// 6.9 TB/s, the input in cache); 256 rows of 4096 3.4 (2.5).  1024 rows of 16384 in registers 10.0,
// read twice 12.7.
#include "int8.hpp"
#include "kernels.hpp"

namespace svdq {
namespace {

constexpr int Q_NT = 256;

// WPR waves per row, NC chunks of 8 values per lane (NC = 0: any length, read twice)
template <typename T, bool VEC, bool SMOOTH, int WPR, int NC>
__global__ __launch_bounds__(Q_NT) void k5_quant(const T* __restrict__ X, int64_t ldx, int64_t M, int K,
                                                 const float* __restrict__ inv_s, int8_t* __restrict__ qX, int ldq,
                                                 float* __restrict__ sX) {
  __shared__ uint32_t part[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = (int64_t)blockIdx.x * (4 / WPR) + wave / WPR;
  if (WPR == 1 && row >= M) return;  // WPR == 4: one row per block, the grid has M blocks
  typedef Row<T, VEC> RowX;
  typedef Row<float, true> RowS;
  const RowX x(X + row * ldx, K);
  const RowS f(inv_s, SMOOTH ? K : 0);
  int8_t* q = qX + row * ldq;
  const int li = (wave % WPR) * 64 + lane;
  constexpr int STEP = 8 * 64 * WPR;

  auto smooth = [&](const typename RowS::Raw& w, int k, float v[8]) {
    if constexpr (SMOOTH) {
      float s[8];
      f.value(w, k, s);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= s[e];
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
  auto store8 = [&](int k, const float v[8], float r) {
    if (k < ldq)
      *reinterpret_cast<uint2*>(q + k) = make_uint2(codes4(v[0], v[1], v[2], v[3], r), codes4(v[4], v[5], v[6], v[7], r));
  };

  uint32_t a = 0;
  float s, r;
  if constexpr (NC > 0) {
    typename RowX::Raw w[NC];
    typename RowS::Raw u[SMOOTH ? NC : 1];
#pragma unroll
    for (int j = 0; j < NC; ++j) w[j] = x.load(8 * li + j * STEP);
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (SMOOTH) u[j] = f.load(8 * li + j * STEP);
    float v[NC][8];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      x.value(w[j], 8 * li + j * STEP, v[j]);
      smooth(u[SMOOTH ? j : 0], 8 * li + j * STEP, v[j]);
      a = amax8(v[j], a);
    }
    row_scale(row_max(a), s, r);
#pragma unroll
    for (int j = 0; j < NC; ++j) store8(8 * li + j * STEP, v[j], r);
  } else {
    auto at = [&](int k, float v[8]) {
      const auto w = x.load(k);
      typename RowS::Raw u = {};
      if (SMOOTH) u = f.load(k);
      x.value(w, k, v);
      smooth(u, k, v);
    };
    for (int k = 8 * li; k < K; k += STEP) {
      float v[8];
      at(k, v);
      a = amax8(v, a);
    }
    row_scale(row_max(a), s, r);
    for (int k = 8 * li; k < ldq; k += STEP) {
      float v[8];
      at(k, v);
      store8(k, v, r);
    }
  }
  if (li == 0) sX[row] = s;
}

template <typename T, bool VEC, bool SMOOTH>
void launch(int64_t M, int64_t K, const T* X, int64_t ldx, const float* inv_s, int8_t* qX, float* sX, hipStream_t st) {
  const int ldq = (int)i8_ld(K);
  // a launch takes fewer than 2^32 threads: more rows than that go in several
  auto go = [&](auto kernel, int64_t per_block) {
    const int64_t slab = per_block << 23;
    for (int64_t m = 0; m < M; m += slab) {
      const int64_t rows = M - m < slab ? M - m : slab;
      hipLaunchKernelGGL(kernel, dim3((uint32_t)((rows + per_block - 1) / per_block)), dim3(Q_NT), 0, st, X + m * ldx, ldx,
                         rows, (int)K, inv_s, qX + m * ldq, ldq, sX + m);
    }
  };
  if (ldq <= 512) go(k5_quant<T, VEC, SMOOTH, 1, 1>, 4);
  else if (ldq <= 1024) go(k5_quant<T, VEC, SMOOTH, 1, 2>, 4);
  else if (ldq <= 2048) go(k5_quant<T, VEC, SMOOTH, 4, 1>, 1);
  else if (ldq <= 4096) go(k5_quant<T, VEC, SMOOTH, 4, 2>, 1);
  else if (ldq <= 8192) go(k5_quant<T, VEC, SMOOTH, 4, 4>, 1);
  else if (ldq <= 16384) go(k5_quant<T, VEC, SMOOTH, 4, 8>, 1);
  else go(k5_quant<T, VEC, SMOOTH, 4, 0>, 1);
}

template <typename T, bool VEC>
void launch_any(int64_t M, int64_t K, const void* X, int64_t ldx, const float* inv_s, int8_t* qX, float* sX, hipStream_t st) {
  const T* x = static_cast<const T*>(X);
  inv_s ? launch<T, VEC, true>(M, K, x, ldx, inv_s, qX, sX, st) : launch<T, VEC, false>(M, K, x, ldx, inv_s, qX, sX, st);
}

}  // namespace

hipError_t launch_quant_i8(int64_t M, int64_t K, const void* X, int xdtype, int64_t ldx, const float* inv_s, int8_t* qX,
                           float* sX, hipStream_t st) {
  if (xdtype == 0) launch_any<float, true>(M, K, X, ldx, inv_s, qX, sX, st);
  else if (rows_aligned4(X, ldx, xdtype)) launch_any<uint16_t, true>(M, K, X, ldx, inv_s, qX, sX, st);
  else launch_any<uint16_t, false>(M, K, X, ldx, inv_s, qX, sX, st);
  return hipGetLastError();
}

}  // namespace svdq
