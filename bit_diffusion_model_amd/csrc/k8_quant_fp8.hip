// Kernel 8: E4M3 activation codes with one scale for each token and block of 128 values along K.
//
// Mathematics (per row and block, in fp32, one rounding per operation): a = max(max |x|, 2^-96); s = a / 448;
// r = 448 / a; q = E4M3(x r).
//
// Design (gfx950): bound by HBM (x read once, a byte per value written).  Blocks of 128 are independent, so a row
// needs no join: 16 lanes hold a block, 8 values each, and meet by lane moves.  A workgroup takes 16 rows x 512
// values, four rows a wave, all four loads in flight; the 64 scales meet in LDS and leave as four runs of 16 (the
// scales' rows run along the tokens, which is how the product reads them).  4608 x 3072 bf16 9.2 us, 16384 x 2048 21.2: 4.7 and
// 4.8 TB/s of what a large copy reaches 5.1.
#include "fp8.hpp"
#include "kernels.hpp"

namespace svdq {
namespace {

constexpr int Q_ROWS = 16, Q_COLS = 512;

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k8_quant(const T* __restrict__ X, int64_t ldx, int64_t M, int K, uint32_t kts,
                                                uint8_t* __restrict__ qX, int64_t ldq, float* __restrict__ sX,
                                                int64_t Mp) {
  __shared__ float sc[Q_COLS / 128][Q_ROWS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t rt = blockIdx.x / kts, kt = blockIdx.x - rt * kts;
  const int64_t m0 = (int64_t)rt * Q_ROWS;
  const int rows = (int)(M - m0 < Q_ROWS ? M - m0 : Q_ROWS);
  const int k = (int)kt * Q_COLS + 8 * lane;
  typedef Row<T, VEC> RowX;
  auto row = [&](int j) {  // past M: no range, zeros
    const int r = wave + 4 * j;
    return RowX(X + (m0 + (r < rows ? r : 0)) * ldx, r < rows ? K : 0);
  };
  typename RowX::Raw w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = row(j).load(k);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = wave + 4 * j;
    float v[8];
    row(j).value(w[j], k, v);
    uint32_t a = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) a = umax(a, abs_bits(v[e]));
    a = wave_umax<16>(a);
    float s, f;
    block_scale(a, s, f);
    if ((lane & 15) == 0) sc[lane >> 4][r] = s;
    if (r < rows && k < ldq)
      *reinterpret_cast<uint2*>(qX + (m0 + r) * ldq + k) =
          make_uint2(e4m3x4(v[0], v[1], v[2], v[3], f), e4m3x4(v[4], v[5], v[6], v[7], f));
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int b = (int)kt * (Q_COLS / 128) + (threadIdx.x >> 4), r = threadIdx.x & 15;
    if (r < rows && (int64_t)b * 128 < ldq) sX[b * Mp + m0 + r] = sc[threadIdx.x >> 4][r];
  }
}

template <typename T, bool VEC>
void launch(int64_t M, int64_t K, const T* X, int64_t ldx, uint8_t* qX, float* sX, hipStream_t st) {
  const int64_t ldq = i8_ld(K), kts = (ldq + Q_COLS - 1) / Q_COLS, Mp = fp8_pad(M);
  // a launch takes fewer than 2^32 threads: more rows than that go in several
  const int64_t slab = (((int64_t)1 << 24) - 1) / kts * Q_ROWS;
  for (int64_t m = 0; m < M; m += slab) {
    const int64_t rows = M - m < slab ? M - m : slab;
    const uint32_t grid = (uint32_t)((rows + Q_ROWS - 1) / Q_ROWS * kts);
    hipLaunchKernelGGL((k8_quant<T, VEC>), dim3(grid), dim3(256), 0, st, X + m * ldx, ldx, rows, (int)K, (uint32_t)kts,
                       qX + m * ldq, ldq, sX + m, Mp);
  }
}

}  // namespace

hipError_t launch_quant_fp8(int64_t M, int64_t K, const void* X, int xdtype, int64_t ldx, uint8_t* qX, float* sX,
                            hipStream_t st) {
  if (xdtype == 0) launch<float, true>(M, K, static_cast<const float*>(X), ldx, qX, sX, st);
  else if (rows_aligned4(X, ldx, xdtype)) launch<uint16_t, true>(M, K, static_cast<const uint16_t*>(X), ldx, qX, sX, st);
  else launch<uint16_t, false>(M, K, static_cast<const uint16_t*>(X), ldx, qX, sX, st);
  return hipGetLastError();
}

}  // namespace svdq
