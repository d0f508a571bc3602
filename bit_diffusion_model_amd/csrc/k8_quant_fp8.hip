// Kernel 8: E4M3 activation codes with one scale for each token and block of 128 values along K.
//
// Mathematics (per row and block, in fp32, one rounding per operation): a = max(max |x|, 2^-96); s = a / 448;
// r = 448 / a; q = E4M3(x r).
//
// Design (gfx950): bound by HBM (x read once, a byte per value written).  Blocks of 128 are independent, so a row
// needs no join: 16 lanes hold a block, 8 values each, and meet by lane moves.  A wave takes 512 values of a row, a
// workgroup four rows, whose scales lie side by side (the scales' rows run along the tokens, which is how the product
// reads them).  4608 x 3072 bf16 8.6 us (10.5 behind a product that has lowered the clock and filled the caches), 16384 x
// 2048 21: 4.8 TB/s of what a large copy reaches 5.1.  (Four rows a wave with 64 scales joined in LDS, whole runs of 16,
// measured in turn: 9.3 against 8.9, and 2.9 against 2.1 at 154 x 768, 7.2 against 6.3 at 3000 x 3072, but 32.0 against 33.4
// at 4608 x 12288.)
#include "fp8.hpp"
#include "kernels.hpp"

namespace svdq {
namespace {

constexpr int Q_ROWS = 4, Q_COLS = 512;

template <typename T, bool VEC>
__global__ __launch_bounds__(64 * Q_ROWS) void k8_quant(const T* __restrict__ X, int64_t ldx, int64_t M, int K,
                                                        uint32_t kts, uint8_t* __restrict__ qX, int64_t ldq,
                                                        float* __restrict__ sX, int64_t Mp) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t rt = blockIdx.x / kts, kt = blockIdx.x - rt * kts;
  const int64_t m = (int64_t)rt * Q_ROWS + wave;
  if (m >= M) return;
  const int k = (int)kt * Q_COLS + 8 * lane;
  const Row<T, VEC> x(X + m * ldx, K);
  float v[8];
  x.value(x.load(k), k, v);
  uint32_t a = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = umax(a, abs_bits(v[e]));
  a = wave_umax<16>(a);
  float s, f;
  block_scale(a, s, f);
  if (k >= ldq) return;
  if ((lane & 15) == 0) sX[(int64_t)(k >> 7) * Mp + m] = s;
  *reinterpret_cast<uint2*>(qX + m * ldq + k) =
      make_uint2(e4m3x4(v[0], v[1], v[2], v[3], f), e4m3x4(v[4], v[5], v[6], v[7], f));
}

template <typename T, bool VEC>
void launch(int64_t M, int64_t K, const T* X, int64_t ldx, uint8_t* qX, float* sX, hipStream_t st) {
  const int64_t ldq = i8_ld(K), kts = (ldq + Q_COLS - 1) / Q_COLS, Mp = fp8_pad(M);
  // a launch takes fewer than 2^32 threads: more rows than that go in several
  const int64_t slab = (((int64_t)1 << 24) - 1) / kts * Q_ROWS;
  for (int64_t m = 0; m < M; m += slab) {
    const int64_t rows = M - m < slab ? M - m : slab;
    const uint32_t grid = (uint32_t)((rows + Q_ROWS - 1) / Q_ROWS * kts);
    hipLaunchKernelGGL((k8_quant<T, VEC>), dim3(grid), dim3(64 * Q_ROWS), 0, st, X + m * ldx, ldx, rows, (int)K,
                       (uint32_t)kts, qX + m * ldq, ldq, sX + m, Mp);
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
