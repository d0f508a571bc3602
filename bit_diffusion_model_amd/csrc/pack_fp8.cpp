// Host pack of the block-scaled 8-bit floating point layer: E4M3 codes with one scale for each 128 x 128 weights, and
// their transpose.  Host code only (built by the host compiler, so it can also be built alone).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "../../include/svdq.h"
#include "host_blocks.hpp"
#include "int8_host.hpp"
#include "internal.hpp"

namespace svdq {
namespace {

constexpr int64_t kTile = 128;

// The E4M3 code nearest to v, ties to the even code, |v| saturating at 448: steps of 2^(e - 3) in the binade of 2^e,
// e >= -6 (below it the steps of 2^-9 that subnormal codes count).
uint8_t e4m3(double v) {
  const uint8_t sign = std::signbit(v) ? 0x80 : 0;
  const double a = std::min(std::fabs(v), 448.0);
  int e = -6;
  if (a >= 0x1p-6) {
    int x;
    std::frexp(a, &x);
    e = x - 1;
  }
  const int steps = (int)std::nearbyint(std::ldexp(a, 3 - e));  // 0..16; 8..16 where normal
  return sign | (uint8_t)(steps + 8 * (e + 6));  // a carry into the next binade is the next code
}

svdq_status check_sizes(int64_t K, int64_t N) {
  if (K < 1 || N < 1) return fail(SVDQ_EINVAL, "K and N must be >= 1 (got %lld, %lld)", (long long)K, (long long)N);
  if (K > kMaxInt8K) return fail(SVDQ_EUNSUPPORTED, "K must be <= %lld (got %lld)", (long long)kMaxInt8K, (long long)K);
  return SVDQ_OK;
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" svdq_status svdq_pack_weights_fp8(int64_t K, int64_t N, const uint16_t* W, uint8_t* qW_out, float* sW_out) {
  if (!W || !qW_out || !sW_out) return fail(SVDQ_EINVAL, "W and the outputs must be non-NULL");
  svdq_status st = check_sizes(K, N);
  if (st != SVDQ_OK) return st;
  const int64_t ld = i8_ld(K), kb = ld / kTile;
  std::atomic<bool> finite{true};
  run_blocks((N + kTile - 1) / kTile, [&](int64_t b) {
    const int64_t n0 = b * kTile, n1 = std::min(N, n0 + kTile);
    for (int64_t c = 0; c < kb; ++c) {
      const int64_t k0 = c * kTile, k1 = std::min(K, k0 + kTile);
      double top = 0.0;
      bool all = true;
      for (int64_t k = k0; k < k1; ++k)
        for (int64_t n = n0; n < n1; ++n) {
          const uint16_t bits = W[k * N + n];
          if ((bits & 0x7F80u) == 0x7F80u) all = false;
          top = std::max(top, std::fabs(bf16_value(bits)));
        }
      if (!all) finite = false;
      const float s = all ? (float)(top / 448.0) : 0.0f;  // no code is made of a NaN or an infinity: the block is zeros
      sW_out[b * kb + c] = s;
      for (int64_t n = n0; n < n1; ++n) {
        uint8_t* out = qW_out + n * ld + k0;
        std::memset(out, 0, (size_t)kTile);
        if (s != 0.0f)
          for (int64_t k = k0; k < k1; ++k) out[k - k0] = e4m3(bf16_value(W[k * N + n]) / (double)s);
      }
    }
  });
  if (!finite) return fail(SVDQ_ENUMERIC, "W must be finite");
  return ok();
}

extern "C" svdq_status svdq_transpose_weights_fp8(int64_t K, int64_t N, const uint8_t* qW, const float* sW,
                                                  uint8_t* qWt_out, float* sWt_out) {
  if (!qW || !sW || !qWt_out || !sWt_out) return fail(SVDQ_EINVAL, "qW, sW and the outputs must be non-NULL");
  svdq_status st = check_sizes(K, N);
  if (st != SVDQ_OK) return st;
  if (N > kMaxInt8K) return fail(SVDQ_EUNSUPPORTED, "N must be <= %lld (got %lld)", (long long)kMaxInt8K, (long long)N);
  const int64_t ld = i8_ld(K), kb = ld / kTile, ldt = i8_ld(N), nb = ldt / kTile;
  run_blocks(kb, [&](int64_t c) {
    const int64_t k0 = c * kTile, k1 = std::min(K, k0 + kTile);
    for (int64_t b = 0; b < nb; ++b) sWt_out[c * nb + b] = sW[b * kb + c];
    for (int64_t k = k0; k < k1; ++k) {
      uint8_t* out = qWt_out + k * ldt;
      for (int64_t n = 0; n < N; ++n) out[n] = qW[n * ld + k];
      std::memset(out + N, 0, (size_t)(ldt - N));
    }
  });
  return ok();
}
