// Host pack of the 8-bit layer: smoothing, one scale per output channel, 8-bit codes.
// Host code only (built by the host compiler, so it can also be built alone).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <exception>
#include <thread>
#include <vector>

#include "../../include/svdq.h"
#include "int8_host.hpp"
#include "internal.hpp"

namespace svdq {
namespace {

double bf16_value(uint16_t b) {
  const uint32_t u = (uint32_t)b << 16;
  float f;
  std::memcpy(&f, &u, 4);
  return (double)f;
}

int host_threads() {
  const char* env = std::getenv("SVDQ_NUM_THREADS");
  if (!env || !*env) env = std::getenv("OMP_NUM_THREADS");
  int n = env ? std::atoi(env) : 0;
  if (n <= 0) n = (int)std::thread::hardware_concurrency();
  return std::max(1, std::min(n, 64));
}

// f(i) for i in [0, n) on as many threads as can be had (f must not throw).
template <class F>
void run_blocks(int64_t n, F&& f) {
  std::atomic<int64_t> next{0};
  auto work = [&] {
    for (int64_t i; (i = next.fetch_add(1)) < n;) f(i);
  };
  const int64_t extra = std::min<int64_t>(host_threads(), n) - 1;
  std::vector<std::thread> th;
  try {
    th.reserve((size_t)std::max<int64_t>(extra, 0));
    for (int64_t t = 0; t < extra; ++t) th.emplace_back(work);
  } catch (const std::exception&) {
    // fewer threads than asked for: this one does the rest
  }
  work();
  for (auto& x : th) x.join();
}

constexpr int64_t kBlock = 64;  // output channels per task: 128 contiguous bytes of a row of W

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" int64_t svdq_int8_ld(int64_t K) { return K < 1 ? 0 : i8_ld(K); }

extern "C" svdq_status svdq_pack_weights_int8(int64_t K, int64_t N, const uint16_t* W, const float* act_absmax,
                                              float alpha, float* s_out, float* inv_s_out, int8_t* qW_out,
                                              float* sW_out) {
  if (!W || !s_out || !inv_s_out || !qW_out || !sW_out) return fail(SVDQ_EINVAL, "W and the outputs must be non-NULL");
  if (K < 1 || N < 1) return fail(SVDQ_EINVAL, "K and N must be >= 1 (got %lld, %lld)", (long long)K, (long long)N);
  if (K > kMaxInt8K) return fail(SVDQ_EUNSUPPORTED, "K must be <= %lld (got %lld)", (long long)kMaxInt8K, (long long)K);
  if (!(alpha >= 0.0f && alpha <= 1.0f)) return fail(SVDQ_EINVAL, "alpha must be in [0, 1]");
  std::atomic<bool> finite{true};
  if (act_absmax)
    for (int64_t k = 0; k < K; ++k)
      if (!std::isfinite(act_absmax[k])) finite = false;
  run_blocks((K + kBlock - 1) / kBlock, [&](int64_t b) {
    for (int64_t k = b * kBlock; k < std::min(K, (b + 1) * kBlock); ++k) {
      double w = 0.0;
      for (int64_t n = 0; n < N; ++n) {
        const uint16_t bits = W[k * N + n];
        if ((bits & 0x7F80u) == 0x7F80u) finite = false;
        w = std::max(w, std::fabs(bf16_value(bits)));
      }
      float s = 1.0f;
      if (act_absmax) {
        const double a = std::max((double)act_absmax[k], 1e-5), al = (double)alpha;
        s = (float)(std::pow(a, al) / std::pow(std::max(w, 1e-5), 1.0 - al));
      }
      s_out[k] = s;
      inv_s_out[k] = 1.0f / s;
    }
  });
  if (!finite) return fail(SVDQ_ENUMERIC, "W and act_absmax must be finite");
  const int64_t ld = i8_ld(K);
  run_blocks((N + kBlock - 1) / kBlock, [&](int64_t b) {
    const int64_t n0 = b * kBlock, nn = std::min(kBlock, N - n0);
    double top[kBlock] = {};
    for (int64_t k = 0; k < K; ++k)
      for (int64_t j = 0; j < nn; ++j)
        top[j] = std::max(top[j], std::fabs((double)s_out[k] * bf16_value(W[k * N + n0 + j])));
    for (int64_t j = 0; j < nn; ++j) {
      sW_out[n0 + j] = (float)(top[j] / 127.0);
      std::memset(qW_out + (n0 + j) * ld, 0, (size_t)ld);
    }
    for (int64_t k = 0; k < K; ++k)
      for (int64_t j = 0; j < nn; ++j) {
        const double s = (double)sW_out[n0 + j];
        if (s == 0.0) continue;
        const double q = std::nearbyint((double)s_out[k] * bf16_value(W[k * N + n0 + j]) / s);
        qW_out[(n0 + j) * ld + k] = (int8_t)std::max(-127.0, std::min(127.0, q));
      }
  });
  return ok();
}

extern "C" size_t svdq_int8_weight_bytes(int64_t K, int64_t N) {
  return K < 1 || N < 1 ? 0 : (size_t)((N + 15) / 16 * 16) * (size_t)i8_ld(K);
}

extern "C" svdq_status svdq_prepare_weights_int8(int64_t K, int64_t N, const int8_t* qW, int8_t* qW_out) {
  if (!qW || !qW_out) return fail(SVDQ_EINVAL, "qW and qW_out must be non-NULL");
  if (K < 1 || N < 1) return fail(SVDQ_EINVAL, "K and N must be >= 1 (got %lld, %lld)", (long long)K, (long long)N);
  if (K > kMaxInt8K) return fail(SVDQ_EUNSUPPORTED, "K must be <= %lld (got %lld)", (long long)kMaxInt8K, (long long)K);
  const int64_t ld = i8_ld(K);
  run_blocks((N + 15) / 16, [&](int64_t b) {
    int8_t* out = qW_out + b * 16 * ld;
    for (int64_t k = 0; k < ld; k += 16)  // 16 codes of each of the block's 16 channels
      for (int64_t c = 0; c < 16; ++c, out += 16) {
        const int64_t n = b * 16 + c;
        if (n < N) std::memcpy(out, qW + n * ld + k, 16);
        else std::memset(out, 0, 16);
      }
  });
  return ok();
}
