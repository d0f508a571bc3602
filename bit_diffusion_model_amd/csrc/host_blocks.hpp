// Host helpers of the offline packs: bf16 values, and a loop over blocks on several threads.
#pragma once
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <exception>
#include <thread>
#include <vector>

namespace svdq {

inline double bf16_value(uint16_t b) {
  const uint32_t u = (uint32_t)b << 16;
  float f;
  std::memcpy(&f, &u, 4);
  return (double)f;
}

inline int host_threads() {
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

}  // namespace svdq
