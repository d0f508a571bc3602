// Sizes of the 8-bit layer and the group norm shared by host and device code.
#pragma once
#include <stdint.h>

namespace svdq {

// Rows of codes are padded with zeros to a multiple of 128 bytes (one K stage of the product).
constexpr int64_t kI8Stage = 128;
constexpr int64_t i8_ld(int64_t K) { return (K + kI8Stage - 1) / kI8Stage * kI8Stage; }
// 127^2 K < 2^31
constexpr int64_t kMaxInt8K = 131072;
// the norm keeps per-channel and per-group values in LDS
constexpr int64_t kMaxNormC = 4096;
constexpr int kMaxNormG = 1024;

// Whether every row (from p, ld values apart; xdtype 0 fp32, 1 bf16) is 4-byte aligned.
inline bool rows_aligned4(const void* p, int64_t ld, int xdtype) {
  return reinterpret_cast<uintptr_t>(p) % 4 == 0 && (xdtype == 0 || ld % 2 == 0);
}

}  // namespace svdq
