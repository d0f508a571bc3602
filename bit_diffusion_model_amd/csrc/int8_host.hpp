// Sizes of the 8-bit layer and the group norm shared by host and device code.
#pragma once
#include <stdint.h>

namespace svdq {

// Rows of codes are padded with zeros to a multiple of 128 bytes (one K stage of the product).
constexpr int64_t kI8Stage = 128;
constexpr int64_t i8_ld(int64_t K) { return (K + kI8Stage - 1) / kI8Stage * kI8Stage; }
// 127^2 K < 2^31
constexpr int64_t kMaxInt8K = 131072;
// the norm keeps per-channel values of a row in LDS
constexpr int64_t kMaxNormC = 4096;

}  // namespace svdq
