// Argument checks that the C ABI's 8-bit layers and norms share (host code).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/svdq.h"
#include "int8_host.hpp"
#include "internal.hpp"

namespace svdq {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t rup(size_t x) { return (x + 255) & ~size_t(255); }
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

inline svdq_status check_xdtype(int32_t xdtype) {
  if (xdtype != SVDQ_F32 && xdtype != SVDQ_BF16) return fail(SVDQ_EUNSUPPORTED, "unsupported input dtype %d", (int)xdtype);
  return SVDQ_OK;
}

inline svdq_status check_k(int64_t K) {
  if (K < 1) return fail(SVDQ_EINVAL, "K must be >= 1 (got %lld)", (long long)K);
  if (K > kMaxInt8K) return fail(SVDQ_EUNSUPPORTED, "K must be <= %lld (got %lld)", (long long)kMaxInt8K, (long long)K);
  return SVDQ_OK;
}

inline svdq_status check_rows(int64_t M) {
  if (M < 0) return fail(SVDQ_EINVAL, "the number of rows must be >= 0");
  if (M > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "the number of rows must be < 2^31");
  return SVDQ_OK;
}

// a launch takes fewer than 2^32 threads: 256 or more to a tile, 512 to 16 channels where there are few tokens
inline svdq_status check_tiles(int64_t M, int64_t N) {
  const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64);
  if (tiles > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "M * N must be < 2^43");
  if (tiles >= int64_t(1) << 24) return fail(SVDQ_EUNSUPPORTED, "ceil(M / 64) * ceil(N / 64) must be < 2^24");
  if ((N + 15) / 16 >= int64_t(1) << 23) return fail(SVDQ_EUNSUPPORTED, "N must be <= 2^27 - 16");
  return SVDQ_OK;
}

inline svdq_status check_out(const void* Y, int64_t ldy, int64_t N, int32_t ydtype) {
  if (ydtype != SVDQ_F32 && ydtype != SVDQ_BF16 && ydtype != SVDQ_BF16_GELU)
    return fail(SVDQ_EUNSUPPORTED, "unsupported output dtype %d", (int)ydtype);
  if (!Y) return fail(SVDQ_EINVAL, "Y must be non-NULL");
  if (!aligned(Y, ydtype == SVDQ_F32 ? 4 : 2)) return fail(SVDQ_EINVAL, "Y must be aligned to its element size");
  if (ldy < N) return fail(SVDQ_EINVAL, "ldy must be >= N");
  if (ldy > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "ldy must be < 2^31");
  return SVDQ_OK;
}

inline svdq_status check_in(const void* X, int32_t xdtype, int64_t ldx, int64_t K) {
  svdq_status st = check_xdtype(xdtype);
  if (st != SVDQ_OK) return st;
  if (!X) return fail(SVDQ_EINVAL, "X must be non-NULL");
  if (!aligned(X, xdtype == SVDQ_F32 ? 4 : 2)) return fail(SVDQ_EINVAL, "X must be aligned to its element size");
  if (ldx < K) return fail(SVDQ_EINVAL, "ldx must be >= the row's length");
  if (ldx > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "ldx must be < 2^31");
  return SVDQ_OK;
}

inline svdq_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return SVDQ_OK;
  if (!ws || have < need) return fail(SVDQ_EINVAL, "workspace too small: need %zu bytes", need);
  if (!aligned(ws, 256)) return fail(SVDQ_EINVAL, "workspace must be 256-byte aligned");
  return SVDQ_OK;
}

}  // namespace svdq
