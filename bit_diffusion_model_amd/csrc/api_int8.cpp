// C ABI of the 8-bit layer and the channels-last group norm: argument validation, error
// reporting and kernel launches for the entry points declared in include/svdq.h.
#include <hip/hip_runtime.h>

#include "../../include/svdq.h"
#include "int8_host.hpp"
#include "internal.hpp"
#include "kernels.hpp"

namespace svdq {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t rup(size_t x) { return (x + 255) & ~size_t(255); }
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

svdq_status check_xdtype(int32_t xdtype) {
  if (xdtype != SVDQ_F32 && xdtype != SVDQ_BF16) return fail(SVDQ_EUNSUPPORTED, "unsupported input dtype %d", (int)xdtype);
  return SVDQ_OK;
}

svdq_status check_k(int64_t K) {
  if (K < 1) return fail(SVDQ_EINVAL, "K must be >= 1 (got %lld)", (long long)K);
  if (K > kMaxInt8K) return fail(SVDQ_EUNSUPPORTED, "K must be <= %lld (got %lld)", (long long)kMaxInt8K, (long long)K);
  return SVDQ_OK;
}

svdq_status check_rows(int64_t M) {
  if (M < 0) return fail(SVDQ_EINVAL, "the number of rows must be >= 0");
  if (M > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "the number of rows must be < 2^31");
  return SVDQ_OK;
}

svdq_status check_dims_int8(const svdq_int8_layer* L) {
  if (!L) return fail(SVDQ_EINVAL, "layer is NULL");
  svdq_status st = check_k(L->K);
  if (st != SVDQ_OK) return st;
  if (L->N < 1) return fail(SVDQ_EINVAL, "N must be >= 1 (got %lld)", (long long)L->N);
  if (L->N > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "N must be < 2^31");
  return SVDQ_OK;
}

// a launch takes fewer than 2^32 threads: 256 or more to a tile, 512 to 16 channels where there are few tokens
svdq_status check_tiles(int64_t M, int64_t N) {
  const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64);
  if (tiles > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "M * N must be < 2^43");
  if (tiles >= int64_t(1) << 24) return fail(SVDQ_EUNSUPPORTED, "ceil(M / 64) * ceil(N / 64) must be < 2^24");
  if ((N + 15) / 16 >= int64_t(1) << 23) return fail(SVDQ_EUNSUPPORTED, "N must be <= 2^27 - 16");
  return SVDQ_OK;
}

svdq_status check_layer_int8(const svdq_int8_layer* L) {
  svdq_status st = check_dims_int8(L);
  if (st != SVDQ_OK) return st;
  if (!L->qW || !L->sW) return fail(SVDQ_EINVAL, "layer qW and sW must be non-NULL");
  if (!aligned(L->qW, 16) || !aligned(L->sW, 16) || !aligned(L->inv_s, 16) || !aligned(L->bias, 16))
    return fail(SVDQ_EINVAL, "layer qW, sW, inv_s and bias must be 16-byte aligned");
  return SVDQ_OK;
}

svdq_status check_out(const void* Y, int64_t ldy, int64_t N, int32_t ydtype) {
  if (ydtype != SVDQ_F32 && ydtype != SVDQ_BF16 && ydtype != SVDQ_BF16_GELU)
    return fail(SVDQ_EUNSUPPORTED, "unsupported output dtype %d", (int)ydtype);
  if (!Y) return fail(SVDQ_EINVAL, "Y must be non-NULL");
  if (!aligned(Y, ydtype == SVDQ_F32 ? 4 : 2)) return fail(SVDQ_EINVAL, "Y must be aligned to its element size");
  if (ldy < N) return fail(SVDQ_EINVAL, "ldy must be >= N");
  if (ldy > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "ldy must be < 2^31");
  return SVDQ_OK;
}

svdq_status check_in(const void* X, int32_t xdtype, int64_t ldx, int64_t K) {
  svdq_status st = check_xdtype(xdtype);
  if (st != SVDQ_OK) return st;
  if (!X) return fail(SVDQ_EINVAL, "X must be non-NULL");
  if (!aligned(X, xdtype == SVDQ_F32 ? 4 : 2)) return fail(SVDQ_EINVAL, "X must be aligned to its element size");
  if (ldx < K) return fail(SVDQ_EINVAL, "ldx must be >= the row's length");
  if (ldx > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "ldx must be < 2^31");
  return SVDQ_OK;
}

svdq_status check_codes(const int8_t* qX, const float* sX) {
  if (!qX || !sX) return fail(SVDQ_EINVAL, "qX and sX must be non-NULL");
  if (!aligned(qX, 16) || !aligned(sX, 4)) return fail(SVDQ_EINVAL, "qX must be 16-byte and sX 4-byte aligned");
  return SVDQ_OK;
}

svdq_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return SVDQ_OK;
  if (!ws || have < need) return fail(SVDQ_EINVAL, "workspace too small: need %zu bytes", need);
  if (!aligned(ws, 256)) return fail(SVDQ_EINVAL, "workspace must be 256-byte aligned");
  return SVDQ_OK;
}

svdq_status check_norm(const svdq_group_norm_desc* n, int64_t B, int64_t S) {
  if (!n) return fail(SVDQ_EINVAL, "norm is NULL");
  if (n->C < 1 || n->groups < 1 || n->C % n->groups != 0)
    return fail(SVDQ_EINVAL, "C must be a positive multiple of groups (got %lld, %d)", (long long)n->C, (int)n->groups);
  if (n->C > kMaxNormC || n->groups > kMaxNormG)
    return fail(SVDQ_EUNSUPPORTED, "C must be <= %lld and groups <= %d", (long long)kMaxNormC, kMaxNormG);
  if (n->act != SVDQ_GN_NONE && n->act != SVDQ_GN_SILU && n->act != SVDQ_GN_GELU)
    return fail(SVDQ_EUNSUPPORTED, "unknown activation %d", (int)n->act);
  if (!(n->eps > 0.0f && n->eps < 3.0e38f)) return fail(SVDQ_EINVAL, "eps must be positive and finite");
  if (!aligned(n->gamma, 16) || !aligned(n->beta, 16)) return fail(SVDQ_EINVAL, "gamma and beta must be 16-byte aligned");
  if (B < 0 || S < 0) return fail(SVDQ_EINVAL, "B and S must be >= 0");
  if (B > 65535 || S > kMaxRows || B * S > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "B must be <= 65535 and B * S < 2^31");
  return SVDQ_OK;
}

svdq_status norm_args(const svdq_group_norm_desc* n, int64_t B, int64_t S, const void* X, int32_t xdtype, int64_t bsx,
                      int64_t ldx, NormArgs& a) {
  svdq_status st = check_in(X, xdtype, ldx, n->C);
  if (st != SVDQ_OK) return st;
  // images are apart, or one and the same (with one image the stride is not used)
  if (B > 1 && bsx >= (int64_t(1) << 46)) return fail(SVDQ_EUNSUPPORTED, "bsx must be < 2^46");
  if (B > 1 && bsx != 0 && (bsx < n->C || (bsx < (S - 1) * ldx + n->C && ldx < (B - 1) * bsx + n->C)))
    return fail(SVDQ_EINVAL, "bsx must be 0 or >= (S - 1) * ldx + C");
  a = NormArgs{B, S, (int)n->C, n->groups, n->act, n->eps, n->gamma, n->beta, X, xdtype, B > 1 ? bsx : 0, ldx};
  return SVDQ_OK;
}

size_t act_bytes(int64_t M, int64_t K) { return rup((size_t)M * (size_t)i8_ld(K)) + rup((size_t)M * 4); }

svdq_status run_gemm(const svdq_int8_layer* L, int64_t M, const int8_t* qX, const float* sX, void* Y, int64_t ldy,
                     int32_t ydtype, void* ws, size_t ws_bytes, void* stream) {
  svdq_status st = check_codes(qX, sX);
  if (st != SVDQ_OK || (st = check_out(Y, ldy, L->N, ydtype)) != SVDQ_OK) return st;
  if ((st = check_tiles(M, L->N)) != SVDQ_OK) return st;
  hipError_t e = launch_w8a8(M, L->K, L->N, qX, sX, L->qW, L->sW, L->bias, Y, ldy, ydtype, ws, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "W8A8 product launch: %s", hipGetErrorString(e));
  return ok();
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" {

size_t svdq_gemm_w8a8_workspace_bytes(const svdq_int8_layer* layer, int64_t M) {
  if (M < 1 || check_dims_int8(layer) != SVDQ_OK || check_rows(M) != SVDQ_OK || check_tiles(M, layer->N) != SVDQ_OK) return 0;
  return rup(plan_w8a8(M, layer->K, layer->N).bytes);
}

size_t svdq_int8_workspace_bytes(const svdq_int8_layer* layer, int64_t M, int32_t xdtype) {
  if (M < 1 || check_dims_int8(layer) != SVDQ_OK || check_rows(M) != SVDQ_OK || check_xdtype(xdtype) != SVDQ_OK ||
      check_tiles(M, layer->N) != SVDQ_OK)
    return 0;
  if (few_layer(M, layer->K)) return 0;
  return act_bytes(M, layer->K) + svdq_gemm_w8a8_workspace_bytes(layer, M);
}

svdq_status svdq_quantize_act_int8(int64_t M, int64_t K, const void* X, int32_t xdtype, int64_t ldx,
                                   const float* inv_s, int8_t* qX, float* sX, void* stream) {
  svdq_status st = check_k(K);
  if (st != SVDQ_OK || (st = check_rows(M)) != SVDQ_OK) return st;
  if (M == 0) return ok();
  if ((st = check_in(X, xdtype, ldx, K)) != SVDQ_OK || (st = check_codes(qX, sX)) != SVDQ_OK) return st;
  if (!aligned(inv_s, 16)) return fail(SVDQ_EINVAL, "inv_s must be 16-byte aligned");
  hipError_t e = launch_quant_i8(M, K, X, xdtype, ldx, inv_s, qX, sX, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "8-bit quantizer launch: %s", hipGetErrorString(e));
  return ok();
}

svdq_status svdq_gemm_w8a8(const svdq_int8_layer* layer, int64_t M, const int8_t* qX, const float* sX, void* Y,
                           int64_t ldy, int32_t ydtype, void* workspace, size_t ws_bytes, void* stream) {
  svdq_status st = check_layer_int8(layer);
  if (st != SVDQ_OK || (st = check_rows(M)) != SVDQ_OK) return st;
  if (M == 0) return ok();
  if ((st = check_ws(workspace, ws_bytes, svdq_gemm_w8a8_workspace_bytes(layer, M))) != SVDQ_OK) return st;
  return run_gemm(layer, M, qX, sX, Y, ldy, ydtype, workspace, ws_bytes, stream);
}

svdq_status svdq_linear_forward_int8(const svdq_int8_layer* layer, int64_t M, const void* X, int32_t xdtype,
                                     int64_t ldx, void* Y, int64_t ldy, int32_t ydtype, void* workspace,
                                     size_t ws_bytes, void* stream) {
  svdq_status st = check_layer_int8(layer);
  if (st != SVDQ_OK || (st = check_rows(M)) != SVDQ_OK) return st;
  if (M == 0) return ok();
  if ((st = check_in(X, xdtype, ldx, layer->K)) != SVDQ_OK || (st = check_out(Y, ldy, layer->N, ydtype)) != SVDQ_OK ||
      (st = check_tiles(M, layer->N)) != SVDQ_OK)
    return st;
  if ((st = check_ws(workspace, ws_bytes, svdq_int8_workspace_bytes(layer, M, xdtype))) != SVDQ_OK) return st;
  hipError_t e;
  if (few_layer(M, layer->K)) {
    e = launch_few_layer(M, layer->K, layer->N, X, xdtype, ldx, layer->inv_s, layer->qW, layer->sW, layer->bias, Y, ldy,
                         ydtype, (hipStream_t)stream);
    if (e != hipSuccess) return fail(SVDQ_EHIP, "8-bit layer launch: %s", hipGetErrorString(e));
    return ok();
  }
  uint8_t* base = static_cast<uint8_t*>(workspace);
  int8_t* qX = reinterpret_cast<int8_t*>(base);
  float* sX = reinterpret_cast<float*>(base + rup((size_t)M * (size_t)i8_ld(layer->K)));
  const size_t used = act_bytes(M, layer->K);
  e = launch_quant_i8(M, layer->K, X, xdtype, ldx, layer->inv_s, qX, sX, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "8-bit quantizer launch: %s", hipGetErrorString(e));
  return run_gemm(layer, M, qX, sX, Y, ldy, ydtype, base + used, ws_bytes - used, stream);
}

size_t svdq_group_norm_quantize_workspace_bytes(const svdq_group_norm_desc* norm, int64_t B, int64_t S) {
  if (check_norm(norm, B, S) != SVDQ_OK || B == 0 || S == 0) return 0;
  return rup(plan_norm(B, S, (int)norm->C, norm->groups).bytes);
}

size_t svdq_group_norm_workspace_bytes(const svdq_group_norm_desc* norm, int64_t B, int64_t S) {
  if (check_norm(norm, B, S) != SVDQ_OK || B == 0 || S == 0) return 0;
  const NormPlan p = plan_norm(B, S, (int)norm->C, norm->groups);
  return p.one ? 0 : rup(p.bytes);  // one launch needs none
}

svdq_status svdq_group_norm(const svdq_group_norm_desc* norm, int64_t B, int64_t S, const void* X, int32_t xdtype,
                            int64_t bsx, int64_t ldx, void* Y, int32_t ydtype, int64_t bsy, int64_t ldy,
                            void* workspace, size_t ws_bytes, void* stream) {
  svdq_status st = check_norm(norm, B, S);
  if (st != SVDQ_OK) return st;
  if (B == 0 || S == 0) return ok();
  NormArgs a;
  if ((st = norm_args(norm, B, S, X, xdtype, bsx, ldx, a)) != SVDQ_OK) return st;
  if (ydtype != SVDQ_F32 && ydtype != SVDQ_BF16) return fail(SVDQ_EUNSUPPORTED, "unsupported output dtype %d", (int)ydtype);
  if ((st = check_out(Y, ldy, norm->C, ydtype)) != SVDQ_OK) return st;
  if (B > 1 && bsy >= (int64_t(1) << 46)) return fail(SVDQ_EUNSUPPORTED, "bsy must be < 2^46");
  if (B > 1 && (bsy < norm->C || (bsy < (S - 1) * ldy + norm->C && ldy < (B - 1) * bsy + norm->C)))
    return fail(SVDQ_EINVAL, "bsy must be >= (S - 1) * ldy + C");
  if ((st = check_ws(workspace, ws_bytes, svdq_group_norm_workspace_bytes(norm, B, S))) != SVDQ_OK) return st;
  hipError_t e = launch_norm(a, Y, ydtype, B > 1 ? bsy : 0, ldy, workspace, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "group norm launch: %s", hipGetErrorString(e));
  return ok();
}

svdq_status svdq_group_norm_quantize_int8(const svdq_group_norm_desc* norm, int64_t B, int64_t S, const void* X,
                                          int32_t xdtype, int64_t bsx, int64_t ldx, const float* inv_s, int8_t* qX,
                                          float* sX, void* workspace, size_t ws_bytes, void* stream) {
  svdq_status st = check_norm(norm, B, S);
  if (st != SVDQ_OK) return st;
  if (B == 0 || S == 0) return ok();
  NormArgs a;
  if ((st = norm_args(norm, B, S, X, xdtype, bsx, ldx, a)) != SVDQ_OK || (st = check_codes(qX, sX)) != SVDQ_OK) return st;
  if (!aligned(inv_s, 16)) return fail(SVDQ_EINVAL, "inv_s must be 16-byte aligned");
  if ((st = check_ws(workspace, ws_bytes, svdq_group_norm_quantize_workspace_bytes(norm, B, S))) != SVDQ_OK) return st;
  hipError_t e = launch_norm_quant(a, inv_s, qX, sX, workspace, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "group norm launch: %s", hipGetErrorString(e));
  return ok();
}

svdq_status svdq_debug_w8a8_plan(const svdq_int8_layer* layer, int64_t M, int32_t plan[4]) {
  svdq_status st = check_dims_int8(layer);
  if (st != SVDQ_OK || (st = check_rows(M)) != SVDQ_OK || (st = check_tiles(M, layer->N)) != SVDQ_OK) return st;
  if (M < 1 || !plan) return fail(SVDQ_EINVAL, "M must be >= 1 and plan non-NULL");
  const W8A8Plan p = plan_w8a8(M, layer->K, layer->N);
  plan[0] = p.tile, plan[1] = p.groups, plan[2] = p.parts, plan[3] = (int32_t)p.halved;
  return ok();
}

svdq_status svdq_debug_group_norm_plan(const svdq_group_norm_desc* norm, int64_t B, int64_t S, int32_t plan[4]) {
  svdq_status st = check_norm(norm, B, S);
  if (st != SVDQ_OK) return st;
  if (B < 1 || S < 1 || !plan) return fail(SVDQ_EINVAL, "B and S must be >= 1 and plan non-NULL");
  const NormPlan p = plan_norm(B, S, (int)norm->C, norm->groups);
  plan[0] = p.one, plan[1] = p.join, plan[2] = (int32_t)p.parts, plan[3] = (int32_t)p.blocks;
  return ok();
}

size_t svdq_norm_linear_int8_workspace_bytes(const svdq_group_norm_desc* norm, const svdq_int8_layer* layer,
                                             int64_t B, int64_t S) {
  const size_t n = svdq_group_norm_quantize_workspace_bytes(norm, B, S);
  if (n == 0 || check_dims_int8(layer) != SVDQ_OK || layer->K != norm->C || check_tiles(B * S, layer->N) != SVDQ_OK) return 0;
  return n + act_bytes(B * S, layer->K) + svdq_gemm_w8a8_workspace_bytes(layer, B * S);
}

svdq_status svdq_norm_linear_forward_int8(const svdq_group_norm_desc* norm, const svdq_int8_layer* layer, int64_t B,
                                          int64_t S, const void* X, int32_t xdtype, int64_t bsx, int64_t ldx, void* Y,
                                          int64_t ldy, int32_t ydtype, void* workspace, size_t ws_bytes,
                                          void* stream) {
  svdq_status st = check_norm(norm, B, S);
  if (st != SVDQ_OK || (st = check_layer_int8(layer)) != SVDQ_OK) return st;
  if (layer->K != norm->C)
    return fail(SVDQ_EINVAL, "the layer's K (%lld) must equal the norm's C (%lld)", (long long)layer->K, (long long)norm->C);
  if (B == 0 || S == 0) return ok();
  const int64_t M = B * S;
  NormArgs a;
  if ((st = norm_args(norm, B, S, X, xdtype, bsx, ldx, a)) != SVDQ_OK ||
      (st = check_out(Y, ldy, layer->N, ydtype)) != SVDQ_OK || (st = check_tiles(M, layer->N)) != SVDQ_OK ||
      (st = check_ws(workspace, ws_bytes, svdq_norm_linear_int8_workspace_bytes(norm, layer, B, S))) != SVDQ_OK)
    return st;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  const size_t q = svdq_group_norm_quantize_workspace_bytes(norm, B, S);
  int8_t* qX = reinterpret_cast<int8_t*>(base + q);
  float* sX = reinterpret_cast<float*>(base + q + rup((size_t)M * (size_t)i8_ld(layer->K)));
  const size_t used = q + act_bytes(M, layer->K);
  hipError_t e = launch_norm_quant(a, layer->inv_s, qX, sX, base, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "group norm launch: %s", hipGetErrorString(e));
  return run_gemm(layer, M, qX, sX, Y, ldy, ydtype, base + used, ws_bytes - used, stream);
}

}  // extern "C"
