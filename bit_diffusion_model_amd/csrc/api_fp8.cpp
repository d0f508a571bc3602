// C ABI of the block-scaled 8-bit floating point layer and the layer norm: argument validation, error reporting and
// kernel launches for the entry points declared in include/svdq.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/svdq.h"
#include "api_checks.hpp"
#include "int8_host.hpp"
#include "internal.hpp"
#include "kernels.hpp"

namespace svdq {
namespace {

constexpr int64_t kMaxStride = int64_t(1) << 46;

svdq_status check_dims_fp8(const svdq_fp8_layer* L) {
  if (!L) return fail(SVDQ_EINVAL, "layer is NULL");
  svdq_status st = check_k(L->K);
  if (st != SVDQ_OK) return st;
  if (L->N < 1) return fail(SVDQ_EINVAL, "N must be >= 1 (got %lld)", (long long)L->N);
  if (L->N > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "N must be < 2^31");
  return SVDQ_OK;
}

svdq_status check_layer_fp8(const svdq_fp8_layer* L) {
  svdq_status st = check_dims_fp8(L);
  if (st != SVDQ_OK) return st;
  if (!L->qW || !L->sW) return fail(SVDQ_EINVAL, "layer qW and sW must be non-NULL");
  if (!aligned(L->qW, 16) || !aligned(L->sW, 16) || !aligned(L->bias, 16))
    return fail(SVDQ_EINVAL, "layer qW, sW and bias must be 16-byte aligned");
  return SVDQ_OK;
}

svdq_status check_codes_fp8(const uint8_t* qX, const float* sX) {
  if (!qX || !sX) return fail(SVDQ_EINVAL, "qX and sX must be non-NULL");
  if (!aligned(qX, 16) || !aligned(sX, 16)) return fail(SVDQ_EINVAL, "qX and sX must be 16-byte aligned");
  return SVDQ_OK;
}

// codes and scales of M rows, each 256-byte aligned
size_t codes_bytes(int64_t M, int64_t K) { return rup((size_t)M * (size_t)i8_ld(K)); }
size_t act_bytes_fp8(int64_t M, int64_t K) {
  return codes_bytes(M, K) + rup((size_t)((M + 3) / 4 * 4) * (size_t)(i8_ld(K) / 128) * 4);
}

svdq_status run_gemm_fp8(const svdq_fp8_layer* L, int64_t M, const uint8_t* qX, const float* sX, void* Y, int64_t ldy,
                         int32_t ydtype, void* ws, void* stream) {
  hipError_t e = launch_gemm_fp8(M, L->K, L->N, qX, sX, L->qW, L->sW, L->bias, Y, ldy, ydtype, ws, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "block-scaled product launch: %s", hipGetErrorString(e));
  return ok();
}

svdq_status check_layer_norm(const svdq_layer_norm_desc* n, int64_t B, int64_t S) {
  if (!n) return fail(SVDQ_EINVAL, "norm is NULL");
  if (n->C < 1) return fail(SVDQ_EINVAL, "C must be >= 1 (got %lld)", (long long)n->C);
  if (n->C > kMaxLayerNormC)
    return fail(SVDQ_EUNSUPPORTED, "C must be <= %lld (got %lld)", (long long)kMaxLayerNormC, (long long)n->C);
  if (!(n->eps >= 1.17549435e-38f && n->eps < 3.0e38f)) return fail(SVDQ_EINVAL, "eps must be positive, normal and finite");
  if (n->one_plus != 0 && n->one_plus != 1) return fail(SVDQ_EINVAL, "one_plus must be 0 or 1");
  if (!aligned(n->gamma, 4) || !aligned(n->beta, 4)) return fail(SVDQ_EINVAL, "gamma and beta must be 4-byte aligned");
  if (B < 0 || S < 0) return fail(SVDQ_EINVAL, "B and S must be >= 0");
  if (B > 65535 || S > kMaxRows || B * S > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "B must be <= 65535 and B * S < 2^31");
  if (n->image_stride != 0 && n->image_stride < n->C) return fail(SVDQ_EINVAL, "image_stride must be 0 or >= C");
  if (n->image_stride >= kMaxStride) return fail(SVDQ_EUNSUPPORTED, "image_stride must be < 2^46");
  return SVDQ_OK;
}

// Images of rows are apart (or, where `same` allows it, one and the same): with one image the stride is not used.
svdq_status check_images(const char* name, int64_t B, int64_t S, int64_t C, int64_t bs, int64_t ld, bool same) {
  if (B <= 1 || (same && bs == 0)) return SVDQ_OK;
  if (bs >= kMaxStride) return fail(SVDQ_EUNSUPPORTED, "%s: the image stride must be < 2^46", name);
  if (bs < C || (bs < (S - 1) * ld + C && ld < (B - 1) * bs + C))
    return fail(SVDQ_EINVAL, "%s: the image stride must be %s>= (S - 1) * row stride + C", name, same ? "0 or " : "");
  return SVDQ_OK;
}

svdq_status layer_norm_args(const svdq_layer_norm_desc* n, int64_t B, int64_t S, const void* X, int32_t xdtype,
                            int64_t bsx, int64_t ldx, LayerNormArgs& a) {
  svdq_status st = check_in(X, xdtype, ldx, n->C);
  if (st != SVDQ_OK || (st = check_images("X", B, S, n->C, bsx, ldx, true)) != SVDQ_OK) return st;
  a = LayerNormArgs{B, S, (int)n->C, n->one_plus != 0, n->eps, n->gamma, n->beta, n->image_stride,
                    X, xdtype, B > 1 ? bsx : 0, ldx, 0, 0};
  return SVDQ_OK;
}

svdq_status check_stats(const float* mean, const float* rstd) {
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return fail(SVDQ_EINVAL, "mean and rstd must be 4-byte aligned");
  return SVDQ_OK;
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" {

size_t svdq_gemm_fp8_workspace_bytes(const svdq_fp8_layer* layer, int64_t M) {
  if (M < 1 || check_dims_fp8(layer) != SVDQ_OK || check_rows(M) != SVDQ_OK || check_tiles(M, layer->N) != SVDQ_OK) return 0;
  return rup(std::max(plan_fp8(M, layer->K, layer->N, false).bytes, plan_fp8(M, layer->K, layer->N, true).bytes));
}

size_t svdq_fp8_workspace_bytes(const svdq_fp8_layer* layer, int64_t M) {
  if (M < 1 || check_dims_fp8(layer) != SVDQ_OK || check_rows(M) != SVDQ_OK || check_tiles(M, layer->N) != SVDQ_OK) return 0;
  if (few_layer_fp8(M, layer->K)) return 0;
  return act_bytes_fp8(M, layer->K) + svdq_gemm_fp8_workspace_bytes(layer, M);
}

svdq_status svdq_quantize_act_fp8(int64_t M, int64_t K, const void* X, int32_t xdtype, int64_t ldx, uint8_t* qX,
                                  float* sX, void* stream) {
  svdq_status st = check_k(K);
  if (st != SVDQ_OK || (st = check_rows(M)) != SVDQ_OK) return st;
  if (M == 0) return ok();
  if ((st = check_in(X, xdtype, ldx, K)) != SVDQ_OK || (st = check_codes_fp8(qX, sX)) != SVDQ_OK) return st;
  hipError_t e = launch_quant_fp8(M, K, X, xdtype, ldx, qX, sX, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "block quantizer launch: %s", hipGetErrorString(e));
  return ok();
}

svdq_status svdq_gemm_fp8(const svdq_fp8_layer* layer, int64_t M, const uint8_t* qX, const float* sX, void* Y,
                          int64_t ldy, int32_t ydtype, void* workspace, size_t ws_bytes, void* stream) {
  svdq_status st = check_layer_fp8(layer);
  if (st != SVDQ_OK || (st = check_rows(M)) != SVDQ_OK) return st;
  if (M == 0) return ok();
  if ((st = check_codes_fp8(qX, sX)) != SVDQ_OK || (st = check_out(Y, ldy, layer->N, ydtype)) != SVDQ_OK ||
      (st = check_tiles(M, layer->N)) != SVDQ_OK ||
      (st = check_ws(workspace, ws_bytes, svdq_gemm_fp8_workspace_bytes(layer, M))) != SVDQ_OK)
    return st;
  return run_gemm_fp8(layer, M, qX, sX, Y, ldy, ydtype, workspace, stream);
}

svdq_status svdq_linear_forward_fp8(const svdq_fp8_layer* layer, int64_t M, const void* X, int32_t xdtype, int64_t ldx,
                                    void* Y, int64_t ldy, int32_t ydtype, void* workspace, size_t ws_bytes,
                                    void* stream) {
  svdq_status st = check_layer_fp8(layer);
  if (st != SVDQ_OK || (st = check_rows(M)) != SVDQ_OK) return st;
  if (M == 0) return ok();
  if ((st = check_in(X, xdtype, ldx, layer->K)) != SVDQ_OK || (st = check_out(Y, ldy, layer->N, ydtype)) != SVDQ_OK ||
      (st = check_tiles(M, layer->N)) != SVDQ_OK ||
      (st = check_ws(workspace, ws_bytes, svdq_fp8_workspace_bytes(layer, M))) != SVDQ_OK)
    return st;
  hipError_t e;
  if (few_layer_fp8(M, layer->K)) {
    e = launch_few_layer_fp8(M, layer->K, layer->N, X, xdtype, ldx, layer->qW, layer->sW, layer->bias, Y, ldy, ydtype,
                             (hipStream_t)stream);
    if (e != hipSuccess) return fail(SVDQ_EHIP, "block-scaled layer launch: %s", hipGetErrorString(e));
    return ok();
  }
  uint8_t* base = static_cast<uint8_t*>(workspace);
  float* sX = reinterpret_cast<float*>(base + codes_bytes(M, layer->K));
  e = launch_quant_fp8(M, layer->K, X, xdtype, ldx, base, sX, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "block quantizer launch: %s", hipGetErrorString(e));
  return run_gemm_fp8(layer, M, base, sX, Y, ldy, ydtype, base + act_bytes_fp8(M, layer->K), stream);
}

svdq_status svdq_debug_fp8_plan(const svdq_fp8_layer* layer, int64_t M, int32_t ydtype, int32_t plan[4]) {
  svdq_status st = check_dims_fp8(layer);
  if (st != SVDQ_OK || (st = check_rows(M)) != SVDQ_OK || (st = check_tiles(M, layer->N)) != SVDQ_OK) return st;
  if (M < 1 || !plan) return fail(SVDQ_EINVAL, "M must be >= 1 and plan non-NULL");
  const Fp8Plan p = plan_fp8(M, layer->K, layer->N, ydtype == SVDQ_F32);
  plan[0] = p.rows, plan[1] = p.cols, plan[2] = p.groups, plan[3] = p.parts;
  return ok();
}

svdq_status svdq_debug_layer_norm_plan(const svdq_layer_norm_desc* norm, int64_t B, int64_t S, int32_t plan[4]) {
  svdq_status st = check_layer_norm(norm, B, S);
  if (st != SVDQ_OK) return st;
  if (B < 1 || S < 1 || !plan) return fail(SVDQ_EINVAL, "B and S must be >= 1 and plan non-NULL");
  const LayerNormPlan p = plan_layer_norm(B * S, (int)norm->C);
  const LayerNormGradPlan g = plan_layer_norm_grad(B, S, (int)norm->C, norm->image_stride != 0, true, true);
  plan[0] = p.lanes, plan[1] = p.chunks, plan[2] = p.waves, plan[3] = g.cw ? -g.cw : (int32_t)g.parts;
  return ok();
}

svdq_status svdq_layer_norm(const svdq_layer_norm_desc* norm, int64_t B, int64_t S, const void* X, int32_t xdtype,
                            int64_t bsx, int64_t ldx, void* Y, int32_t ydtype, int64_t bsy, int64_t ldy, float* mean,
                            float* rstd, void* stream) {
  svdq_status st = check_layer_norm(norm, B, S);
  if (st != SVDQ_OK) return st;
  if (B == 0 || S == 0) return ok();
  LayerNormArgs a;
  if ((st = layer_norm_args(norm, B, S, X, xdtype, bsx, ldx, a)) != SVDQ_OK) return st;
  if (ydtype != SVDQ_F32 && ydtype != SVDQ_BF16) return fail(SVDQ_EUNSUPPORTED, "unsupported output dtype %d", (int)ydtype);
  if ((st = check_out(Y, ldy, norm->C, ydtype)) != SVDQ_OK ||
      (st = check_images("Y", B, S, norm->C, bsy, ldy, false)) != SVDQ_OK || (st = check_stats(mean, rstd)) != SVDQ_OK)
    return st;
  hipError_t e = launch_layer_norm(a, Y, ydtype, B > 1 ? bsy : 0, ldy, mean, rstd, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "layer norm launch: %s", hipGetErrorString(e));
  return ok();
}

svdq_status svdq_layer_norm_quantize_fp8(const svdq_layer_norm_desc* norm, int64_t B, int64_t S, const void* X,
                                         int32_t xdtype, int64_t bsx, int64_t ldx, uint8_t* qX, float* sX, float* mean,
                                         float* rstd, void* stream) {
  svdq_status st = check_layer_norm(norm, B, S);
  if (st != SVDQ_OK) return st;
  if (B == 0 || S == 0) return ok();
  LayerNormArgs a;
  if ((st = layer_norm_args(norm, B, S, X, xdtype, bsx, ldx, a)) != SVDQ_OK || (st = check_codes_fp8(qX, sX)) != SVDQ_OK ||
      (st = check_stats(mean, rstd)) != SVDQ_OK)
    return st;
  hipError_t e = launch_layer_norm_fp8(a, qX, sX, mean, rstd, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "layer norm launch: %s", hipGetErrorString(e));
  return ok();
}

size_t svdq_norm_linear_fp8_workspace_bytes(const svdq_layer_norm_desc* norm, const svdq_fp8_layer* layer, int64_t B,
                                            int64_t S) {
  if (check_layer_norm(norm, B, S) != SVDQ_OK || B == 0 || S == 0) return 0;
  if (check_dims_fp8(layer) != SVDQ_OK || layer->K != norm->C || check_tiles(B * S, layer->N) != SVDQ_OK) return 0;
  return act_bytes_fp8(B * S, layer->K) + svdq_gemm_fp8_workspace_bytes(layer, B * S);
}

svdq_status svdq_norm_linear_forward_fp8(const svdq_layer_norm_desc* norm, const svdq_fp8_layer* layer, int64_t B,
                                         int64_t S, const void* X, int32_t xdtype, int64_t bsx, int64_t ldx, void* Y,
                                         int64_t ldy, int32_t ydtype, float* mean, float* rstd, void* workspace,
                                         size_t ws_bytes, void* stream) {
  svdq_status st = check_layer_norm(norm, B, S);
  if (st != SVDQ_OK || (st = check_layer_fp8(layer)) != SVDQ_OK) return st;
  if (layer->K != norm->C)
    return fail(SVDQ_EINVAL, "the layer's K (%lld) must equal the norm's C (%lld)", (long long)layer->K, (long long)norm->C);
  if (B == 0 || S == 0) return ok();
  const int64_t M = B * S;
  LayerNormArgs a;
  if ((st = layer_norm_args(norm, B, S, X, xdtype, bsx, ldx, a)) != SVDQ_OK ||
      (st = check_out(Y, ldy, layer->N, ydtype)) != SVDQ_OK || (st = check_tiles(M, layer->N)) != SVDQ_OK ||
      (st = check_stats(mean, rstd)) != SVDQ_OK ||
      (st = check_ws(workspace, ws_bytes, svdq_norm_linear_fp8_workspace_bytes(norm, layer, B, S))) != SVDQ_OK)
    return st;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  float* sX = reinterpret_cast<float*>(base + codes_bytes(M, layer->K));
  hipError_t e = launch_layer_norm_fp8(a, base, sX, mean, rstd, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "layer norm launch: %s", hipGetErrorString(e));
  return run_gemm_fp8(layer, M, base, sX, Y, ldy, ydtype, base + act_bytes_fp8(M, layer->K), stream);
}

size_t svdq_layer_norm_backward_workspace_bytes(const svdq_layer_norm_desc* norm, int64_t B, int64_t S) {
  if (check_layer_norm(norm, B, S) != SVDQ_OK || B == 0 || S == 0) return 0;
  return rup(plan_layer_norm_grad(B, S, (int)norm->C, norm->image_stride != 0, true, false).bytes);
}

svdq_status svdq_layer_norm_backward(const svdq_layer_norm_desc* norm, int64_t B, int64_t S, const void* dY,
                                     int32_t dydtype, int64_t bsdy, int64_t lddy, const void* X, int32_t xdtype,
                                     int64_t bsx, int64_t ldx, const float* mean, const float* rstd, void* dX,
                                     int64_t bsdx, int64_t lddx, float* dgamma, float* dbeta, void* workspace,
                                     size_t ws_bytes, void* stream) {
  svdq_status st = check_layer_norm(norm, B, S);
  if (st != SVDQ_OK) return st;
  if (!aligned(dgamma, 4) || !aligned(dbeta, 4)) return fail(SVDQ_EINVAL, "dgamma and dbeta must be 4-byte aligned");
  if (B == 0 || S == 0) {  // no rows: empty sums
    const int64_t runs = norm->image_stride ? B : 1;
    if (runs == 0 || (!dgamma && !dbeta)) return ok();
    hipError_t e = launch_layer_norm_no_rows(runs, (int)norm->C, dgamma, dbeta, (hipStream_t)stream);
    if (e != hipSuccess) return fail(SVDQ_EHIP, "layer norm gradient launch: %s", hipGetErrorString(e));
    return ok();
  }
  LayerNormArgs a;
  if ((st = layer_norm_args(norm, B, S, X, xdtype, bsx, ldx, a)) != SVDQ_OK) return st;
  if ((st = check_xdtype(dydtype)) != SVDQ_OK) return st;
  if (!dY || !aligned(dY, dydtype == SVDQ_F32 ? 4 : 2) || lddy < norm->C)
    return fail(SVDQ_EINVAL, "dY must be non-NULL, aligned to its element size, and its row stride >= C");
  if (lddy > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "dY: the row stride must be < 2^31");
  if ((st = check_images("dY", B, S, norm->C, bsdy, lddy, true)) != SVDQ_OK) return st;
  if (!mean || !rstd) return fail(SVDQ_EINVAL, "mean and rstd must be non-NULL");
  if ((st = check_stats(mean, rstd)) != SVDQ_OK) return st;
  if (!dX || !aligned(dX, xdtype == SVDQ_F32 ? 4 : 2) || lddx < norm->C)
    return fail(SVDQ_EINVAL, "dX must be non-NULL, aligned to its element size, and its row stride >= C");
  if (lddx > kMaxRows) return fail(SVDQ_EUNSUPPORTED, "dX: the row stride must be < 2^31");
  if ((st = check_images("dX", B, S, norm->C, bsdx, lddx, false)) != SVDQ_OK) return st;
  if ((dgamma || dbeta) &&
      (st = check_ws(workspace, ws_bytes, svdq_layer_norm_backward_workspace_bytes(norm, B, S))) != SVDQ_OK)
    return st;
  hipError_t e = launch_layer_norm_grad(a, dY, dydtype, B > 1 ? bsdy : 0, lddy, mean, rstd, dX, B > 1 ? bsdx : 0, lddx,
                                        dgamma, dbeta, workspace, (hipStream_t)stream);
  if (e != hipSuccess) return fail(SVDQ_EHIP, "layer norm gradient launch: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"
