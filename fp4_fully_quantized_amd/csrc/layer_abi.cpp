// layer_abi.cpp -- C entry points of the operators around the FP4 product
// (declared in include/fp4.h; fp4_gemm_fused is in abi.cpp with the product):
// argument validation, then kernel launches on the caller's stream.
#include "layer_internal.hpp"

#include <cmath>
#include <cstdint>

#include "layer_checks.hpp"

using namespace fp4chk;

namespace {

constexpr int64_t kWsAlign = 256;

fp4_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return FP4_OK;
  if (!ws || have < need || reinterpret_cast<uintptr_t>(ws) % kWsAlign != 0) return FP4_ERR_WORKSPACE;
  return FP4_OK;
}

}  // namespace

extern "C" {

fp4_status fp4_mx8_quantize(const void* src, fp4_dtype src_t, int64_t ld, const fp4_mx8* q, fp4_stream_t stream) {
  if (!src || !q) return FP4_ERR_NULL;
  if (!dtype_ok(src_t)) return FP4_ERR_ARG;
  fp4_status st = check_mat(src, src_t, q->rows, q->cols, ld);
  if (st == FP4_OK) st = check_mx8(q, q->rows, q->cols);
  if (st != FP4_OK) return st;
  fp4i_launch_mx8_quant(src, src_t == FP4_DTYPE_BF16, ld, *q, reinterpret_cast<hipStream_t>(stream));
  return launched();
}

fp4_status fp4_mx8_dequantize(const fp4_mx8* q, fp4_dtype dst_t, void* dst, int64_t ld, fp4_stream_t stream) {
  if (!dst || !q) return FP4_ERR_NULL;
  if (!dtype_ok(dst_t)) return FP4_ERR_ARG;
  fp4_status st = check_mat(dst, dst_t, q->rows, q->cols, ld);
  if (st == FP4_OK) st = check_mx8(q, q->rows, q->cols);
  if (st != FP4_OK) return st;
  fp4i_launch_mx8_dequant(*q, dst_t == FP4_DTYPE_BF16, dst, ld, reinterpret_cast<hipStream_t>(stream));
  return launched();
}

fp4_status fp4_rmsnorm(const fp4_rmsnorm_fwd* n, fp4_stream_t stream) {
  if (!n || !n->x || !n->gamma || !(n->h || n->y || n->y8 || n->h8)) return FP4_ERR_NULL;
  if (n->amax && !n->y && !n->y8) return FP4_ERR_NULL;  // of no stored values
  if (!dtype_ok(n->dtype) || !dtype_ok(n->gamma_t)) return FP4_ERR_ARG;
  if (!(n->eps >= 0.0f) || std::isinf(n->eps)) return FP4_ERR_ARG;
  const int64_t R = n->rows, C = n->cols;
  fp4_status st = check_mat(n->x, n->dtype, R, C, n->ld_x);
  if (st == FP4_OK) st = check_opt(n->residual, n->dtype, R, C, n->ld_residual);
  if (st == FP4_OK) st = check_opt(n->h, n->dtype, R, C, n->ld_h);
  if (st == FP4_OK) st = check_opt(n->y, n->dtype, R, C, n->ld_y);
  if (st == FP4_OK) st = check_mat(n->gamma, n->gamma_t, 1, C, C);
  if (st == FP4_OK && n->y8) st = check_mx8(n->y8, R, C);
  if (st == FP4_OK && n->h8) st = check_mx8(n->h8, R, C);
  if (st == FP4_OK && (!aligned(n->rstd, 4) || !aligned(n->amax, 4))) st = FP4_ERR_ALIGN;
  if (st == FP4_OK) st = check_over(n->h, n->ld_h, n->x, n->ld_x, R);
  if (st == FP4_OK) st = check_over(n->h, n->ld_h, n->residual, n->ld_residual, R);
  if (st == FP4_OK) st = check_over(n->y, n->ld_y, n->x, n->ld_x, R);
  if (st == FP4_OK) st = check_over(n->y, n->ld_y, n->residual, n->ld_residual, R);
  if (st != FP4_OK) return st;
  fp4i_launch_rmsnorm(*n, reinterpret_cast<hipStream_t>(stream));
  return launched();
}

size_t fp4_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (!dims_ok(rows, cols)) return 0;
  const int64_t parts = fp4i_rmsnorm_bwd_parts(rows, cols);
  return parts > 1 ? (size_t)parts * (size_t)cols * 4 : 0;
}

fp4_status fp4_rmsnorm_backward(const fp4_rmsnorm_bwd* n, fp4_stream_t stream) {
  if (!n || !n->dy || !n->gamma || !n->rstd || !n->dx || (!n->h && !n->h8)) return FP4_ERR_NULL;
  if (!dtype_ok(n->dtype) || !dtype_ok(n->gamma_t) || (n->h && n->h8)) return FP4_ERR_ARG;
  const int64_t R = n->rows, C = n->cols;
  fp4_status st = check_mat(n->dy, n->dtype, R, C, n->ld_dy);
  if (st == FP4_OK) st = check_mat(n->dx, n->dtype, R, C, n->ld_dx);
  if (st == FP4_OK) st = check_opt(n->h, n->dtype, R, C, n->ld_h);
  if (st == FP4_OK) st = check_opt(n->dres, n->dtype, R, C, n->ld_dres);
  if (st == FP4_OK) st = check_mat(n->gamma, n->gamma_t, 1, C, C);
  if (st == FP4_OK && n->h8) st = check_mx8(n->h8, R, C);
  if (st == FP4_OK && (!aligned(n->rstd, 4) || !aligned(n->dgamma, 4))) st = FP4_ERR_ALIGN;
  if (st == FP4_OK && n->dgamma) st = check_ws(n->ws, n->ws_bytes, fp4_rmsnorm_backward_workspace_bytes(R, C));
  if (st == FP4_OK) st = check_over(n->dx, n->ld_dx, n->dy, n->ld_dy, R);
  if (st == FP4_OK) st = check_over(n->dx, n->ld_dx, n->dres, n->ld_dres, R);
  if (st != FP4_OK) return st;
  fp4i_launch_rmsnorm_bwd(*n, reinterpret_cast<hipStream_t>(stream));
  return launched();
}

size_t fp4_act_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (!dims_ok(rows, cols)) return 0;
  const ActPlan p = fp4i_act_plan(rows, cols);
  return p.parts * p.slabs == 1 ? 0 : (size_t)p.parts * ((size_t)cols + (size_t)p.slabs) * 4;
}

fp4_status fp4_act_backward(const fp4_act_bwd* n, fp4_stream_t stream) {
  if (!n || !n->dy || !n->dz || (!n->z && !n->z8)) return FP4_ERR_NULL;
  if (!dtype_ok(n->dtype) || !act_ok(n->act) || (n->z && n->z8)) return FP4_ERR_ARG;
  const int64_t R = n->rows, C = n->cols;
  fp4_status st = check_mat(n->dy, n->dtype, R, C, n->ld_dy);
  if (st == FP4_OK) st = check_mat(n->dz, n->dtype, R, C, n->ld_dz);
  if (st == FP4_OK) st = check_opt(n->z, n->dtype, R, C, n->ld_z);
  if (st == FP4_OK && n->z8) st = check_mx8(n->z8, R, C);
  if (st == FP4_OK && (!aligned(n->dbias, 4) || !aligned(n->amax, 4))) st = FP4_ERR_ALIGN;
  if (st == FP4_OK && (n->dbias || n->amax)) st = check_ws(n->ws, n->ws_bytes, fp4_act_backward_workspace_bytes(R, C));
  if (st == FP4_OK) st = check_over(n->dz, n->ld_dz, n->dy, n->ld_dy, R);
  if (st != FP4_OK) return st;
  fp4i_launch_act_bwd(*n, reinterpret_cast<hipStream_t>(stream));
  return launched();
}

}  // extern "C"
