// Entry points of the norm behind a residual addition: argument validation and
// launches.
#include <cmath>

#include "host.h"
#include "internal.h"
#include "row_args.h"

using namespace qlora;

extern "C" {

int qlora_add_norm_fwd(const void* x, int64_t ldx, int x_dtype, const void* residual, int64_t ldr,
                       int r_dtype, int64_t M, int64_t N, int norm, const void* gamma,
                       const void* beta, int w_dtype, float eps, void* h, int64_t ldh, void* y,
                       int64_t ldy, int y_dtype, float* scales, float* stats, void* stream) {
  if (M < 0 || (norm != QLORA_NORM_LAYER && norm != QLORA_NORM_RMS) || !std::isfinite(eps) ||
      eps < 0.0f)
    return QLORA_ERR_INVALID_ARG;
  if (!norm_shape_ok(M, N) || !stride_ok(M, N, ldx) || !stride_ok(M, N, ldy) ||
      (residual && (!stride_ok(M, N, ldr) || !stride_ok(M, N, ldh))))
    return QLORA_ERR_SHAPE;
  const bool codes = y_dtype == QLORA_DTYPE_E4M3;
  if (!float_type(x_dtype) || (residual && !float_type(r_dtype)) || !float_type(w_dtype) ||
      !(codes || float_type(y_dtype)))
    return QLORA_ERR_DTYPE;
  if (M == 0) return QLORA_OK;
  if ((residual != nullptr) != (h != nullptr)) return QLORA_ERR_INVALID_ARG;
  if (codes != (scales != nullptr)) return QLORA_ERR_INVALID_ARG;
  if (!x || !y) return QLORA_ERR_INVALID_ARG;
  if (!residual) r_dtype = x_dtype;
  if (!aligned_elem(x, x_dtype) || !aligned_elem(residual, r_dtype) ||
      !aligned_elem(gamma, w_dtype) || !aligned_elem(beta, w_dtype) || !aligned_elem(h, r_dtype) ||
      (!codes && !aligned_elem(y, y_dtype)) || !aligned_elem(scales, QLORA_DTYPE_F32) ||
      !aligned_elem(stats, QLORA_DTYPE_F32))
    return QLORA_ERR_ALIGN;
  const Span in = matrix(x, M, N, ldx, x_dtype), add = matrix(residual, M, N, ldr, r_dtype);
  const Span sum = matrix(h, M, N, ldh, r_dtype);
  const Span out = codes ? span_of(y, M, N, ldy, 1) : matrix(y, M, N, ldy, y_dtype);
  const Span kept = array(stats, 2 * M, QLORA_DTYPE_F32), sc = array(scales, M, QLORA_DTYPE_F32);
  const Span g = array(gamma, N, w_dtype), b = array(beta, N, w_dtype);
  // h may be x (in the same type) or the residual itself.
  const Span in_h = x_dtype == r_dtype ? unless_same(in, sum) : in, add_h = unless_same(add, sum);
  if (any_meet({sum, out, kept, sc}, {in_h, add_h, g, b}) || any_meet({out, kept, sc}, {in, add}))
    return QLORA_ERR_INVALID_ARG;
  return launch_status(launch_add_norm_fwd(
      x, ldx, x_dtype == QLORA_DTYPE_BF16, residual, ldr, r_dtype == QLORA_DTYPE_BF16, M, N,
      norm == QLORA_NORM_LAYER, gamma, beta, w_dtype == QLORA_DTYPE_BF16, eps, h, ldh, y, ldy,
      codes ? 2 : y_dtype == QLORA_DTYPE_BF16 ? 1 : 0, scales, stats,
      static_cast<hipStream_t>(stream)));
}

int qlora_add_norm_bwd(const void* dY, int64_t ldy, int dy_dtype, const void* dH, int64_t lddh,
                       const void* h, int64_t ldh, int h_dtype, int64_t M, int64_t N, int norm,
                       const void* gamma, int w_dtype, float eps, const float* stats, void* dX,
                       int64_t lddx, int dx_dtype, void* dgamma, void* dbeta, int grad_dtype,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!dX || !dH)  // nothing to add, or nothing to add it to: the norm's own gradient
    return qlora_norm_bwd(dY, ldy, dy_dtype, h, ldh, h_dtype, M, N, norm, gamma, w_dtype, eps,
                          stats, dX, lddx, dx_dtype, dgamma, dbeta, grad_dtype, workspace,
                          workspace_bytes, stream);
  if (M < 0 || (norm != QLORA_NORM_LAYER && norm != QLORA_NORM_RMS) || !std::isfinite(eps) ||
      eps < 0.0f)
    return QLORA_ERR_INVALID_ARG;
  if (!norm_shape_ok(M, N) || !stride_ok(M, N, ldy) || !stride_ok(M, N, lddh) ||
      !stride_ok(M, N, ldh) || !stride_ok(M, N, lddx))
    return QLORA_ERR_SHAPE;
  if (!float_type(dy_dtype) || !float_type(h_dtype) || !float_type(w_dtype) ||
      !float_type(dx_dtype) || !float_type(grad_dtype))
    return QLORA_ERR_DTYPE;
  if (M > 0 && (!dY || !h)) return QLORA_ERR_INVALID_ARG;
  if (!aligned_elem(dY, dy_dtype) || !aligned_elem(dH, dx_dtype) || !aligned_elem(h, h_dtype) ||
      !aligned_elem(gamma, w_dtype) || !aligned_elem(stats, QLORA_DTYPE_F32) ||
      !aligned_elem(dX, dx_dtype) || !aligned_elem(dgamma, grad_dtype) ||
      !aligned_elem(dbeta, grad_dtype) || !aligned16(workspace))
    return QLORA_ERR_ALIGN;
  const bool grads = dgamma || dbeta;
  const size_t need = grads ? qlora_norm_bwd_workspace_bytes(M, N) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return QLORA_ERR_WORKSPACE;
  if (M == 0 && !grads) return QLORA_OK;
  const Span dx = matrix(dX, M, N, lddx, dx_dtype), dh = matrix(dH, M, N, lddh, dx_dtype);
  const Span in = matrix(h, M, N, ldh, h_dtype), dy = matrix(dY, M, N, ldy, dy_dtype);
  const Span dg = array(dgamma, N, grad_dtype), db = array(dbeta, N, grad_dtype);
  const Span part = bytes(grads ? workspace : nullptr, need);
  const Span in_dx = h_dtype == dx_dtype ? unless_same(in, dx) : in;
  const Span dy_dx = dy_dtype == dx_dtype ? unless_same(dy, dx) : dy;
  if (any_meet({dx, dg, db, part}, {in_dx, dy_dx, unless_same(dh, dx), array(gamma, N, w_dtype),
                                    array(stats, 2 * M, QLORA_DTYPE_F32)}) ||
      any_meet({dg, db, part}, {in, dy, dh}))
    return QLORA_ERR_INVALID_ARG;
  return launch_status(launch_add_norm_bwd(
      dY, ldy, dy_dtype == QLORA_DTYPE_BF16, dH, lddh, h, ldh, h_dtype == QLORA_DTYPE_BF16, M, N,
      norm == QLORA_NORM_LAYER, gamma, w_dtype == QLORA_DTYPE_BF16, eps, stats, dX, lddx,
      dx_dtype == QLORA_DTYPE_BF16, dgamma, dbeta, grad_dtype == QLORA_DTYPE_BF16,
      static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
