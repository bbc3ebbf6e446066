// The row operators' entry points (token embedding, norm, distillation):
// argument validation, workspace layout and launches. As with the linear
// layer's entry points every check runs on the host before anything is
// enqueued.
#include <cmath>

#include "host.h"
#include "internal.h"
#include "spans.h"

namespace qlora {
namespace {

constexpr int64_t kMaxIds = ((int64_t)1 << 31) - 2;  // ids are held in 32 bits, one value is taken
constexpr int64_t kMaxEmbedWidth = (int64_t)1 << 24;

bool float_type(int d) { return d == QLORA_DTYPE_F32 || d == QLORA_DTYPE_BF16; }
bool index_type(int d) { return d == QLORA_DTYPE_I32 || d == QLORA_DTYPE_I64; }
int64_t elem_bytes(int dtype) { return dtype == QLORA_DTYPE_BF16 ? 2 : dtype == QLORA_DTYPE_I64 ? 8 : 4; }

// The alignment of an element of a QLORA_DTYPE_* type.
bool aligned_elem(const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(elem_bytes(dtype) - 1)) == 0;
}

// What an argument occupies, for the check that no output lies on an input:
// rows of a matrix, or a contiguous array.
Span matrix(const void* p, int64_t rows, int64_t width, int64_t ld, int dtype) {
  return span_of(p, rows, width, ld, elem_bytes(dtype));
}
Span array(const void* p, int64_t count, int dtype) { return span_of(p, count * elem_bytes(dtype)); }
Span bytes(const void* p, size_t n) { return span_of(p, (int64_t)n); }
// An output that may be the input `in` itself, at the same address and stride
// in the same type: no span of its own then.
Span unless_same(const Span& in, const Span& out) { return in.same(out) ? Span{} : in; }

// Rows of `width` elements every `ld`: the last row's end stays countable.
bool stride_ok(int64_t M, int64_t width, int64_t ld) {
  return ld >= width && ld <= kMaxElems / (M > 0 ? M : 1);
}

bool embed_shape_ok(int64_t V, int64_t D) {
  return V >= 1 && V <= kMaxIds && D >= 1 && D <= kMaxEmbedWidth && V <= kMaxElems / D;
}

struct EmbedLayout {
  size_t sorted = 0, part = 0, total = 0;
};

EmbedLayout embed_layout(int64_t M, int64_t D) {
  EmbedLayout L;
  if (M == 0) return L;
  Carve c;
  const size_t tiles = (size_t)((M + embed_tile(M) - 1) / embed_tile(M));
  L.sorted = c.take((4 * (size_t)((M + 63) / 64 * 64) + 1 + tiles) * 4);
  L.part = c.take(tiles * 2 * (size_t)((D + 7) / 8 * 8) * 4);
  L.total = c.off;
  return L;
}

bool norm_shape_ok(int64_t M, int64_t N) {
  return M >= 0 && M <= QLORA_MAX_ROWS && N >= 1 && N <= QLORA_MAX_NORM_WIDTH;
}

size_t norm_bwd_bytes(int64_t M, int64_t N) {
  return M == 0 ? 0 : round_up((size_t)norm_bwd_parts(M, N) * 2 * (size_t)((N + 7) / 8 * 8) * 4);
}

size_t distill_fwd_bytes(int64_t M, int64_t V) {
  return M == 0 ? 0 : round_up((size_t)M * distill_parts(V) * 2 * sizeof(float));
}

// The checks that both directions of the distillation share.
int distill_check(int64_t ldz, int z_dtype, int64_t M, int64_t V, int ids_dtype, int t_dtype, int k,
                  float temperature) {
  if (M < 0 || !(temperature >= 0x1p-20f && temperature <= 0x1p20f)) return QLORA_ERR_INVALID_ARG;
  if (M > QLORA_MAX_ROWS || V < 1 || V > kMaxIds || k < 1 || k > QLORA_MAX_TOP ||
      !stride_ok(M, V, ldz))
    return QLORA_ERR_SHAPE;
  if (!float_type(z_dtype) || !index_type(ids_dtype) || !float_type(t_dtype))
    return QLORA_ERR_DTYPE;
  return QLORA_OK;
}

}  // namespace
}  // namespace qlora

using namespace qlora;

extern "C" {

int qlora_embed_fwd(const void* W, int64_t ldw, int w_dtype, int64_t V, int64_t D,
                    const void* ids, int ids_dtype, int64_t M, float scale, void* out,
                    int64_t ldo, int out_dtype, void* stream) {
  if (M < 0 || !std::isfinite(scale)) return QLORA_ERR_INVALID_ARG;
  if (!embed_shape_ok(V, D) || M > QLORA_MAX_ROWS || !stride_ok(V, D, ldw) ||
      !stride_ok(M, D, ldo))
    return QLORA_ERR_SHAPE;
  if (!float_type(w_dtype) || !index_type(ids_dtype) || !float_type(out_dtype))
    return QLORA_ERR_DTYPE;
  if (M == 0) return QLORA_OK;
  if (!W || !ids || !out) return QLORA_ERR_INVALID_ARG;
  if (!aligned_elem(W, w_dtype) || !aligned_elem(ids, ids_dtype) || !aligned_elem(out, out_dtype))
    return QLORA_ERR_ALIGN;
  if (any_meet({matrix(out, M, D, ldo, out_dtype)},
               {matrix(W, V, D, ldw, w_dtype), array(ids, M, ids_dtype)}))
    return QLORA_ERR_INVALID_ARG;
  return launch_status(launch_embed_fwd(W, ldw, w_dtype == QLORA_DTYPE_BF16, V, D, ids,
                                        ids_dtype == QLORA_DTYPE_I64, M, scale, out, ldo,
                                        out_dtype == QLORA_DTYPE_BF16,
                                        static_cast<hipStream_t>(stream)));
}

size_t qlora_embed_bwd_workspace_bytes(int64_t M, int64_t D) {
  if (M < 0 || M > QLORA_MAX_SORTED || D < 1 || D > kMaxEmbedWidth) return 0;
  return embed_layout(M, D).total;
}

int qlora_embed_bwd(const void* dY, int64_t ldy, int dy_dtype, const void* ids, int ids_dtype,
                    int64_t M, int64_t V, int64_t D, float scale, void* dW, int grad_dtype,
                    int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (M < 0 || !std::isfinite(scale)) return QLORA_ERR_INVALID_ARG;
  if (!embed_shape_ok(V, D) || M > QLORA_MAX_SORTED || !stride_ok(M, D, ldy))
    return QLORA_ERR_SHAPE;
  if (!float_type(dy_dtype) || !index_type(ids_dtype) || !float_type(grad_dtype))
    return QLORA_ERR_DTYPE;
  if (!dW || (M > 0 && (!dY || !ids))) return QLORA_ERR_INVALID_ARG;
  if (!aligned16(dW) || (workspace && !aligned16(workspace)) ||
      (M > 0 && (!aligned_elem(dY, dy_dtype) || !aligned_elem(ids, ids_dtype))))
    return QLORA_ERR_ALIGN;
  const EmbedLayout L = embed_layout(M, D);
  if (M > 0 && (!workspace || workspace_bytes < L.total)) return QLORA_ERR_WORKSPACE;
  if (any_meet({array(dW, V * D, grad_dtype), bytes(workspace, L.total)},
               {matrix(dY, M, D, ldy, dy_dtype), array(ids, M, ids_dtype)}))
    return QLORA_ERR_INVALID_ARG;
  return launch_status(launch_embed_bwd(
      dY, ldy, dy_dtype == QLORA_DTYPE_BF16, ids, ids_dtype == QLORA_DTYPE_I64, M, V, D, scale, dW,
      grad_dtype == QLORA_DTYPE_BF16, accumulate != 0,
      M > 0 ? at<int32_t>(workspace, L.sorted) : nullptr,
      M > 0 ? at<float>(workspace, L.part) : nullptr, static_cast<hipStream_t>(stream)));
}

int qlora_norm_fwd(const void* x, int64_t ldx, int x_dtype, int64_t M, int64_t N, int norm,
                   const void* gamma, const void* beta, int w_dtype, float eps, void* y,
                   int64_t ldy, int y_dtype, float* stats, void* stream) {
  if (M < 0 || (norm != QLORA_NORM_LAYER && norm != QLORA_NORM_RMS) || !std::isfinite(eps) ||
      eps < 0.0f)
    return QLORA_ERR_INVALID_ARG;
  if (!norm_shape_ok(M, N) || !stride_ok(M, N, ldx) || !stride_ok(M, N, ldy))
    return QLORA_ERR_SHAPE;
  if (!float_type(x_dtype) || !float_type(w_dtype) || !float_type(y_dtype)) return QLORA_ERR_DTYPE;
  if (M == 0) return QLORA_OK;
  if (!x || !y) return QLORA_ERR_INVALID_ARG;
  if (!aligned_elem(x, x_dtype) || !aligned_elem(gamma, w_dtype) || !aligned_elem(beta, w_dtype) ||
      !aligned_elem(y, y_dtype) || !aligned_elem(stats, QLORA_DTYPE_F32))
    return QLORA_ERR_ALIGN;
  const Span out = matrix(y, M, N, ldy, y_dtype), in = matrix(x, M, N, ldx, x_dtype);
  const Span kept = array(stats, 2 * M, QLORA_DTYPE_F32);
  if (any_meet({out, kept}, {unless_same(in, out), array(gamma, N, w_dtype), array(beta, N, w_dtype)}) ||
      meet(kept, in))
    return QLORA_ERR_INVALID_ARG;
  return launch_status(launch_norm_fwd(x, ldx, x_dtype == QLORA_DTYPE_BF16, M, N,
                                       norm == QLORA_NORM_LAYER, gamma, beta,
                                       w_dtype == QLORA_DTYPE_BF16, eps, y, ldy,
                                       y_dtype == QLORA_DTYPE_BF16, stats,
                                       static_cast<hipStream_t>(stream)));
}

size_t qlora_norm_bwd_workspace_bytes(int64_t M, int64_t N) {
  return norm_shape_ok(M, N) ? norm_bwd_bytes(M, N) : 0;
}

int qlora_norm_bwd(const void* dY, int64_t ldy, int dy_dtype, const void* x, int64_t ldx,
                   int x_dtype, int64_t M, int64_t N, int norm, const void* gamma, int w_dtype,
                   float eps, const float* stats, void* dX, int64_t lddx, int dx_dtype,
                   void* dgamma, void* dbeta, int grad_dtype, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (M < 0 || (norm != QLORA_NORM_LAYER && norm != QLORA_NORM_RMS) || !std::isfinite(eps) ||
      eps < 0.0f)
    return QLORA_ERR_INVALID_ARG;
  if (!norm_shape_ok(M, N) || !stride_ok(M, N, ldy) || !stride_ok(M, N, ldx) ||
      (dX && !stride_ok(M, N, lddx)))
    return QLORA_ERR_SHAPE;
  if (!float_type(dy_dtype) || !float_type(x_dtype) || !float_type(w_dtype) ||
      !float_type(dx_dtype) || !float_type(grad_dtype))
    return QLORA_ERR_DTYPE;
  if (M > 0 && (!dY || !x)) return QLORA_ERR_INVALID_ARG;
  if (!aligned_elem(dY, dy_dtype) || !aligned_elem(x, x_dtype) || !aligned_elem(gamma, w_dtype) ||
      !aligned_elem(stats, QLORA_DTYPE_F32) || !aligned_elem(dX, dx_dtype) ||
      !aligned_elem(dgamma, grad_dtype) || !aligned_elem(dbeta, grad_dtype) ||
      !aligned16(workspace))
    return QLORA_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool gbf = grad_dtype == QLORA_DTYPE_BF16, grads = dgamma || dbeta;
  if (grads && M > 0 && (!workspace || workspace_bytes < norm_bwd_bytes(M, N)))
    return QLORA_ERR_WORKSPACE;
  if (!dX && !grads) return QLORA_OK;
  if (M == 0 && !grads) return QLORA_OK;
  const Span dx = matrix(dX, M, N, lddx, dx_dtype);
  const Span in = matrix(x, M, N, ldx, x_dtype), dy = matrix(dY, M, N, ldy, dy_dtype);
  const Span dg = array(dgamma, N, grad_dtype), db = array(dbeta, N, grad_dtype);
  const Span part = bytes(grads ? workspace : nullptr, norm_bwd_bytes(M, N));
  if (any_meet({dx, dg, db, part},
               {unless_same(in, dx), unless_same(dy, dx), array(gamma, N, w_dtype),
                array(stats, 2 * M, QLORA_DTYPE_F32)}) ||
      any_meet({dg, db, part}, {in, dy}))
    return QLORA_ERR_INVALID_ARG;
  return launch_status(launch_norm_bwd(dY, ldy, dy_dtype == QLORA_DTYPE_BF16, x, ldx,
                                       x_dtype == QLORA_DTYPE_BF16, M, N, norm == QLORA_NORM_LAYER,
                                       gamma, w_dtype == QLORA_DTYPE_BF16, eps, stats, dX, lddx,
                                       dx_dtype == QLORA_DTYPE_BF16, dgamma, dbeta, gbf,
                                       static_cast<float*>(workspace), st));
}

size_t qlora_distill_fwd_workspace_bytes(int64_t M, int64_t V) {
  if (M < 0 || M > QLORA_MAX_ROWS || V < 1 || V > kMaxIds) return 0;
  return distill_fwd_bytes(M, V);
}

int qlora_distill_fwd(const void* logits, int64_t ldz, int z_dtype, int64_t M, int64_t V,
                      const void* top_ids, int ids_dtype, const void* top_logits, int t_dtype,
                      int k, float temperature, float* loss, float* stats, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (const int st = distill_check(ldz, z_dtype, M, V, ids_dtype, t_dtype, k, temperature))
    return st;
  if (M == 0) return QLORA_OK;
  if (!logits || !top_ids || !top_logits || !loss) return QLORA_ERR_INVALID_ARG;
  if (!aligned_elem(logits, z_dtype) || !aligned_elem(top_ids, ids_dtype) ||
      !aligned_elem(top_logits, t_dtype) || !aligned_elem(loss, QLORA_DTYPE_F32) ||
      !aligned_elem(stats, QLORA_DTYPE_F32) || !aligned16(workspace))
    return QLORA_ERR_ALIGN;
  const size_t need = distill_fwd_bytes(M, V);
  if (need > 0 && (!workspace || workspace_bytes < need)) return QLORA_ERR_WORKSPACE;
  if (any_meet({array(loss, M, QLORA_DTYPE_F32), array(stats, 2 * M, QLORA_DTYPE_F32),
                bytes(workspace, need)},
               {matrix(logits, M, V, ldz, z_dtype), array(top_ids, M * k, ids_dtype),
                array(top_logits, M * k, t_dtype)}))
    return QLORA_ERR_INVALID_ARG;
  return launch_status(launch_distill_fwd(
      logits, ldz, z_dtype == QLORA_DTYPE_BF16, M, V, top_ids, ids_dtype == QLORA_DTYPE_I64,
      top_logits, t_dtype == QLORA_DTYPE_BF16, k, temperature, loss, stats,
      static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

int qlora_distill_bwd(const void* logits, int64_t ldz, int z_dtype, int64_t M, int64_t V,
                      const void* top_ids, int ids_dtype, const void* top_logits, int t_dtype,
                      int k, float temperature, const float* stats, const float* dloss,
                      void* dlogits, int64_t ldg, int grad_dtype, void* stream) {
  if (const int st = distill_check(ldz, z_dtype, M, V, ids_dtype, t_dtype, k, temperature))
    return st;
  if (!stride_ok(M, V, ldg)) return QLORA_ERR_SHAPE;
  if (!float_type(grad_dtype)) return QLORA_ERR_DTYPE;
  if (M == 0) return QLORA_OK;
  if (!logits || !top_ids || !top_logits || !stats || !dloss || !dlogits)
    return QLORA_ERR_INVALID_ARG;
  if (!aligned_elem(logits, z_dtype) || !aligned_elem(top_ids, ids_dtype) ||
      !aligned_elem(top_logits, t_dtype) || !aligned_elem(stats, QLORA_DTYPE_F32) ||
      !aligned_elem(dloss, QLORA_DTYPE_F32) || !aligned_elem(dlogits, grad_dtype))
    return QLORA_ERR_ALIGN;
  if (any_meet({matrix(dlogits, M, V, ldg, grad_dtype)},
               {matrix(logits, M, V, ldz, z_dtype), array(top_ids, M * k, ids_dtype),
                array(top_logits, M * k, t_dtype), array(stats, 2 * M, QLORA_DTYPE_F32),
                array(dloss, M, QLORA_DTYPE_F32)}))
    return QLORA_ERR_INVALID_ARG;
  return launch_status(launch_distill_bwd(
      logits, ldz, z_dtype == QLORA_DTYPE_BF16, M, V, top_ids, ids_dtype == QLORA_DTYPE_I64,
      top_logits, t_dtype == QLORA_DTYPE_BF16, k, temperature, stats, dloss, dlogits, ldg,
      grad_dtype == QLORA_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
