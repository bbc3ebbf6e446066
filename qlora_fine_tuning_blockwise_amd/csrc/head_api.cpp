// Entry points of the vocabulary head's loss: argument validation, workspace
// layout, the cut into pieces of the vocabulary, and launches.
#include <cmath>

#include "head.h"
#include "internal.h"
#include "row_args.h"

namespace qlora {
namespace {

constexpr int64_t kMaxVocab = ((int64_t)1 << 31) - 2;

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Whether the tile kernels read W from where it lies: rows of whole steps, 16
// bytes aligned, a tile's rows within 32-bit offsets.
bool in_place(const void* W, int64_t ldw, int64_t K) {
  return K % kStep == 0 && ldw % 8 == 0 && ldw <= (1 << 20) && aligned16(W);
}

bool shape_ok(int64_t M, int64_t V, int64_t K) {
  return M <= QLORA_MAX_SORTED && V >= 1 && V <= kMaxVocab && K >= 1 &&
         K <= QLORA_MAX_HEAD_WIDTH && V <= kMaxElems / K;
}

// Entries of the vocabulary in a copy of W's rows: 128 MB of them at most, all
// copies alike.
int64_t copy_rows(int64_t V, int64_t Kp) {
  const int64_t most = ((int64_t)1 << 26) / Kp, pieces = (V + most - 1) / most;
  return up((V + pieces - 1) / pieces, kTile);
}

struct Layout {
  int64_t rows_pad = 0, Kp = 0, piece = 0;
  size_t map = 0, inv = 0, count = 0, cols = 0, xs = 0, at_label = 0, part = 0, copy = 0;
  size_t P = 0, Q = 0, xr = 0, acc = 0, rest = 0, total = 0;
};

void rows_layout(Layout& L, Carve& c, int64_t M, int64_t K) {
  L.rows_pad = up(M, kTile);
  L.Kp = up(K, kStep);
  L.map = c.take((size_t)M * 4);
  L.inv = c.take((size_t)M * 4);
  L.count = c.take(8);
  L.cols = c.take((size_t)L.rows_pad * sizeof(HeadColumn));
  L.xs = c.take((size_t)L.rows_pad * L.Kp * 2);
}

constexpr int64_t kFewEntries = (int64_t)1 << 29;  // of the vocabulary in a launch of few rows
int64_t few_parts(int64_t V, int64_t M) { return (V + few_entries(V, M) - 1) / few_entries(V, M); }

Layout fwd_layout(int64_t M, int64_t V, int64_t K, bool copy) {
  Layout L;
  if (M == 0) return L;
  Carve c;
  if (M <= kFewRows) {  // one pass over W where it lies
    L.at_label = c.take((size_t)M * 4);
    L.part = c.take((size_t)few_parts(V, M) * M * sizeof(float2));
    L.total = c.off;
    return L;
  }
  rows_layout(L, c, M, K);
  L.at_label = c.take((size_t)L.rows_pad * 4);
  L.part = c.take((size_t)(up(V, kTile) / kTile) * L.rows_pad * sizeof(float2));
  L.piece = copy ? copy_rows(V, L.Kp) : 0;
  if (copy) L.copy = c.take((size_t)L.piece * L.Kp * 2);
  L.total = c.off;
  return L;
}

// Entries of the vocabulary in a piece of the backward: 2^26 probabilities (128
// MB of bf16), 2048 entries at least, all pieces alike; where W is copied 32768 of
// its rows at most.
int64_t piece_of(int64_t M, int64_t V, bool copy) {
  int64_t n = ((int64_t)1 << 26) / up(M, kTile) / kTile * kTile;
  n = n < 2048 ? 2048 : n > 32768 && copy ? 32768 : n;
  const int64_t pieces = (V + n - 1) / n;
  return up((V + pieces - 1) / pieces, kTile);
}

// bf16 numbers that a probability or a logit's gradient is split into.
int terms(int dtype) { return dtype == QLORA_DTYPE_F32 ? 3 : 1; }

// Whether the backward's tile kernels read W, for logits or for dX.
bool tiles_read_w(int64_t M, int64_t K, bool dx) { return M > kFewRows || (dx && !few_dx(M, K)); }

// dx, dw: the outputs' types, negative for one that is not wanted.
Layout bwd_layout(int64_t M, int64_t V, int64_t K, bool copy, int dx, int dw) {
  Layout L;
  if (M == 0) return L;
  Carve c;
  rows_layout(L, c, M, K);
  L.piece = piece_of(M, V, copy);
  if (copy && tiles_read_w(M, K, dx >= 0)) L.copy = c.take((size_t)L.piece * L.Kp * 2);
  if (dx >= 0 && few_dx(M, K)) {
    L.acc = c.take((size_t)few_dx_sums(M, V, K) * 4);
  } else if (dx >= 0) {
    L.P = c.take((size_t)L.rows_pad * L.piece * terms(dx) * 2);
    L.acc = c.take((size_t)head_sums(M, K) * kTile * kTile * 4);
  }
  if (dx >= 0) L.rest = c.take((size_t)M * 4);
  if (dw >= 0) {
    L.Q = c.take((size_t)L.rows_pad * L.piece * terms(dw) * 2);
    L.xr = c.take((size_t)L.rows_pad * L.Kp * 2);
  }
  L.total = c.off;
  return L;
}

}  // namespace
}  // namespace qlora

using namespace qlora;

extern "C" {

size_t qlora_head_loss_fwd_workspace_bytes(int64_t M, int64_t V, int64_t K, int w_copy) {
  return M < 0 || !shape_ok(M, V, K) ? 0 : fwd_layout(M, V, K, w_copy != 0).total;
}

int qlora_head_loss_fwd(const uint16_t* x, int64_t ldx, const uint16_t* W, int64_t ldw, int64_t M,
                        int64_t V, int64_t K, const void* labels, int ids_dtype, float scale,
                        float* loss, float* stats, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (M < 0 || !std::isfinite(scale)) return QLORA_ERR_INVALID_ARG;
  if (!shape_ok(M, V, K) || !stride_ok(M, K, ldx) || !stride_ok(V, K, ldw)) return QLORA_ERR_SHAPE;
  if (!index_type(ids_dtype)) return QLORA_ERR_DTYPE;
  if (M == 0) return QLORA_OK;
  if (!x || !W || !labels || !loss) return QLORA_ERR_INVALID_ARG;
  if (!aligned_elem(x, QLORA_DTYPE_BF16) || !aligned_elem(W, QLORA_DTYPE_BF16) ||
      !aligned_elem(labels, ids_dtype) || !aligned_elem(loss, QLORA_DTYPE_F32) ||
      !aligned_elem(stats, QLORA_DTYPE_F32) || !aligned16(workspace))
    return QLORA_ERR_ALIGN;
  const bool copy = !in_place(W, ldw, K);
  const Layout L = fwd_layout(M, V, K, copy);
  if (!workspace || workspace_bytes < L.total) return QLORA_ERR_WORKSPACE;
  if (any_meet({array(loss, M, QLORA_DTYPE_F32), array(stats, 2 * M, QLORA_DTYPE_F32),
                bytes(workspace, L.total)},
               {matrix(x, M, K, ldx, QLORA_DTYPE_BF16), matrix(W, V, K, ldw, QLORA_DTYPE_BF16),
                array(labels, M, ids_dtype)}))
    return QLORA_ERR_INVALID_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (M <= kFewRows) {
    HeadFew f{};
    f.ldw = ldw;
    f.x = x;
    f.ldx = ldx;
    f.M = M;
    f.K = K;
    f.V = V;
    f.entries = few_entries(V, M);
    f.scale = scale;
    f.labels = labels;
    f.ids64 = ids_dtype == QLORA_DTYPE_I64;
    f.part = at<float2>(workspace, L.part);
    f.parts = few_parts(V, M);
    f.at_label = at<float>(workspace, L.at_label);
    // Four threads an entry: fewer than 2^32 of them a launch.
    hipError_t e = hipSuccess;
    for (int64_t v0 = 0; v0 < V && e == hipSuccess; v0 += kFewEntries) {
      f.W = W + v0 * ldw;
      f.v0 = v0;
      f.vocab = V - v0 < kFewEntries ? V - v0 : kFewEntries;
      e = launch_head_few_stats(f, st);
    }
    if (e == hipSuccess)
      e = launch_head_few_loss(f.part, f.parts, f.at_label, labels, f.ids64, M, V, loss, stats, st);
    return launch_status(e);
  }
  HeadRows r{};
  r.labels = labels;
  r.ids64 = ids_dtype == QLORA_DTYPE_I64;
  r.scale = scale;
  r.M = M;
  r.V = V;
  r.map = at<int32_t>(workspace, L.map);
  r.inv = at<int32_t>(workspace, L.inv);
  r.count = at<int32_t>(workspace, L.count);
  r.cols = at<HeadColumn>(workspace, L.cols);
  uint16_t* xs = at<uint16_t>(workspace, L.xs);
  hipError_t e = launch_head_rows(r, st);
  if (e == hipSuccess) e = launch_head_pack_rows(x, ldx, r.map, r.count, M, K, xs, st);
  HeadTiles t{};
  t.b = xs;
  t.b_steps = t.steps = L.Kp / kStep;
  t.count = r.count;
  t.rows_most = M;
  t.K = K;
  t.scale = scale;
  t.cols = r.cols;
  t.part = at<float2>(workspace, L.part);
  t.rows_pad = L.rows_pad;
  t.at_label = at<float>(workspace, L.at_label);
  // Pieces of W that are copied, or all of it; grids stay below 2^22 workgroups.
  int64_t step = ((int64_t)1 << 22) / (L.rows_pad / kTile) * kTile;
  if (copy && L.piece < step) step = L.piece;
  for (int64_t v0 = 0; v0 < V && e == hipSuccess; v0 += step) {
    t.v0 = v0;
    t.vocab = V - v0 < step ? V - v0 : step;
    t.a = W + v0 * ldw;
    t.lda = ldw;
    if (copy) {
      uint16_t* Wc = at<uint16_t>(workspace, L.copy);
      e = launch_head_copy(t.a, ldw, nullptr, r.count, t.vocab, K, L.Kp, Wc, st);
      t.a = Wc;
      t.lda = L.Kp;
    }
    if (e == hipSuccess) e = launch_head_stats(t, st);
  }
  if (e == hipSuccess)
    e = launch_head_loss(t.part, up(V, kTile) / kTile, L.rows_pad, t.at_label, r.inv, M, loss, stats,
                         st);
  return launch_status(e);
}

size_t qlora_head_loss_bwd_workspace_bytes(int64_t M, int64_t V, int64_t K, int w_copy,
                                           int dx_dtype, int grad_dtype) {
  if (M < 0 || !shape_ok(M, V, K)) return 0;
  return bwd_layout(M, V, K, w_copy != 0, dx_dtype, grad_dtype).total;
}

int qlora_head_loss_bwd(const uint16_t* x, int64_t ldx, const uint16_t* W, int64_t ldw, int64_t M,
                        int64_t V, int64_t K, const void* labels, int ids_dtype, float scale,
                        const float* stats, const float* dloss, void* dX, int64_t lddx,
                        int dx_dtype, void* dW, int grad_dtype, int accumulate, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (M < 0 || !std::isfinite(scale)) return QLORA_ERR_INVALID_ARG;
  if (!shape_ok(M, V, K) || !stride_ok(M, K, ldx) || !stride_ok(V, K, ldw) ||
      (dX && !stride_ok(M, K, lddx)))
    return QLORA_ERR_SHAPE;
  if (!index_type(ids_dtype) || (dX && !float_type(dx_dtype)) || (dW && !float_type(grad_dtype)))
    return QLORA_ERR_DTYPE;
  if (M > 0 && (!x || !W || !labels || !stats || !dloss)) return QLORA_ERR_INVALID_ARG;
  if (!aligned_elem(x, QLORA_DTYPE_BF16) || !aligned_elem(W, QLORA_DTYPE_BF16) ||
      !aligned_elem(labels, ids_dtype) || !aligned_elem(stats, QLORA_DTYPE_F32) ||
      !aligned_elem(dloss, QLORA_DTYPE_F32) || (dX && !aligned_elem(dX, dx_dtype)) ||
      !aligned16(dW) || !aligned16(workspace))
    return QLORA_ERR_ALIGN;
  if (!dX && !dW) return QLORA_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (M == 0) {  // no rows: the gradient of W is zero
    if (!dW || accumulate) return QLORA_OK;
    if (W && meet(array(dW, V * K, grad_dtype), matrix(W, V, K, ldw, QLORA_DTYPE_BF16)))
      return QLORA_ERR_INVALID_ARG;
    return launch_status(launch_head_zero(dW, V * K * elem_bytes(grad_dtype), st));
  }
  const bool few = M <= kFewRows, once = dX && few_dx(M, K), tiles = dX && !once;
  const bool unlike = !in_place(W, ldw, K), copy = unlike && tiles_read_w(M, K, dX != nullptr);
  const Layout L = bwd_layout(M, V, K, unlike, dX ? dx_dtype : -1, dW ? grad_dtype : -1);
  if (!workspace || workspace_bytes < L.total) return QLORA_ERR_WORKSPACE;
  if (any_meet({dX ? matrix(dX, M, K, lddx, dx_dtype) : Span{},
                dW ? array(dW, V * K, grad_dtype) : Span{}, bytes(workspace, L.total)},
               {matrix(x, M, K, ldx, QLORA_DTYPE_BF16), matrix(W, V, K, ldw, QLORA_DTYPE_BF16),
                array(labels, M, ids_dtype), array(stats, 2 * M, QLORA_DTYPE_F32),
                array(dloss, M, QLORA_DTYPE_F32)}))
    return QLORA_ERR_INVALID_ARG;
  HeadRows r{};
  r.labels = labels;
  r.ids64 = ids_dtype == QLORA_DTYPE_I64;
  r.dloss = dloss;
  r.stats = stats;
  r.scale = scale;
  r.M = M;
  r.V = V;
  r.K = K;
  // The first piece's pairs of steps decide the splits, so that every piece adds to
  // the same sums.
  r.pairs = tiles ? (int)(up(V < L.piece ? V : L.piece, 2 * kStep) / (2 * kStep) * terms(dx_dtype)) : 0;
  r.map = at<int32_t>(workspace, L.map);
  r.inv = at<int32_t>(workspace, L.inv);
  r.count = at<int32_t>(workspace, L.count);
  r.cols = at<HeadColumn>(workspace, L.cols);
  uint16_t* xs = at<uint16_t>(workspace, L.xs);
  uint16_t* xr = at<uint16_t>(workspace, L.xr);
  hipError_t e = launch_head_rows(r, st);
  if (e == hipSuccess && !few) e = launch_head_pack_rows(x, ldx, r.map, r.count, M, K, xs, st);
  if (e == hipSuccess && once) {
    HeadFewDx f{};
    f.W = W;
    f.ldw = ldw;
    f.x = x;
    f.ldx = ldx;
    f.M = M;
    f.V = V;
    f.K = K;
    f.scale = scale;
    f.map = r.map;
    f.inv = r.inv;
    f.count = r.count;
    f.cols = r.cols;
    f.part = at<float>(workspace, L.acc);
    f.rest = at<float>(workspace, L.rest);
    f.groups = few_dx_groups(V);
    f.dX = dX;
    f.lddx = lddx;
    e = launch_head_few_dx(f, dx_dtype == QLORA_DTYPE_BF16, st);
  }
  if (once && !dW) return launch_status(e);
  if (e == hipSuccess && dW)
    e = launch_head_copy(x, ldx, r.map, r.count, M, K, L.Kp, xr, st);
  HeadTiles t{};
  t.count = r.count;
  t.rows_most = M;
  t.K = K;
  t.scale = scale;
  t.cols = r.cols;
  t.rows_pad = L.rows_pad;
  t.steps = L.Kp / kStep;
  t.p_terms = tiles ? terms(dx_dtype) : 0;
  t.q_terms = dW ? terms(grad_dtype) : 0;
  t.ldp = L.piece * t.p_terms;
  t.ldq = L.piece;
  t.q_plane = L.rows_pad * L.piece;
  t.acc = at<float>(workspace, L.acc);
  t.rest = tiles ? at<float>(workspace, L.rest) : nullptr;
  t.dW = dW;
  t.dw_bf16 = grad_dtype == QLORA_DTYPE_BF16;
  t.accumulate = accumulate != 0;
  for (int64_t v0 = 0; v0 < V && e == hipSuccess; v0 += L.piece) {
    t.v0 = v0;
    t.vocab = V - v0 < L.piece ? V - v0 : L.piece;
    const uint16_t* Wv = W + v0 * ldw;  // the piece's rows, as the kernels read them
    int64_t ldv = ldw;
    if (copy) {
      uint16_t* Wc = at<uint16_t>(workspace, L.copy);
      e = launch_head_copy(Wv, ldw, nullptr, r.count, t.vocab, K, L.Kp, Wc, st);
      Wv = Wc;
      ldv = L.Kp;
    }
    t.a = Wv;
    t.lda = ldv;
    t.b = xs;
    t.b_steps = t.steps;
    t.P = tiles ? at<uint16_t>(workspace, L.P) : nullptr;
    t.Q = dW ? at<uint16_t>(workspace, L.Q) : nullptr;
    if (e == hipSuccess && few) {
      HeadFew f{};
      f.W = W + v0 * ldw;
      f.ldw = ldw;
      f.x = x;
      f.ldx = ldx;
      f.M = M;
      f.K = K;
      f.V = V;
      f.v0 = v0;
      f.vocab = t.vocab;
      f.entries = few_entries(t.vocab, M);
      f.scale = scale;
      f.map = r.map;
      f.count = r.count;
      f.cols = r.cols;
      f.rest = t.rest;
      f.P = t.P;
      f.ldp = t.ldp;
      f.p_plane = up(t.vocab, 2 * kStep);
      f.p_terms = t.p_terms;
      f.Q = t.Q;
      f.ldq = t.ldq;
      f.q_plane = t.q_plane;
      f.q_terms = t.q_terms;
      e = launch_head_few_probs(f, st);
    } else if (e == hipSuccess) {
      e = launch_head_probs(t, st);
    }
    if (e == hipSuccess && tiles) {
      t.a = t.P;
      t.lda = t.ldp;
      t.b = Wv;
      t.ldb = ldv;
      t.b_width = copy ? ldv : K;
      t.vocab_left = copy ? t.vocab : V - v0;
      t.add = v0 > 0;
      e = launch_head_dx(t, st);
    }
    if (e == hipSuccess && dW) {
      t.a = xr;
      t.lda = L.Kp;
      t.b = t.Q;
      t.ldb = t.b_width = t.ldq;
      e = launch_head_dw(t, st);
    }
  }
  if (e == hipSuccess && tiles) {
    const HeadDx d{t.acc, t.rest, r.map, r.inv, r.count, r.cols, W, ldw, M, K, dX, lddx};
    e = launch_head_dx_finish(d, dx_dtype == QLORA_DTYPE_BF16, st);
  }
  return launch_status(e);
}

}  // extern "C"
