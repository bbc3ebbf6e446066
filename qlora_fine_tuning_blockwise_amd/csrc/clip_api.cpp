// Entry points of the gradients' global norm and its clipping: validation, the
// cut into chunks and the launches, and the optimizer step that takes the
// factor from the device.
#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "host.h"
#include "internal.h"
#include "spans.h"
#include "spans_table.h"

namespace qlora {
namespace {

int64_t tensor_elem(const qlora_tensor& t) { return t.dtype == QLORA_DTYPE_BF16 ? 2 : 4; }

int tensors_check(const qlora_tensor* t, int64_t count, int64_t* total) {
  *total = 0;
  if (count < 0 || (count > 0 && !t)) return QLORA_ERR_INVALID_ARG;
  if (count > QLORA_MAX_TENSORS) return QLORA_ERR_SHAPE;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n < 0 || t[i].reserved != 0) return QLORA_ERR_INVALID_ARG;
    if (t[i].n > kMaxElems - *total) return QLORA_ERR_SHAPE;
    if (t[i].dtype != QLORA_DTYPE_F32 && t[i].dtype != QLORA_DTYPE_BF16) return QLORA_ERR_DTYPE;
    if (t[i].n > 0 && !t[i].data) return QLORA_ERR_INVALID_ARG;
    if (t[i].n > 0 && (reinterpret_cast<uintptr_t>(t[i].data) & (uintptr_t)(tensor_elem(t[i]) - 1)))
      return QLORA_ERR_ALIGN;
    *total += t[i].n;
  }
  return QLORA_OK;
}

int64_t tensor_bytes(const qlora_tensor& t) { return t.n * tensor_elem(t); }

// Bytes of a chunk: 32 KB, and more where that leaves over 2^14 chunks, so that
// the sums stay few (2^14 of them are 128 KB).
int64_t chunk_bytes(const qlora_tensor* t, int64_t count) {
  int64_t all = 0, c = 32768;
  for (int64_t i = 0; i < count; ++i) all += tensor_bytes(t[i]);
  while (all / c > 16384) c *= 2;
  return c;
}

int64_t chunks_of(const qlora_tensor& t, int64_t chunk) { return (tensor_bytes(t) + chunk - 1) / chunk; }
int64_t chunks_of(const qlora_tensor* t, int64_t count, int64_t chunk) {
  int64_t c = 0;
  for (int64_t i = 0; i < count; ++i) c += chunks_of(t[i], chunk);
  return c;
}

size_t norm_bytes(const qlora_tensor* t, int64_t count) {
  return round_up((size_t)chunks_of(t, count, chunk_bytes(t, count)) * sizeof(double));
}

// Calls launch(table, chunks, chunks before) for the tensors, kSpans at a time.
template <typename F>
hipError_t in_launches(const qlora_tensor* in, const qlora_tensor* out, int64_t count,
                       int64_t chunk, F launch) {
  SpanTable t;
  int64_t before = 0;
  for (int64_t i = 0; i < count;) {
    t.count = 0;
    t.chunk = chunk;
    for (uint64_t& b : t.bf16_bits) b = 0;
    uint32_t chunks = 0;
    for (; i < count && t.count < kSpans; ++i) {
      if (in[i].n == 0) continue;
      const int k = t.count++;
      t.in[k] = in[i].data;
      t.out[k] = out ? out[i].data : nullptr;
      t.n[k] = in[i].n;
      if (in[i].dtype == QLORA_DTYPE_BF16) t.bf16_bits[k >> 6] |= (uint64_t)1 << (k & 63);
      chunks += (uint32_t)chunks_of(in[i], chunk);
      t.end[k] = chunks;
    }
    if (t.count == 0) break;
    for (int k = t.count; k < kSpans; ++k) {
      t.in[k] = t.out[k] = nullptr;
      t.n[k] = 0;
      t.end[k] = chunks;
    }
    const hipError_t e = launch(t, chunks, before);
    if (e != hipSuccess) return e;
    before += chunks;
  }
  return hipSuccess;
}

Span tensor_span(const qlora_tensor& t) { return span_of(t.data, tensor_bytes(t)); }

struct Run {
  uintptr_t first, end;
  bool operator<(const Run& o) const { return first < o.first; }
};

// Runs in the order of their addresses, as the tensors of one buffer come.
void in_order(Run* r, int64_t n) {
  if (!std::is_sorted(r, r + n)) std::sort(r, r + n);
}

// Whether a written run shares memory with another written one, or with one that
// is read (of these some may share with each other).
bool runs_meet(Run* written, int64_t n, Run* read, int64_t m) {
  in_order(written, n);
  in_order(read, m);
  for (int64_t i = 0; i + 1 < n; ++i)
    if (written[i + 1].first < written[i].end) return true;
  // Written runs lie apart now, so their ends are in order too: each read run
  // against the first one that ends behind its start.
  int64_t i = 0;
  for (int64_t j = 0; j < m; ++j) {
    while (i < n && written[i].end <= read[j].first) ++i;
    if (i < n && written[i].first < read[j].end) return true;
  }
  return false;
}

// The address at which kernels reach an array: device memory itself, or pinned
// host memory by its mapping (the paged optimizer state). NULL for pageable memory.
void* reached(void* p) {
  hipPointerAttribute_t a{};
  if (hipPointerGetAttributes(&a, p) != hipSuccess) {
    (void)hipGetLastError();  // the lookup's failure is not a launch's
    return nullptr;
  }
  if (a.type == hipMemoryTypeDevice || a.type == hipMemoryTypeManaged || a.isManaged) return p;
  if (a.type == hipMemoryTypeHost && a.devicePointer && a.hostPointer)
    return static_cast<char*>(a.devicePointer) +
           (static_cast<char*>(p) - static_cast<char*>(a.hostPointer));
  return nullptr;
}

}  // namespace
}  // namespace qlora

using namespace qlora;

extern "C" {

size_t qlora_tensor_table_bytes(const qlora_tensor* tensors, int64_t count) {
  int64_t total;
  if (tensors_check(tensors, count, &total) != QLORA_OK) return 0;
  return (size_t)chunks_of(tensors, count, chunk_bytes(tensors, count)) * sizeof(ChunkEntry);
}

int qlora_tensor_table(const qlora_tensor* tensors, int64_t count, void* table,
                       size_t table_bytes) {
  int64_t total;
  if (const int st = tensors_check(tensors, count, &total)) return st;
  const int64_t chunk = chunk_bytes(tensors, count);
  const int64_t chunks = chunks_of(tensors, count, chunk);
  if (chunks == 0) return QLORA_OK;
  if (!table) return QLORA_ERR_INVALID_ARG;
  if (!aligned16(table)) return QLORA_ERR_ALIGN;
  if (table_bytes < (size_t)chunks * sizeof(ChunkEntry)) return QLORA_ERR_WORKSPACE;
  ChunkEntry* e = static_cast<ChunkEntry*>(table);
  for (int64_t i = 0; i < count; ++i) {
    const int64_t size = tensor_elem(tensors[i]), bytes = tensor_bytes(tensors[i]);
    for (int64_t at = 0; at < bytes; at += chunk)
      *e++ = ChunkEntry{(uint64_t)reinterpret_cast<uintptr_t>(tensors[i].data) + (uint64_t)at,
                        (uint32_t)((bytes - at < chunk ? bytes - at : chunk) / size),
                        (uint32_t)(tensors[i].dtype == QLORA_DTYPE_BF16)};
  }
  return QLORA_OK;
}

size_t qlora_grad_norm_workspace_bytes(const qlora_tensor* grads, int64_t count) {
  int64_t total;
  return tensors_check(grads, count, &total) == QLORA_OK ? norm_bytes(grads, count) : 0;
}

int qlora_grad_norm(const qlora_tensor* grads, int64_t count, const void* table, float max_norm,
                    float* result, void* workspace, size_t workspace_bytes, void* stream) {
  if (!(max_norm >= 0.0f)) return QLORA_ERR_INVALID_ARG;
  int64_t total;
  if (const int st = tensors_check(grads, count, &total)) return st;
  if (!result) return QLORA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(result) & 3) || !aligned16(workspace) || !aligned16(table))
    return QLORA_ERR_ALIGN;
  const int64_t chunk = chunk_bytes(grads, count), chunks = chunks_of(grads, count, chunk);
  const size_t need = round_up((size_t)chunks * sizeof(double));
  if (need > 0 && (!workspace || workspace_bytes < need)) return QLORA_ERR_WORKSPACE;
  const Span out = span_of(result, 8), ws = span_of(workspace, (int64_t)need);
  const Span entries = span_of(table, chunks * (int64_t)sizeof(ChunkEntry));
  if (meet(out, ws) || meet(out, entries) || meet(ws, entries)) return QLORA_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i)
    if (meet(out, tensor_span(grads[i])) || meet(ws, tensor_span(grads[i])))
      return QLORA_ERR_INVALID_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  hipError_t e = hipSuccess;
  if (table && chunks > 0)
    e = launch_grad_norm_table(static_cast<const ChunkEntry*>(table), (uint32_t)chunks, part, st);
  else
    e = in_launches(grads, nullptr, count, chunk,
                    [&](const SpanTable& t, uint32_t n, int64_t before) {
                      return launch_grad_norm(t, n, part + before, st);
                    });
  if (e == hipSuccess) e = launch_grad_norm_join(part, chunks, max_norm, result, st);
  return launch_status(e);
}

int qlora_grad_scale(const qlora_tensor* grads, const qlora_tensor* out, int64_t count,
                     const void* table, const void* out_table, const float* factor,
                     void* stream) {
  if (!out) out = grads, out_table = table;
  int64_t total, same;
  if (const int st = tensors_check(grads, count, &total)) return st;
  if (out != grads) {
    if (const int st = tensors_check(out, count, &same)) return st;
    for (int64_t i = 0; i < count; ++i) {
      if (out[i].n != grads[i].n) return QLORA_ERR_SHAPE;
      if (out[i].dtype != grads[i].dtype) return QLORA_ERR_DTYPE;
    }
  }
  if (!factor) return QLORA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(factor) & 3) || !aligned16(table) || !aligned16(out_table))
    return QLORA_ERR_ALIGN;
  if (total == 0) return QLORA_OK;
  const int64_t chunk = chunk_bytes(grads, count), chunks = chunks_of(grads, count, chunk);
  Run* written = static_cast<Run*>(std::malloc((size_t)(2 * count + 3) * sizeof(Run)));
  if (!written) return QLORA_ERR_INTERNAL;
  Run* const read = written + count;
  int64_t n = 0, m = 0;
  const auto add = [](Run* to, int64_t& k, const Span& s) {
    if (!s.empty()) to[k++] = Run{s.p, s.end()};
  };
  for (int64_t i = 0; i < count; ++i) {
    add(written, n, tensor_span(out[i]));
    if (grads[i].data != out[i].data) add(read, m, tensor_span(grads[i]));
  }
  add(read, m, span_of(factor, 4));
  add(read, m, span_of(table, chunks * (int64_t)sizeof(ChunkEntry)));
  add(read, m, span_of(out_table, chunks * (int64_t)sizeof(ChunkEntry)));
  const bool shared = runs_meet(written, n, read, m);
  std::free(written);
  if (shared) return QLORA_ERR_INVALID_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (table && out_table)
    return launch_status(launch_grad_scale_table(static_cast<const ChunkEntry*>(table),
                                                 static_cast<const ChunkEntry*>(out_table),
                                                 (uint32_t)chunks, factor, st));
  return launch_status(in_launches(grads, out, count, chunk,
                                   [&](const SpanTable& t, uint32_t k, int64_t) {
                                     return launch_grad_scale(t, k, factor, st);
                                   }));
}

int qlora_adamw_step_scaled(float* param, const void* grad, int grad_dtype, const float* factor,
                            float* exp_avg, float* exp_avg_sq, uint16_t* param_bf16, int64_t n,
                            double lr, double beta1, double beta2, double eps, double weight_decay,
                            int64_t step, void* stream) {
  if (n < 0 || step < 1) return QLORA_ERR_INVALID_ARG;
  if (grad_dtype != QLORA_DTYPE_F32 && grad_dtype != QLORA_DTYPE_BF16) return QLORA_ERR_DTYPE;
  if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0)) return QLORA_ERR_INVALID_ARG;
  if (!std::isfinite(lr) || !std::isfinite(eps) || !std::isfinite(weight_decay))
    return QLORA_ERR_INVALID_ARG;
  if (n == 0) return QLORA_OK;
  if (!param || !grad || !factor || !exp_avg || !exp_avg_sq) return QLORA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(factor) & 3) return QLORA_ERR_ALIGN;
  void* view[5] = {param, const_cast<void*>(grad), exp_avg, exp_avg_sq, param_bf16};
  for (const void* p : view)
    if (p && !aligned16(p)) return QLORA_ERR_ALIGN;
  for (void*& p : view) {
    if (p && !(p = reached(p))) return QLORA_ERR_INVALID_ARG;
    if (p && !aligned16(p)) return QLORA_ERR_ALIGN;  // the mapped address, too
  }
  // Every workgroup reads the factor: not from what others have written.
  const Span f = span_of(factor, 4);
  for (int i : {0, 2, 3, 4})
    if (meet(span_of(view[i], n * (i == 4 ? 2 : 4)), f)) return QLORA_ERR_INVALID_ARG;
  const double b1t = std::pow(beta1, (double)step), b2t = std::pow(beta2, (double)step);
  AdamScalars s;
  s.b1 = (float)beta1;
  s.b2 = (float)beta2;
  s.eps = (float)eps;
  s.decay = (float)(1.0 - lr * weight_decay);
  s.c1 = (float)(1.0 - beta1);
  s.c2 = (float)(1.0 - beta2);
  s.step_size = (float)(lr / (1.0 - b1t));
  s.bc2_sqrt = (float)std::sqrt(1.0 - b2t);
  return launch_status(launch_adamw_scaled(
      static_cast<float*>(view[0]), view[1], grad_dtype == QLORA_DTYPE_BF16,
      static_cast<float*>(view[2]), static_cast<float*>(view[3]), static_cast<uint16_t*>(view[4]), n,
      s, factor, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
