// Checks of arguments that the row operators' entry points share.
#pragma once

#include "host.h"
#include "spans.h"

namespace qlora {

inline bool float_type(int d) { return d == QLORA_DTYPE_F32 || d == QLORA_DTYPE_BF16; }
inline bool index_type(int d) { return d == QLORA_DTYPE_I32 || d == QLORA_DTYPE_I64; }
inline int64_t elem_bytes(int dtype) { return dtype == QLORA_DTYPE_BF16 ? 2 : dtype == QLORA_DTYPE_I64 ? 8 : 4; }

// The alignment of an element of a QLORA_DTYPE_* type.
inline bool aligned_elem(const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(elem_bytes(dtype) - 1)) == 0;
}

// What an argument occupies, for the check that no output lies on an input:
// rows of a matrix, or a contiguous array.
inline Span matrix(const void* p, int64_t rows, int64_t width, int64_t ld, int dtype) {
  return span_of(p, rows, width, ld, elem_bytes(dtype));
}
inline Span array(const void* p, int64_t count, int dtype) { return span_of(p, count * elem_bytes(dtype)); }
inline Span bytes(const void* p, size_t n) { return span_of(p, (int64_t)n); }
// An output that may be the input `in` itself, at the same address and stride
// in the same type: no span of its own then.
inline Span unless_same(const Span& in, const Span& out) { return in.same(out) ? Span{} : in; }

// Rows of `width` elements every `ld`: the last row's end stays countable.
inline bool stride_ok(int64_t M, int64_t width, int64_t ld) {
  return ld >= width && ld <= kMaxElems / (M > 0 ? M : 1);
}

inline bool norm_shape_ok(int64_t M, int64_t N) {
  return M >= 0 && M <= QLORA_MAX_ROWS && N >= 1 && N <= QLORA_MAX_NORM_WIDTH;
}

}  // namespace qlora
