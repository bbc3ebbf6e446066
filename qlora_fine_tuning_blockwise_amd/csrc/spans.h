// Whether two strided matrices share memory, decided on the host from their
// addresses and strides alone (the row operators refuse outputs over inputs).
// Plain C++: no HIP types, so that it can be checked on a host by itself.
#pragma once

#include <cstdint>
#include <initializer_list>

namespace qlora {

// `rows` runs of `width` bytes, the first at p, each `step` bytes after the
// last (step >= width). NULL or without bytes: nothing.
struct Span {
  uintptr_t p = 0;
  int64_t rows = 0, width = 0, step = 0;

  bool empty() const { return p == 0 || rows <= 0 || width <= 0; }
  uintptr_t end() const { return p + (uintptr_t)((rows - 1) * step + width); }
  bool same(const Span& o) const {
    return p == o.p && rows == o.rows && width == o.width && (rows <= 1 || step == o.step);
  }
};

inline Span span_of(const void* p, int64_t rows, int64_t width, int64_t ld, int64_t size) {
  return {reinterpret_cast<uintptr_t>(p), rows, width * size, ld * size};
}
inline Span span_of(const void* p, int64_t bytes) {
  return {reinterpret_cast<uintptr_t>(p), 1, bytes, bytes};
}

// Quotient towards minus infinity.
inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && (a < 0) != (b < 0)); }

inline bool meet(const Span& a, const Span& b) {
  if (a.empty() || b.empty() || a.end() <= b.p || b.end() <= a.p) return false;
  // One run has any step: it takes the other's.
  const int64_t step = a.rows > 1 ? a.step : b.step;
  const int64_t d = (int64_t)(b.p - a.p);
  if (a.rows == 1 || b.rows == 1 || a.step == b.step) {
    // Row j of b lies d + k step, k = j - i, behind row i of a: they meet where
    // that is in (-b.width, a.width). Columns of one wider matrix do not.
    int64_t least = floor_div(-b.width - d, step) + 1, most = -floor_div(d - a.width, step) - 1;
    if (least < 1 - a.rows) least = 1 - a.rows;
    if (most > b.rows - 1) most = b.rows - 1;
    return least <= most;
  }
  // Different steps: the rows in the order of their addresses, whole gaps at once.
  int64_t i = 0, j = 0;
  while (i < a.rows && j < b.rows) {
    const int64_t x = i * a.step, y = d + j * b.step;  // places behind a.p
    if (x + a.width <= y)
      i += 1 + (y - x - a.width) / a.step;
    else if (y + b.width <= x)
      j += 1 + (x - y - b.width) / b.step;
    else
      return true;
  }
  return false;
}

// Whether an output lies on an input or on another output.
inline bool any_meet(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (const Span* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Span& in : inputs)
      if (meet(*o, in)) return true;
    for (const Span* other = o + 1; other != outputs.end(); ++other)
      if (meet(*o, *other)) return true;
  }
  return false;
}

}  // namespace qlora
