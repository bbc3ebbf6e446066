// What the kernels of the vocabulary head's loss share: values split into bf16
// terms.
#pragma once

#include "head.h"
#include "rows.h"

namespace qlora {

// Term kTerm of four values that are written as sums of bf16 numbers: each is the
// nearest to what those before it leave.
template <int kTerm>
__device__ __forceinline__ u32x2_t term_of(float a, float b, float c, float d) {
  u32x2_t q = {pack_bf16x2(a, b), pack_bf16x2(c, d)};
  if constexpr (kTerm > 0) {
    q = term_of<kTerm - 1>(a - bf16_lo(q[0]), b - bf16_hi(q[0]), c - bf16_lo(q[1]), d - bf16_hi(q[1]));
  }
  return q;
}

// One term, or all three, `plane` elements apart.
__device__ __forceinline__ void store_terms(uint16_t* to, int64_t plane, int terms, const float (&v)[4]) {
  *reinterpret_cast<u32x2_t*>(to) = term_of<0>(v[0], v[1], v[2], v[3]);
  if (terms == 1) return;
  *reinterpret_cast<u32x2_t*>(to + plane) = term_of<1>(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<u32x2_t*>(to + 2 * plane) = term_of<2>(v[0], v[1], v[2], v[3]);
}

}  // namespace qlora
