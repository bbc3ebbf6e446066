// What the kernels of the vocabulary head's loss share: values split into bf16
// terms.
#pragma once

#include "head.h"
#include "rows.h"

namespace qlora {

// Four values in bf16, and with two terms what they lost, `plane` elements on.
__device__ __forceinline__ void store_terms(uint16_t* to, int64_t plane, int terms, const float (&v)[4]) {
  const u32x2_t hi = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  *reinterpret_cast<u32x2_t*>(to) = hi;
  if (terms == 2)
    *reinterpret_cast<u32x2_t*>(to + plane) =
        u32x2_t{pack_bf16x2(v[0] - bf16_lo(hi[0]), v[1] - bf16_hi(hi[0])),
                pack_bf16x2(v[2] - bf16_lo(hi[1]), v[3] - bf16_hi(hi[1]))};
}

}  // namespace qlora
