// Device-side helpers of the row operators (embedding, norm, distillation):
// access to rows of bf16 or fp32 at any element alignment, and reductions
// over a wave or a workgroup.
#pragma once

#include "device.h"

namespace qlora {

// 16-byte accesses that need only their element's alignment: gfx950 takes a
// global access of four dwords at any byte address, so rows of odd width or
// stride run the same code as aligned ones.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight consecutive elements of a row as they lie in memory.
template <bool kBf16>
struct Row8 {
  u32x4_t q[kBf16 ? 1 : 2];
};

template <bool kBf16>
using elem_t = typename std::conditional<kBf16, uint16_t, float>::type;

template <bool kBf16, bool kNt = false>
__device__ __forceinline__ Row8<kBf16> load8(const elem_t<kBf16>* p) {
  Row8<kBf16> r;
  if constexpr (kBf16) {
    const u32x4_a2* v = reinterpret_cast<const u32x4_a2*>(p);
    r.q[0] = kNt ? __builtin_nontemporal_load(v) : *v;
  } else {
    const u32x4_a4* v = reinterpret_cast<const u32x4_a4*>(p);
    r.q[0] = kNt ? __builtin_nontemporal_load(v) : v[0];
    r.q[1] = kNt ? __builtin_nontemporal_load(v + 1) : v[1];
  }
  return r;
}

template <bool kBf16>
__device__ __forceinline__ Row8<kBf16> zero8() {
  Row8<kBf16> r;
  r.q[0] = zero4();
  if constexpr (!kBf16) r.q[1] = zero4();
  return r;
}

// The first n < 8 of the eight (the rest +0): a row's last elements.
template <bool kBf16>
__device__ __forceinline__ Row8<kBf16> load8_part(const elem_t<kBf16>* p, int n) {
  uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) {
      if constexpr (kBf16)
        w[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
      else
        w[e] = __float_as_uint(p[e]);
    }
  Row8<kBf16> r;
  r.q[0] = u32x4_t{w[0], w[1], w[2], w[3]};
  if constexpr (!kBf16) r.q[1] = u32x4_t{w[4], w[5], w[6], w[7]};
  return r;
}

template <bool kBf16>
__device__ __forceinline__ void to_float(const Row8<kBf16>& r, float v[8]) {
  if constexpr (kBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(r.q[0][i]);
      v[2 * i + 1] = bf16_hi(r.q[0][i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.q[i / 4][i % 4]);
  }
}

// Stores round to nearest even, once.
template <bool kBf16, bool kNt = false>
__device__ __forceinline__ void store8(elem_t<kBf16>* p, const float v[8]) {
  if constexpr (kBf16) {
    const u32x4_t q = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7])};
    u32x4_a2* d = reinterpret_cast<u32x4_a2*>(p);
    if (kNt)
      __builtin_nontemporal_store(q, d);
    else
      *d = q;
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4_t q = {__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                         __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])};
      u32x4_a4* d = reinterpret_cast<u32x4_a4*>(p) + h;
      if (kNt)
        __builtin_nontemporal_store(q, d);
      else
        *d = q;
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ void store1(elem_t<kBf16>* p, float v) {
  if constexpr (kBf16)
    *p = (uint16_t)pack_bf16x2(v, 0.0f);
  else
    *p = v;
}

template <bool kBf16>
__device__ __forceinline__ void store8_part(elem_t<kBf16>* p, const float v[8], int n) {
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) store1<kBf16>(p + e, v[e]);
}

// Eight elements (or the first n) of an array whose type is a run-time value.
__device__ __forceinline__ void load_any8(const void* p, bool bf16, int64_t at, int n, float v[8]) {
  if (bf16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    to_float<true>(n >= 8 ? load8<true>(q) : load8_part<true>(q, n), v);
  } else {
    const float* q = static_cast<const float*>(p) + at;
    to_float<false>(n >= 8 ? load8<false>(q) : load8_part<false>(q, n), v);
  }
}

__device__ __forceinline__ float load_any(const void* p, bool bf16, int64_t at) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[at] << 16)
              : static_cast<const float*>(p)[at];
}

// An index of one of the two integer types.
__device__ __forceinline__ int64_t load_index(const void* p, bool i64, int64_t at) {
  return i64 ? static_cast<const int64_t*>(p)[at] : (int64_t)static_cast<const int32_t*>(p)[at];
}

// ------------------------------------------------------------- reductions
// Butterflies over the 64 lanes: every lane gets the result, with the same
// bits (the additions of a pair commute). Within 16 lanes the partner comes
// by DPP (no LDS round trip), then the rows of 16 and the halves are
// exchanged by the permlane swaps.
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), kCtrl, 0xF, 0xF, false));
}

struct OpSum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// The larger one; a NaN is passed over (it reaches the sum that follows).
struct OpMax {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

template <typename Op>
__device__ __forceinline__ float wave_reduce(float v, Op op) {
  v = op(v, dpp<0xB1>(v));   // lane ^ 1
  v = op(v, dpp<0x4E>(v));   // lane ^ 2
  v = op(v, dpp<0x141>(v));  // the other four of eight (mirrored)
  v = op(v, dpp<0x140>(v));  // the other eight of sixteen (mirrored)
  const uint32_t b = __float_as_uint(v);
  const auto s16 = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  v = op(__uint_as_float(s16[0]), __uint_as_float(s16[1]));
  const uint32_t c = __float_as_uint(v);
  const auto s32 = __builtin_amdgcn_permlane32_swap(c, c, false, false);
  return op(__uint_as_float(s32[0]), __uint_as_float(s32[1]));
}

// K values reduced over the T threads of a group of a workgroup (T a multiple
// of 64; `red` holds 2 * K * (waves of the workgroup) floats). The two halves
// of `red` are used in turn (`par`), so one barrier a reduction is enough: a
// wave writes a half again only after a barrier that every wave reaches once
// it has read it. All threads of the workgroup call it.
template <int T, int K, typename Op>
__device__ __forceinline__ void group_reduce(float (&v)[K], float* red, int waves, int& par,
                                             Op op) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_reduce(v[k], op);
  if constexpr (T > 64) {
    const int wave = threadIdx.x >> 6;
    float* half = red + par * K * waves;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) half[k * waves + wave] = v[k];
    }
    __syncthreads();
    const int first = wave & ~(T / 64 - 1);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = half[k * waves + first];
#pragma unroll
      for (int w = 1; w < T / 64; ++w) s = op(s, half[k * waves + first + w]);
      v[k] = s;
    }
    par ^= 1;
  }
}

}  // namespace qlora
