// Device-side helpers of the row operators (embedding, norm, distillation):
// access to rows of bf16 or fp32 at any element alignment, and reductions
// over a wave or a workgroup.
#pragma once

#include <type_traits>

#include "device.h"

namespace qlora {

// Accesses of 8 and 16 bytes that need only their element's alignment: gfx950
// takes a global access of several dwords at any byte address, so rows of odd
// width or stride run the same code as aligned ones.
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

template <bool kBf16>
using elem_t = typename std::conditional<kBf16, uint16_t, float>::type;

// E consecutive elements of a row as they lie in memory: 8 bf16 in 16 bytes,
// or 4 elements (a row operator that touches fp32 takes all its rows by four,
// so that every access of a wave is one run without gaps).
template <bool kBf16, int E>
struct Vec {
  static_assert(E == 8 || E == 4, "elements of a vector");
  static constexpr int kWords = kBf16 ? E / 2 : E;
  uint32_t w[kWords];
};

template <bool kBf16, int E, bool kNt = false>
__device__ __forceinline__ Vec<kBf16, E> load_vec(const elem_t<kBf16>* p) {
  Vec<kBf16, E> r;
  if constexpr (kBf16 && E == 4) {
    const u32x2_a2* v = reinterpret_cast<const u32x2_a2*>(p);
    const u32x2_a2 q = kNt ? __builtin_nontemporal_load(v) : *v;
    r.w[0] = q[0];
    r.w[1] = q[1];
  } else {
    using V = typename std::conditional<kBf16, u32x4_a2, u32x4_a4>::type;
#pragma unroll
    for (int h = 0; h < Vec<kBf16, E>::kWords / 4; ++h) {
      const V* v = reinterpret_cast<const V*>(p) + h;
      const V q = kNt ? __builtin_nontemporal_load(v) : *v;
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[4 * h + i] = q[i];
    }
  }
  return r;
}

// A vector of one value, given by its bits: 0, or -infinity for a maximum.
constexpr uint32_t kNegInf = 0xFF800000u;

template <bool kBf16, int E, uint32_t kFill = 0u>
__device__ __forceinline__ Vec<kBf16, E> fill_vec() {
  Vec<kBf16, E> r;
#pragma unroll
  for (int i = 0; i < Vec<kBf16, E>::kWords; ++i)
    r.w[i] = kBf16 ? (kFill & 0xFFFF0000u) | kFill >> 16 : kFill;
  return r;
}
template <bool kBf16, int E>
__device__ __forceinline__ Vec<kBf16, E> zero_vec() {
  return fill_vec<kBf16, E>();
}

// The elements first <= e < n of the vector (the others the fill value): a
// row's ends.
template <bool kBf16, int E, uint32_t kFill = 0u>
__device__ __forceinline__ Vec<kBf16, E> load_part(const elem_t<kBf16>* p, int n, int first = 0) {
  Vec<kBf16, E> r = fill_vec<kBf16, E, kFill>();
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (e >= first && e < n) {
      if constexpr (kBf16)
        r.w[e / 2] = e & 1 ? (r.w[e / 2] & 0xFFFFu) | (uint32_t)p[e] << 16
                           : (r.w[e / 2] & 0xFFFF0000u) | p[e];
      else
        r.w[e] = __float_as_uint(p[e]);
    }
  return r;
}

template <bool kBf16, int E>
__device__ __forceinline__ void to_float(const Vec<kBf16, E>& r, float (&v)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if constexpr (kBf16)
      v[i] = i & 1 ? bf16_hi(r.w[i / 2]) : bf16_lo(r.w[i / 2]);
    else
      v[i] = __uint_as_float(r.w[i]);
  }
}

// Stores round to nearest even, once.
template <bool kBf16, int E, bool kNt = false>
__device__ __forceinline__ void store_vec(elem_t<kBf16>* p, const float (&v)[E]) {
  if constexpr (kBf16 && E == 4) {
    const u32x2_t q = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    u32x2_a2* d = reinterpret_cast<u32x2_a2*>(p);
    if (kNt)
      __builtin_nontemporal_store(q, d);
    else
      *d = q;
  } else if constexpr (kBf16) {
    const u32x4_t q = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7])};
    u32x4_a2* d = reinterpret_cast<u32x4_a2*>(p);
    if (kNt)
      __builtin_nontemporal_store(q, d);
    else
      *d = q;
  } else {
#pragma unroll
    for (int h = 0; h < E / 4; ++h) {
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

template <bool kBf16, int E>
__device__ __forceinline__ void store_part(elem_t<kBf16>* p, const float (&v)[E], int n,
                                           int first = 0) {
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (e >= first && e < n) store1<kBf16>(p + e, v[e]);
}

// How many of a vector's E elements at `at` lie below `end`.
template <int E>
__device__ __forceinline__ int count_below(int64_t at, int64_t end) {
  const int64_t left = end - at;
  return left >= E ? E : left < 0 ? 0 : (int)left;
}

// An element of an array whose type is a run-time value.
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
// of 64). `red` holds two halves of kMostReduced values for each wave of the
// workgroup, used in turn (`par`), so one barrier a reduction is enough: a
// wave writes a half again only after a barrier that every wave reaches once
// it has read it. The halves lie at the same places whatever K is: reductions
// of one and of two values follow each other. All threads of the workgroup
// call it.
constexpr int kMostReduced = 2;
template <int T, int K, typename Op>
__device__ __forceinline__ void group_reduce(float (&v)[K], float* red, int waves, int& par,
                                             Op op) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_reduce(v[k], op);
  if constexpr (T > 64) {
    const int wave = threadIdx.x >> 6;
    static_assert(K <= kMostReduced, "values of a reduction");
    float* half = red + par * kMostReduced * waves;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) half[k * waves + wave] = v[k];
    }
    __syncthreads();
    // lane l takes the value of wave l % W of its group; the W lanes join
    constexpr int W = T / 64;
    static_assert(W == 2 || W == 4 || W == 8 || W == 16, "waves of a group");
    const int from = (wave & ~(W - 1)) + (threadIdx.x & (W - 1));
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = half[k * waves + from];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = op(v[k], dpp<0xB1>(v[k]));
      if constexpr (W >= 4) v[k] = op(v[k], dpp<0x4E>(v[k]));
      if constexpr (W >= 8) v[k] = op(v[k], dpp<0x141>(v[k]));
      if constexpr (W >= 16) v[k] = op(v[k], dpp<0x140>(v[k]));
    }
    par ^= 1;
  }
}

}  // namespace qlora
