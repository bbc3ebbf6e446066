// The global norm of many gradients and its clipping on gfx950:
//   norm   = sqrt(sum over all tensors of g^2)
//   factor = max_norm / norm where norm > max_norm, else 1
//   out    = g * factor
//
// The squares are formed and summed in 64 bits: the square of an fp32 value is
// exact there, nothing overflows (gradients of 2^100 have a norm), and the
// order of the additions is beyond what the fp32 result shows. It costs no
// time, memory bounds the pass: a CU sees 4 bf16 elements a cycle at 5 TB/s and
// has 64 fused operations of 64 bits a cycle.
//
// A tensor is cut into chunks of 32 KB (more where there would be over 2^14 of
// them), a workgroup each. A program whose gradients stay where they are keeps a
// table of the chunks on the device: one launch for all tensors, one load to find
// a chunk. Without it the tensors travel in the launches' own arguments, 128 of
// them a launch, and a workgroup finds its tensor by a ballot over the chunks'
// ends (448 adapter gradients, 80 MB: norm and scale 71 us in eight launches).
//
// The norm reads with plain loads, the scaling reads for the last time and writes
// with the nontemporal hint, so that what the norm has read is still in the
// Infinity Cache when it is scaled (134 MB of fp32: 52 us a pair, without the hints
// 68 us, with the hint in the norm too 63 us; the bytes alone are 47 us).
#include "rows.h"
#include "spans_table.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;

// A workgroup's chunk.
struct Chunk {
  const void* in;
  void* out;
  int64_t n;
  bool bf16;
};

// The tensor that chunk `c` of a launch belongs to is the number of tensors that
// end at or before it.
__device__ __forceinline__ Chunk chunk_of(const SpanTable& t, uint32_t c) {
  const int lane = threadIdx.x & 63;
  int s = 0;
#pragma unroll
  for (int k = 0; k < kSpans; k += 64)
    s += __popcll(__ballot(k + lane < t.count && t.end[k + lane] <= c));
  s = __builtin_amdgcn_readfirstlane(s);
  const bool bf16 = t.bf16(s);
  const int64_t most = t.chunk >> (bf16 ? 1 : 2);
  const int64_t first = (int64_t)(c - (s ? t.end[s - 1] : 0u)) * most, left = t.n[s] - first;
  const int64_t at = first << (bf16 ? 1 : 2);
  return Chunk{static_cast<const char*>(t.in[s]) + at,
               t.out[s] ? static_cast<char*>(t.out[s]) + at : nullptr, left < most ? left : most, bf16};
}

struct Tables {
  const ChunkEntry* in;
  const ChunkEntry* out;  // NULL for the norm
};

__device__ __forceinline__ Chunk chunk_of(const Tables& t, uint32_t c) {
  const ChunkEntry e = t.in[c];
  return Chunk{reinterpret_cast<const void*>(e.data),
               t.out ? reinterpret_cast<void*>(t.out[c].data) : nullptr, (int64_t)e.n, e.bf16 != 0};
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Sum over a workgroup; thread 0 has it.
template <int kWaves>
__device__ __forceinline__ double block_sum(double v, double* red) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = red[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s += red[w];
  return s;
}

constexpr int kDepth = 4;  // vectors of a thread whose loads are in flight together

template <bool kBf16>
__device__ __forceinline__ double squares(const Chunk& c) {
  constexpr int E = kBf16 ? 8 : 4;
  const elem_t<kBf16>* p = static_cast<const elem_t<kBf16>*>(c.in);
  const int64_t last = c.n;
  double s[2] = {0.0, 0.0};
  int64_t at = (int64_t)threadIdx.x * E;
  for (; at + (int64_t)(kDepth - 1) * kThreads * E + E <= last; at += (int64_t)kDepth * kThreads * E) {
    Vec<kBf16, E> r[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) r[d] = load_vec<kBf16, E>(p + at + (int64_t)d * kThreads * E);
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      float v[E];
      to_float<kBf16, E>(r[d], v);
#pragma unroll
      for (int e = 0; e < E; ++e) s[e & 1] = fma((double)v[e], (double)v[e], s[e & 1]);
    }
  }
  for (; at < last; at += (int64_t)kThreads * E) {
    const int n = count_below<E>(at, last);
    const Vec<kBf16, E> r = n == E ? load_vec<kBf16, E>(p + at) : load_part<kBf16, E>(p + at, n);
    float v[E];
    to_float<kBf16, E>(r, v);
#pragma unroll
    for (int e = 0; e < E; ++e) s[e & 1] = fma((double)v[e], (double)v[e], s[e & 1]);
  }
  return s[0] + s[1];
}

template <typename Table>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(Table t, double* part) {
  __shared__ double red[kThreads / 64];
  const Chunk c = chunk_of(t, blockIdx.x);
  const double all = block_sum<kThreads / 64>(c.bf16 ? squares<true>(c) : squares<false>(c), red);
  if (threadIdx.x == 0) part[blockIdx.x] = all;
}

constexpr int kJoin = 1024;

// result = (norm, factor) from the chunks' sums, thread by thread in order.
__global__ __launch_bounds__(kJoin) void grad_norm_join_kernel(const double* part, int64_t parts,
                                                               float max_norm, float* result) {
  __shared__ double red[kJoin / 64];
  double s = 0.0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < parts; i += kJoin) s += part[i];
  const double all = block_sum<kJoin / 64>(s, red);
  if (threadIdx.x == 0) {
    const double norm = __builtin_sqrt(all);
    result[0] = (float)norm;
    // a NaN stays one; an infinite norm has the factor 0
    result[1] = norm > (double)max_norm ? (float)((double)max_norm / norm)
                                        : norm == norm ? 1.0f : (float)norm;
  }
}

template <bool kBf16>
__device__ __forceinline__ void scale(const Chunk& c, float f) {
  constexpr int E = kBf16 ? 8 : 4;
  const elem_t<kBf16>* p = static_cast<const elem_t<kBf16>*>(c.in);
  elem_t<kBf16>* out = static_cast<elem_t<kBf16>*>(c.out);
  const int64_t last = c.n;
  int64_t at = (int64_t)threadIdx.x * E;
  for (; at + (int64_t)(kDepth - 1) * kThreads * E + E <= last; at += (int64_t)kDepth * kThreads * E) {
    Vec<kBf16, E> r[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) r[d] = load_vec<kBf16, E, true>(p + at + (int64_t)d * kThreads * E);
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      float v[E];
      to_float<kBf16, E>(r[d], v);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] *= f;
      store_vec<kBf16, E, true>(out + at + (int64_t)d * kThreads * E, v);
    }
  }
  for (; at < last; at += (int64_t)kThreads * E) {
    const int n = count_below<E>(at, last);
    const Vec<kBf16, E> r = n == E ? load_vec<kBf16, E, true>(p + at) : load_part<kBf16, E>(p + at, n);
    float v[E];
    to_float<kBf16, E>(r, v);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= f;
    if (n == E)
      store_vec<kBf16, E, true>(out + at, v);
    else
      store_part<kBf16, E>(out + at, v, n);
  }
}

// In place a factor of 1 changes nothing, and nothing is read or written.
template <typename Table>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(Table t, const float* factor) {
  const float f = *factor;
  const Chunk c = chunk_of(t, blockIdx.x);
  if (f == 1.0f && c.in == c.out) return;
  if (c.bf16)
    scale<true>(c, f);
  else
    scale<false>(c, f);
}

}  // namespace

hipError_t launch_grad_norm(const SpanTable& t, uint32_t chunks, double* part, hipStream_t st) {
  hipLaunchKernelGGL(grad_norm_kernel<SpanTable>, dim3(chunks), dim3(kThreads), 0, st, t, part);
  return hipGetLastError();
}

hipError_t launch_grad_norm_table(const ChunkEntry* in, uint32_t chunks, double* part,
                                  hipStream_t st) {
  hipLaunchKernelGGL(grad_norm_kernel<Tables>, dim3(chunks), dim3(kThreads), 0, st,
                     Tables{in, nullptr}, part);
  return hipGetLastError();
}

hipError_t launch_grad_norm_join(const double* part, int64_t parts, float max_norm, float* result,
                                 hipStream_t st) {
  hipLaunchKernelGGL(grad_norm_join_kernel, dim3(1), dim3(kJoin), 0, st, part, parts, max_norm,
                     result);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const SpanTable& t, uint32_t chunks, const float* factor,
                             hipStream_t st) {
  hipLaunchKernelGGL(grad_scale_kernel<SpanTable>, dim3(chunks), dim3(kThreads), 0, st, t, factor);
  return hipGetLastError();
}

hipError_t launch_grad_scale_table(const ChunkEntry* in, const ChunkEntry* out, uint32_t chunks,
                                   const float* factor, hipStream_t st) {
  hipLaunchKernelGGL(grad_scale_kernel<Tables>, dim3(chunks), dim3(kThreads), 0, st, Tables{in, out},
                     factor);
  return hipGetLastError();
}

}  // namespace qlora
