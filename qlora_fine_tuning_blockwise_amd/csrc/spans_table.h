// Many tensors as the kernels of the gradients' norm take them: cut into chunks,
// a workgroup each.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace qlora {

// One chunk of a tensor, as a program's own table of them on the device holds it.
struct ChunkEntry {
  uint64_t data;
  uint32_t n, bf16;
};
static_assert(sizeof(ChunkEntry) == 16, "one load");

// Tensors of a launch without such a table: its own arguments, which stay below
// 4 KB, the size that every HIP runtime passes.
constexpr int kSpans = 128;

struct SpanTable {
  const void* in[kSpans];
  void* out[kSpans];     // where the scaled elements go; not used by the norm
  int64_t n[kSpans];     // elements
  uint32_t end[kSpans];  // chunks up to and with this tensor
  uint64_t bf16_bits[kSpans / 64];  // fp32 where the bit is not set
  int64_t chunk;                    // bytes of a chunk, a multiple of 16
  int count;

  __host__ __device__ bool bf16(int s) const { return bf16_bits[s >> 6] >> (s & 63) & 1; }
};
static_assert(sizeof(SpanTable) <= 4096 - 64, "a launch's arguments");

hipError_t launch_grad_norm(const SpanTable& t, uint32_t chunks, double* part, hipStream_t st);
hipError_t launch_grad_scale(const SpanTable& t, uint32_t chunks, const float* factor,
                             hipStream_t st);
// The same with tables on the device.
hipError_t launch_grad_norm_table(const ChunkEntry* in, uint32_t chunks, double* part,
                                  hipStream_t st);
hipError_t launch_grad_scale_table(const ChunkEntry* in, const ChunkEntry* out, uint32_t chunks,
                                   const float* factor, hipStream_t st);

hipError_t launch_grad_norm_join(const double* part, int64_t parts, float max_norm, float* result,
                                 hipStream_t st);

}  // namespace qlora
