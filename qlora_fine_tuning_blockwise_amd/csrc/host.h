// Host helpers that the files of entry points share: alignment, sizes, and the
// carving of a workspace.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/qlora_amd.h"
#include "internal.h"

namespace qlora {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Every product of two of M, N and K stays at most 2^40 (a bf16 matrix of
// 2 TiB, far beyond one GPU's memory), so no byte count, workspace size or
// offset formed from them can overflow 64 bits.
constexpr int64_t kMaxElems = int64_t(1) << 40;

inline size_t round_up(size_t v) { return (v + 255) & ~(size_t)255; }

// Workspace carve-up, shared by the size query and the entry points.
struct Carve {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t o = off;
    off += round_up(bytes);
    return o;
  }
};

template <typename T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(base) + off);
}

inline int launch_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_LAUNCH; }

}  // namespace qlora
