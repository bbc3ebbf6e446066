// Token embedding on gfx950: the scaled lookup and its dense gradient.
//
//   out[m] = scale W[id_m];   dW[v] = scale * sum over m with id_m = v of dY[m]
//
// An id outside of [0, V) has no row of the table: its output row is zero and
// its dY row is not read.
//
// The gradient sorts the tokens by id (ties by position), so that each table
// row is one sum in token order, whatever the launch: no atomics, the same
// bits every time.
//   1. Workgroups of the first launch sort runs of kRun tokens in LDS; the
//      others fill dW with zeros, which is most of the call's traffic and
//      hides the sort.
//   2. With more than one run, a token's place is its place in its own run
//      plus, by binary search, the count of smaller keys in the others.
//   3. The sorted tokens are cut into tiles. A wave adds one tile's rows over
//      512 columns in fp32 and writes each id whose tokens all lie in the
//      tile; a sum that passes a tile's border goes to the workspace.
//   4. The tile in which such a sum begins collects its parts in tile order.
#include <type_traits>

#include "rows.h"

namespace qlora {
namespace {

constexpr int kRun = 4096;           // tokens sorted in one workgroup
constexpr int32_t kDead = 0x7fffffff;  // sort key of an id outside of the table

// ------------------------------------------------------------------ lookup
struct EmbedFwd {
  const void* W;
  int64_t ldw, V;
  int D;
  const void* ids;
  bool ids64;
  int64_t M;
  float scale;
  void* out;
  int64_t ldo;
};

template <bool WB, bool OB, int T>
__global__ __launch_bounds__(256) void embed_fwd_kernel(EmbedFwd a) {
  constexpr int kRows = 256 / T;
  const int t = threadIdx.x % T;
  const int full = a.D / 8, tail = a.D % 8;
  for (int64_t m = (int64_t)blockIdx.x * kRows + threadIdx.x / T; m < a.M;
       m += (int64_t)gridDim.x * kRows) {
    const int64_t id = load_index(a.ids, a.ids64, m);
    const bool live = id >= 0 && id < a.V;
    const elem_t<WB>* w = static_cast<const elem_t<WB>*>(a.W) + (live ? id : 0) * a.ldw;
    elem_t<OB>* o = static_cast<elem_t<OB>*>(a.out) + m * a.ldo;
    for (int c0 = t; c0 < full; c0 += 4 * T) {
      Vec<WB, 8> r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        r[u] = live && c0 + u * T < full ? load_vec<WB, 8>(w + (c0 + u * T) * 8) : zero_vec<WB, 8>();
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c0 + u * T < full) {
          float v[8];
          to_float<WB, 8>(r[u], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = live ? v[e] * a.scale : 0.0f;
          store_vec<OB, 8>(o + (c0 + u * T) * 8, v);
        }
    }
    if (t < tail) {
      const int c = full * 8 + t;
      store1<OB>(o + c, live ? load_any(w, WB, c) * a.scale : 0.0f);
    }
  }
}

// ---------------------------------------------------------------- the sort
__device__ __forceinline__ int32_t sort_key(const void* ids, bool i64, int64_t m, int64_t V) {
  const int64_t id = load_index(ids, i64, m);
  return id >= 0 && id < V ? (int32_t)id : kDead;
}

// Workgroup b < runs sorts tokens [b kRun, (b + 1) kRun) by (key, position)
// with a bitonic network in LDS; the rest write zeros over dW.
__global__ __launch_bounds__(1024) void embed_sort_kernel(const void* ids, bool i64, int64_t M,
                                                          int64_t V, int runs, int32_t* key,
                                                          int32_t* pos, u32x4_t* dW,
                                                          int64_t halves) {
  __shared__ uint64_t s[kRun];
  if ((int)blockIdx.x >= runs) {
    // halves: two-byte units of dW, whose base is 16-byte aligned
    const int64_t quads = halves / 8, stride = (int64_t)(gridDim.x - runs) * 1024;
    const int64_t first = (int64_t)(blockIdx.x - runs) * 1024 + threadIdx.x;
    for (int64_t i = first; i < quads; i += stride) dW[i] = zero4();
    if (first < halves % 8) reinterpret_cast<uint16_t*>(dW)[quads * 8 + first] = 0;
    return;
  }
  const int64_t base = (int64_t)blockIdx.x * kRun;
  const int n = (int)(M - base < kRun ? M - base : kRun);
  int n2 = 2;
  while (n2 < n) n2 *= 2;
  for (int i = threadIdx.x; i < n2; i += 1024)
    s[i] = i < n ? (uint64_t)(uint32_t)sort_key(ids, i64, base + i, V) << 32 | (uint32_t)i
                 : ~(uint64_t)0;
  __syncthreads();
  for (int k = 2; k <= n2; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      for (int p = threadIdx.x; p < n2 / 2; p += 1024) {
        const int i = (p & ~(j - 1)) * 2 + (p & (j - 1));
        const uint64_t a = s[i], b = s[i + j];
        if ((a > b) == ((i & k) == 0)) {
          s[i] = b;
          s[i + j] = a;
        }
      }
      __syncthreads();
    }
  for (int i = threadIdx.x; i < n; i += 1024) {
    key[base + i] = (int32_t)(s[i] >> 32);
    pos[base + i] = (int32_t)(base + (int32_t)(uint32_t)s[i]);
  }
}

__global__ __launch_bounds__(256) void embed_rank_kernel(const int32_t* __restrict__ key,
                                                         const int32_t* __restrict__ pos,
                                                         int64_t M, int runs,
                                                         int32_t* __restrict__ key_out,
                                                         int32_t* __restrict__ pos_out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= M) return;
  const int own = (int)(i / kRun);
  const int32_t k = key[i];
  int64_t rank = i - (int64_t)own * kRun;
  for (int r = 0; r < runs; ++r) {
    if (r == own) continue;
    // keys before k: those below it, and in an earlier run its equals too
    const int32_t* p = key + (int64_t)r * kRun;
    const int n = (int)(M - (int64_t)r * kRun < kRun ? M - (int64_t)r * kRun : kRun);
    const bool equals = r < own;
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      const int32_t v = p[mid];
      if (v < k || (equals && v == k))
        lo = mid + 1;
      else
        hi = mid;
    }
    rank += lo;
  }
  key_out[rank] = k;
  pos_out[rank] = pos[i];
}

// ---------------------------------------------------------------- the sums
struct EmbedBwd {
  const void* dY;
  int64_t ldy, M;
  int D;
  float scale;
  bool accumulate;
  void* dW;
  const int32_t* key;
  const int32_t* pos;
  float* part;  // [tiles][2][ldp]: the sum that began before the tile, the one that passes its end
  int ldp, tile;
};

template <bool GB>
__device__ __forceinline__ void write_row(const EmbedBwd& a, int32_t id, int c, int n,
                                          const float (&acc)[8]) {
  elem_t<GB>* p = static_cast<elem_t<GB>*>(a.dW) + (int64_t)id * a.D + c;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = acc[e] * a.scale;
  if (a.accumulate) {
    float old[8];
    to_float<GB, 8>(n >= 8 ? load_vec<GB, 8>(p) : load_part<GB, 8>(p, n), old);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += old[e];
  }
  if (n >= 8)
    store_vec<GB, 8>(p, v);
  else
    store_part<GB, 8>(p, v, n);
}

template <bool YB, bool GB>
__global__ __launch_bounds__(64) void embed_sum_kernel(EmbedBwd a) {
  const int64_t tile = blockIdx.x;
  const int64_t first = tile * a.tile;
  const int n = (int)(a.M - first < a.tile ? a.M - first : a.tile);  // at most 62
  const int lane = threadIdx.x;
  // lane i holds the key before, at (1..n) and after the tile's tokens
  const int64_t at = first + lane - 1;
  const int32_t keys = at >= 0 && at < a.M && lane < n + 2 ? a.key[at] : -1;
  const int32_t poss = lane < n ? a.pos[first + lane] : 0;
  const int c = (blockIdx.y * 64 + lane) * 8;
  const int left = a.D - c < 0 ? 0 : a.D - c < 8 ? a.D - c : 8;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  constexpr int U = 8;
  for (int i0 = 0; i0 < n; i0 += U) {
    Vec<YB, 8> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r[u] = zero_vec<YB, 8>();
      const int i = i0 + u;
      if (i >= n || __builtin_amdgcn_readlane(keys, i + 1) == kDead) continue;
      const elem_t<YB>* p = static_cast<const elem_t<YB>*>(a.dY) +
                            (int64_t)__builtin_amdgcn_readlane(poss, i) * a.ldy + c;
      if (left == 8)
        r[u] = load_vec<YB, 8>(p);
      else if (left > 0)
        r[u] = load_part<YB, 8>(p, left);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      if (i >= n) break;
      const int32_t id = __builtin_amdgcn_readlane(keys, i + 1);
      if (id == kDead) break;  // sorted last: nothing follows
      float v[8];
      to_float<YB, 8>(r[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += v[e];
      const bool ends = __builtin_amdgcn_readlane(keys, i + 2) != id;
      if (!ends && i + 1 < n) continue;
      const bool begins = __builtin_amdgcn_readlane(keys, 0) != id;
      if (left > 0) {
        if (ends && begins) {
          write_row<GB>(a, id, c, left, acc);
        } else {
          // a sum that covers the whole tile counts as one that began before it
          float* p = a.part + (tile * 2 + (begins ? 1 : 0)) * a.ldp + c;
          store_vec<false, 8>(p, acc);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    }
  }
}

// Workgroup (tile, 512 columns): if a sum begins in the tile and passes its
// end, it is this workgroup's. The following tiles' parts are dealt to the
// waves in consecutive ranges, whose sums are added in order.
constexpr int kJoinWaves = 4;

template <bool GB>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_join_kernel(EmbedBwd a, int64_t tiles) {
  __shared__ float join[kJoinWaves][64 * 8];
  const int64_t tile = blockIdx.x;
  const int64_t end = (tile + 1) * a.tile;  // the last tile is not launched: end < M
  const int32_t id = a.key[end - 1];
  if (id == kDead || a.key[end] != id) return;
  if (a.key[tile * a.tile] == id && tile > 0 && a.key[tile * a.tile - 1] == id) return;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  // The tiles after this one that begin with the id.
  int64_t n = 0;
  for (;;) {
    const int64_t f = (tile + 1 + n + lane) * a.tile;
    const uint64_t yes = __ballot(f < a.M && a.key[f < a.M ? f : 0] == id);
    const int run = yes == ~(uint64_t)0 ? 64 : __builtin_ctzll(~yes);
    n += run;
    if (run < 64) break;
  }
  const int c = (blockIdx.y * 64 + lane) * 8;
  const int left = a.D - c < 0 ? 0 : a.D - c < 8 ? a.D - c : 8;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  const int64_t per = (n + kJoinWaves - 1) / kJoinWaves;
  const int64_t stop = (wave + 1) * per < n ? (wave + 1) * per : n;
  if (left > 0) {
#pragma unroll 4
    for (int64_t i = wave * per; i < stop; ++i) {
      float v[8];
      to_float<false, 8>(load_vec<false, 8>(a.part + (tile + 1 + i) * 2 * a.ldp + c), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += v[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) join[wave][lane * 8 + e] = acc[e];
  __syncthreads();
  if (wave || !left) return;
  float v[8];
  to_float<false, 8>(load_vec<false, 8>(a.part + (tile * 2 + 1) * a.ldp + c), v);
  for (int w = 0; w < kJoinWaves; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += join[w][lane * 8 + e];
  write_row<GB>(a, id, c, left, v);
}

template <bool WB, bool OB>
hipError_t fwd(const EmbedFwd& a, hipStream_t st) {
  const int64_t rows = a.D > 1024 ? 1 : 4;
  const int64_t blocks = (a.M + rows - 1) / rows;
  const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
  if (a.D > 1024)
    hipLaunchKernelGGL((embed_fwd_kernel<WB, OB, 256>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((embed_fwd_kernel<WB, OB, 64>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

template <bool YB, bool GB>
hipError_t sums(const EmbedBwd& a, hipStream_t st) {
  const unsigned tiles = (unsigned)((a.M + a.tile - 1) / a.tile);
  const unsigned cols = (unsigned)((a.D + 511) / 512);
  hipLaunchKernelGGL((embed_sum_kernel<YB, GB>), dim3(tiles, cols), dim3(64), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && tiles > 1) {
    hipLaunchKernelGGL((embed_join_kernel<GB>), dim3(tiles - 1, cols), dim3(64 * kJoinWaves), 0, st,
                       a, (int64_t)tiles);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

int embed_tile(int64_t M) { return M <= 512 ? 4 : M <= 4096 ? 16 : 32; }

hipError_t launch_embed_fwd(const void* W, int64_t ldw, bool w_bf16, int64_t V, int64_t D,
                            const void* ids, bool ids64, int64_t M, float scale, void* out,
                            int64_t ldo, bool out_bf16, hipStream_t st) {
  const EmbedFwd a{W, ldw, V, (int)D, ids, ids64, M, scale, out, ldo};
  if (w_bf16) return out_bf16 ? fwd<true, true>(a, st) : fwd<true, false>(a, st);
  return out_bf16 ? fwd<false, true>(a, st) : fwd<false, false>(a, st);
}

hipError_t launch_embed_bwd(const void* dY, int64_t ldy, bool dy_bf16, const void* ids, bool ids64,
                            int64_t M, int64_t V, int64_t D, float scale, void* dW, bool grad_bf16,
                            bool accumulate, int32_t* sorted, float* part, hipStream_t st) {
  const int runs = (int)((M + kRun - 1) / kRun);
  const int64_t Mp = (M + 63) / 64 * 64;
  int32_t *key = sorted, *pos = sorted + Mp;
  const int64_t halves = accumulate ? 0 : V * D * (grad_bf16 ? 1 : 2);
  const int64_t fills = (halves / 8 + 4095) / 4096;
  const int64_t fill = halves ? (fills < 1 ? 1 : fills > 2048 ? 2048 : fills) : 0;
  if (runs + fill > 0) {
    hipLaunchKernelGGL(embed_sort_kernel, dim3((unsigned)(runs + fill)), dim3(1024), 0, st, ids,
                       ids64, M, V, runs, key, pos, static_cast<u32x4_t*>(dW), halves);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (M == 0) return hipSuccess;
  if (runs > 1) {
    hipLaunchKernelGGL(embed_rank_kernel, dim3((unsigned)((M + 255) / 256)), dim3(256), 0, st, key,
                       pos, M, runs, sorted + 2 * Mp, sorted + 3 * Mp);
    if (const hipError_t e = hipGetLastError()) return e;
    key = sorted + 2 * Mp;
    pos = sorted + 3 * Mp;
  }
  const EmbedBwd a{dY, ldy, M, (int)D, scale, accumulate, dW, key, pos, part,
                   (int)((D + 7) / 8 * 8), embed_tile(M)};
  if (dy_bf16) return grad_bf16 ? sums<true, true>(a, st) : sums<true, false>(a, st);
  return grad_bf16 ? sums<false, true>(a, st) : sums<false, false>(a, st);
}

}  // namespace qlora
