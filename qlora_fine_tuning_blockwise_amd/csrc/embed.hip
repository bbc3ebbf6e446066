// Token embedding on gfx950: the scaled lookup and its dense gradient.
//
//   out[m] = scale W[id_m];   dW[v] = scale * sum over m with id_m = v of dY[m]
//
// An id outside of [0, V) has no row of the table: its output row is zero and
// its dY row is not read.
//
// The gradient sorts the tokens by id (ties by position), so that each table
// row is one sum in token order, whatever the launch: no floating-point
// atomics, the same bits every time.
//   1. Small workgroups count for each token how many tokens of its run come
//      before it, which is its place in the run. Beside them dW is filled with
//      zeros, which is most of the call's traffic.
//   2. With more than one run, a token's place among all is its place in its
//      own run plus, by binary search, the count of smaller keys in the others.
//      Most of the fill then runs beside this launch.
//   3. The sorted tokens are cut into tiles. A wave adds one tile's rows over
//      64 vectors of columns in fp32 and writes each id whose tokens all lie in
//      the tile; a sum that passes a tile's border goes to the workspace, and
//      the tile in which it begins is noted in a list.
//   4. Workgroups take the list's sums and collect their parts in tile order.
#include "rows.h"

namespace qlora {
namespace {

constexpr int32_t kDead = 0x7fffffff;  // key of an id outside of the table: sorted last

// Tokens of a run. The count compares each token with its run, the search
// walks through every other run: up to kMaxRun tokens are one run (the search
// is a launch of 6 us). Measured with runs of 512, 1024 and 2048 tokens: 16000
// tokens of 1024 columns 43.2, 41.5 and 44.0 us; with 1024, 2048 and 4096: 30000
// tokens of 500 columns 57.8, 54.9 and 61.4 us. Every token searches every other
// run, so the search grows with the square of the tokens and is most of the call
// from 65536 on: bf16 rows into 32000 x 1024 fp32, 32768, 65536, 131072, 262144
// and 2^20 tokens: 70, 132, 297, 837 and 9980 us.
constexpr int kMaxRun = 4096;
int run_length(int64_t M) { return M <= kMaxRun ? kMaxRun : M <= 20000 ? 1024 : 2048; }

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

// T threads take a token's row, four vectors each in flight. The copy of 4096
// rows of 4096 bf16 runs at 4.7 TB/s (10.4 us), 8192 rows of 8192 at 4.7 TB/s;
// 64 and 128 threads a row measured the same and 8% slower there.
template <bool WB, bool OB, int T>
__global__ __launch_bounds__(256) void embed_fwd_kernel(EmbedFwd a) {
  constexpr int kRows = 256 / T, E = WB && OB ? 8 : 4, U = 4;
  const int t = threadIdx.x % T;
  const int full = a.D / E, tail = a.D % E;
  for (int64_t m = (int64_t)blockIdx.x * kRows + threadIdx.x / T; m < a.M;
       m += (int64_t)gridDim.x * kRows) {
    const int64_t id = load_index(a.ids, a.ids64, m);
    const bool live = id >= 0 && id < a.V;
    const elem_t<WB>* w = static_cast<const elem_t<WB>*>(a.W) + (live ? id : 0) * a.ldw;
    elem_t<OB>* o = static_cast<elem_t<OB>*>(a.out) + m * a.ldo;
    for (int c0 = t; c0 < full; c0 += U * T) {
      Vec<WB, E> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        r[u] = live && c0 + u * T < full ? load_vec<WB, E>(w + (c0 + u * T) * E) : zero_vec<WB, E>();
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * T < full) {
          float v[E];
          to_float<WB, E>(r[u], v);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = live ? v[e] * a.scale : 0.0f;
          store_vec<OB, E>(o + (c0 + u * T) * E, v);
        }
    }
    if (t < tail) {
      const int c = full * E + t;
      store1<OB>(o + c, live ? load_any(w, WB, c) * a.scale : 0.0f);
    }
  }
}

// ---------------------------------------------------------------- the sort
// The first workgroups order 16 tokens each (sixteen threads a token, each of
// which compares it with every sixteenth group of four of its run's keys); the
// others write zeros over dW or a part of it. The fill is nontemporal: with
// plain stores it leaves the Infinity Cache full of lines that have yet to reach
// memory, and the sums that follow wait for them (4096 tokens, 32000 x 4096
// fp32: the sums take 23 against 13.7 us, the call 115 against 99 us). A
// workgroup writes 4 KB and ends: with a quarter as many, four stores a thread,
// the call takes 101 us, with 8192 and sixteen stores 130 us.
constexpr int kOrderTokens = 16, kOrderThreads = 256;

// The keys of a run's n tokens into LDS, up to the next multiple of four, with
// the loads of eight rounds of the workgroup in flight. What lies behind the
// last token counts as dead: it comes after every token, its place is later.
template <typename T>
__device__ __forceinline__ void stage_keys(const T* ids, int n, int64_t V, int32_t* keys) {
  constexpr int B = 8;
  const int end = (n + 3) / 4 * 4;
  for (int i0 = threadIdx.x; i0 < end; i0 += B * kOrderThreads) {
    T id[B];
#pragma unroll
    for (int b = 0; b < B; ++b) id[b] = i0 + b * kOrderThreads < n ? ids[i0 + b * kOrderThreads] : -1;
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (i0 + b * kOrderThreads < end)
        keys[i0 + b * kOrderThreads] = id[b] >= 0 && id[b] < V ? (int32_t)id[b] : kDead;
  }
}

// Zeros over the sixteen-byte units [first, end) of dW and `tail` two-byte
// units behind them, by `groups` workgroups of which this is number `at`.
struct Fill {
  u32x4_t* dW;
  int64_t first, end;
  int tail;
};
__device__ __forceinline__ void fill_zeros(const Fill& f, int64_t at, int64_t groups) {
  for (int64_t i = f.first + at * kOrderThreads + threadIdx.x; i < f.end; i += groups * kOrderThreads)
    __builtin_nontemporal_store(zero4(), f.dW + i);
  if (at == 0 && (int)threadIdx.x < f.tail)
    reinterpret_cast<uint16_t*>(f.dW + f.end)[threadIdx.x] = 0;
}

__global__ __launch_bounds__(kOrderThreads) void embed_order_kernel(
    const void* ids, bool i64, int64_t M, int64_t V, int run, int orders, int32_t* key, int32_t* pos,
    int32_t* count, Fill fill) {
  __shared__ __align__(16) int32_t keys[kMaxRun];
  const int t = threadIdx.x;
  if ((int)blockIdx.x >= orders) {
    fill_zeros(fill, (int)blockIdx.x - orders, gridDim.x - orders);
    return;
  }
  if (blockIdx.x == 0 && t == 0) *count = 0;  // the list of embed_sum_kernel is empty
  const int64_t token = (int64_t)blockIdx.x * kOrderTokens;  // run is a multiple of kOrderTokens
  const int64_t base = token / run * run;
  const int n = (int)(M - base < run ? M - base : run);
  if (i64)
    stage_keys(static_cast<const int64_t*>(ids) + base, n, V, keys);
  else
    stage_keys(static_cast<const int32_t*>(ids) + base, n, V, keys);
  __syncthreads();
  const int own = (int)(token - base) + t / 16, part = t % 16;
  const bool live = own < n;
  const int32_t k = live ? keys[own] : 0;
  int before = 0;
#pragma unroll 4
  for (int i = part * 4; i < n; i += 64) {
    const u32x4_t q = *reinterpret_cast<const u32x4_t*>(keys + i);
#pragma unroll
    for (int e = 0; e < 4; ++e)  // below k, or its equal at an earlier place
      before += q[e] < (uint32_t)k + (uint32_t)(i + e < own);
  }
#pragma unroll
  for (int m = 1; m < 16; m *= 2) before += __shfl_xor(before, m, 64);
  if (live && part == 0) {
    key[base + before] = k;
    pos[base + before] = (int32_t)(base + own);
  }
}

// The place of each token among all: its place in its run and, for every
// other run, the count of keys before it by binary search. Sixteen lanes work
// on a token, each on four runs at a time, so that the searches' loads fly
// together; they wait more than they move, and the workgroups behind the first
// `ranks` fill dW meanwhile.
constexpr int kRankLanes = 16;

__global__ __launch_bounds__(256) void embed_rank_kernel(const int32_t* __restrict__ key,
                                                         const int32_t* __restrict__ pos,
                                                         int64_t M, int run, int runs, int ranks,
                                                         int32_t* __restrict__ key_out,
                                                         int32_t* __restrict__ pos_out, Fill fill) {
  if ((int)blockIdx.x >= ranks) {
    fill_zeros(fill, (int)blockIdx.x - ranks, gridDim.x - ranks);
    return;
  }
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / kRankLanes;
  const int part = threadIdx.x % kRankLanes;
  const bool live = i < M;
  const int own = live ? (int)(i / run) : 0;
  const int32_t k = live ? key[i] : 0;
  int count = 0;
  constexpr int B = 4;
  for (int r0 = part; live && r0 < runs; r0 += B * kRankLanes) {
    int lo[B], n[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int r = r0 + b * kRankLanes;
      const int64_t left = M - (int64_t)r * run;
      n[b] = r == own || left < 0 ? 0 : left < run ? (int)left : run;
      lo[b] = 0;
    }
    for (int step = run; step > 0; step /= 2)  // run is a power of two
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int at = lo[b] + step, r = r0 + b * kRankLanes;
        if (at > n[b]) continue;
        const int32_t v = key[(int64_t)r * run + at - 1];
        // before k: what is below it, and in an earlier run its equals too
        if (v < k || (r < own && v == k)) lo[b] = at;
      }
#pragma unroll
    for (int b = 0; b < B; ++b) count += lo[b];
  }
#pragma unroll
  for (int m = 1; m < kRankLanes; m *= 2) count += __shfl_xor(count, m, 64);
  if (live && part == 0) {
    const int64_t rank = i - (int64_t)own * run + count;
    key_out[rank] = k;
    pos_out[rank] = pos[i];
  }
}

// ---------------------------------------------------------------- the sums
// Four, eight and sixteen waves: 16000 tokens, half of them one id, 50, 46 and
// 47 us; 4096 tokens of 4096 columns, many short sums, 128, 130 and 137 us.
constexpr int kJoinWaves = 8;

struct EmbedBwd {
  const void* dY;
  int64_t ldy, M;
  int D;
  float scale;
  bool accumulate;
  void* dW;
  const int32_t* key;
  const int32_t* pos;
  int32_t* list;  // [0]: count, then the tiles in which a sum begins that passes their end
  float* part;    // [tiles][2][ldp]: the sum that began before the tile, the one that passes its end
  int ldp, tile;
};

// The columns of a lane: a whole vector, moved back where it would pass the
// row's end. Its elements below `first` are then another lane's too and are
// read, but only [first, n) are written (an accumulated element is written
// once). n = 0: none; a row shorter than a vector is all of lane 0's.
template <int E>
struct Columns {
  int at, first, n;
  __device__ __forceinline__ Columns(int c, int D) {
    at = c + E <= D || D < E ? c : D - E;
    first = c - at < E ? c - at : E;
    n = c >= D ? 0 : D < E ? D : E;
  }
  __device__ __forceinline__ bool whole() const { return first == 0 && n == E; }
};

template <bool kBf16, int E>
__device__ __forceinline__ Vec<kBf16, E> load_columns(const elem_t<kBf16>* row, const Columns<E>& c,
                                                      int D) {
  if (c.n == 0) return zero_vec<kBf16, E>();
  return D < E ? load_part<kBf16, E>(row + c.at, c.n) : load_vec<kBf16, E>(row + c.at);
}

template <bool kBf16, int E>
__device__ __forceinline__ void store_columns(elem_t<kBf16>* row, const Columns<E>& c,
                                              const float (&v)[E]) {
  if (c.whole())
    store_vec<kBf16, E>(row + c.at, v);
  else
    store_part<kBf16, E>(row + c.at, v, c.n, c.first);
}

template <bool GB, int E>
__device__ __forceinline__ void write_row(const EmbedBwd& a, int32_t id, const Columns<E>& c,
                                          const float (&acc)[E]) {
  elem_t<GB>* p = static_cast<elem_t<GB>*>(a.dW) + (int64_t)id * a.D;
  float v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = acc[e] * a.scale;
  if (a.accumulate) {
    float old[E];
    to_float<GB, E>(load_columns<GB, E>(p, c, a.D), old);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] += old[e];
  }
  store_columns<GB, E>(p, c, v);
}

// Wave (64 E columns, tile). The loads of kRows rows fly together.
template <bool YB, bool GB>
__global__ __launch_bounds__(64) void embed_sum_kernel(EmbedBwd a) {
  constexpr int E = YB && GB ? 8 : 4, kRows = 8;
  const int64_t tile = blockIdx.y;
  const int64_t begin = tile * a.tile;
  const int lane = threadIdx.x;
  // Lane i < n holds token i of the tile and its key; `before` and `after` are
  // the keys next to the tile.
  const int size = (int)(a.M - begin < a.tile ? a.M - begin : a.tile);
  const int32_t key = lane < size ? a.key[begin + lane] : kDead;
  const int32_t pos = lane < size ? a.pos[begin + lane] : 0;
  const int32_t before = tile > 0 ? a.key[begin - 1] : -1;
  const int32_t after = begin + size < a.M ? a.key[begin + size] : -1;
  const int n = __popcll(__ballot(key != kDead));  // the dead come last
  if (n == 0) return;
  const int32_t next = __shfl_down(key, 1);
  // bit i: the sum that token i belongs to ends with it
  const uint64_t ends = __ballot(lane < n && (lane + 1 < size ? next : after) != key);
  bool open = __builtin_amdgcn_readfirstlane(key) == before;  // the sum began before the tile
  const Columns<E> c(((int)blockIdx.x * 64 + lane) * E, a.D);
  const elem_t<YB>* dY = static_cast<const elem_t<YB>*>(a.dY);
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  for (int i0 = 0; i0 < n; i0 += kRows) {
    Vec<YB, E> r[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {  // behind the last token its row again
      const int i = i0 + u < n ? i0 + u : n - 1;
      r[u] = load_columns<YB, E>(dY + (int64_t)__builtin_amdgcn_readlane(pos, i) * a.ldy, c, a.D);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = i0 + u;
      if (i >= n) break;
      float v[E];
      to_float<YB, E>(r[u], v);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += v[e];
      const bool end = ends >> i & 1;
      if (!end && i + 1 < size) continue;
      if (end && !open) {
        if (c.n) write_row<GB, E>(a, __builtin_amdgcn_readlane(key, i), c, acc);
      } else {
        // a sum that covers the whole tile counts as one that began before it
        if (c.n) store_columns<false, E>(a.part + (tile * 2 + (open ? 0 : 1)) * a.ldp, c, acc);
        if (!open && blockIdx.x == 0 && lane == 0)
          a.list[1 + atomicAdd(a.list, 1)] = (int32_t)tile;  // its order does not matter
      }
      open = false;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    }
  }
}

// Workgroup (256 columns, some of the list): a sum that begins in a tile and
// passes its end. The following tiles' parts are dealt to the waves in
// consecutive ranges, whose sums are added in order.
template <bool GB>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_join_kernel(EmbedBwd a) {
  __shared__ float join[kJoinWaves][64 * 4];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int col = ((int)blockIdx.x * 64 + lane) * 4;  // the workspace's rows are whole vectors
  const Columns<4> c(col, a.D);
  const int sums = a.list[0];
  for (int at = blockIdx.y; at < sums; at += gridDim.y) {
    const int64_t tile = a.list[1 + at];
    const int32_t id = a.key[(tile + 1) * a.tile - 1];
    // The tiles after this one that begin with the id.
    int64_t n = 0;
    for (;;) {
      const int64_t f = (tile + 1 + n + lane) * a.tile;
      const uint64_t yes = __ballot(f < a.M && a.key[f < a.M ? f : 0] == id);
      const int run = yes == ~(uint64_t)0 ? 64 : __builtin_ctzll(~yes);
      n += run;
      if (run < 64) break;
    }
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t per = (n + kJoinWaves - 1) / kJoinWaves;
    const int64_t stop = (wave + 1) * per < n ? (wave + 1) * per : n;
    if (c.n) {
      const float* p = a.part + (tile + 1) * 2 * a.ldp + c.at;
      for (int64_t i0 = wave * per; i0 < stop; i0 += 8) {
        Vec<false, 4> r[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          r[u] = i0 + u < stop ? load_vec<false, 4>(p + (i0 + u) * 2 * a.ldp) : zero_vec<false, 4>();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          float v[4];
          to_float<false, 4>(r[u], v);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] += v[e];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) join[wave][lane * 4 + e] = acc[e];
    __syncthreads();
    if (wave == 0 && c.n) {
      float v[4];
      to_float<false, 4>(load_vec<false, 4>(a.part + (tile * 2 + 1) * a.ldp + c.at), v);
      for (int w = 0; w < kJoinWaves; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += join[w][lane * 4 + e];
      write_row<GB, 4>(a, id, c, v);
    }
    __syncthreads();  // `join` is written anew for the next sum
  }
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

// At most 2^20 tokens (QLORA_MAX_SORTED): 2^15 tiles, within a grid's second
// dimension.
template <bool YB, bool GB>
hipError_t sums(const EmbedBwd& a, hipStream_t st) {
  const unsigned tiles = (unsigned)((a.M + a.tile - 1) / a.tile);
  constexpr int kCols = 64 * (YB && GB ? 8 : 4);
  hipLaunchKernelGGL((embed_sum_kernel<YB, GB>), dim3((unsigned)((a.D + kCols - 1) / kCols), tiles),
                     dim3(64), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && tiles > 1) {
    hipLaunchKernelGGL((embed_join_kernel<GB>),
                       dim3((unsigned)((a.D + 255) / 256), tiles < 256 ? tiles : 256),
                       dim3(64 * kJoinWaves), 0, st, a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

// Tokens of a tile (a wave's lanes hold at most 64). Up to 32 tokens are
// one tile, so that nothing is left to join (20 tokens of 4096 columns: 14.3
// against 16.8 us); above, shorter tiles give more waves and longer ones fewer
// parts (tiles of 8, 16 and 32: 4096 x 256 24.8, 24.1 and 27.6 us, 16000 x 1024
// 54, 46 and 44 us, 32768 x 2048 109, 98 and 96 us; by the count of waves
// instead, 16000 x 64 would take 36 us with tiles of 8 against 30 us).
int embed_tile(int64_t M) { return M <= 32 ? 32 : M <= 4096 ? 16 : 32; }

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
  const int run = run_length(M);
  const int runs = (int)((M + run - 1) / run);
  const int64_t Mp = (M + 63) / 64 * 64;
  int32_t *key = sorted, *pos = sorted + Mp, *list = sorted + 4 * Mp;
  const int64_t halves = accumulate ? 0 : V * D * (grad_bf16 ? 1 : 2), quads = halves / 8;
  // With a search to come, the count takes a quarter of the fill and the search
  // the rest: a quarter, half, three quarters and all beside the count take 41.5,
  // 41.9, 43.7 and 45.3 us on 16000 tokens of 1024 columns (65 MB of bf16), 79.9,
  // 79.9, 80.5 and 85.6 us on 16384 of 2048 (262 MB of fp32).
  const int64_t split = runs > 1 ? quads / 4 : quads;
  const Fill before{static_cast<u32x4_t*>(dW), 0, split, runs > 1 ? 0 : (int)(halves % 8)};
  const Fill beside{static_cast<u32x4_t*>(dW), split, quads, (int)(halves % 8)};
  const auto groups = [](const Fill& f) {
    const int64_t n = (f.end - f.first + kOrderThreads - 1) / kOrderThreads;
    return n < 1 ? (int64_t)(f.tail > 0) : n > (1 << 20) ? (int64_t)(1 << 20) : n;
  };
  const int orders = (int)((M + kOrderTokens - 1) / kOrderTokens);
  const int64_t fill = groups(before);
  if (orders + fill > 0) {
    hipLaunchKernelGGL(embed_order_kernel, dim3((unsigned)(orders + fill)), dim3(kOrderThreads), 0,
                       st, ids, ids64, M, V, run, orders, key, pos, list, before);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (M == 0) return hipSuccess;
  if (runs > 1) {
    const int ranks = (int)((M * kRankLanes + 255) / 256);
    hipLaunchKernelGGL(embed_rank_kernel, dim3((unsigned)(ranks + groups(beside))), dim3(256), 0, st,
                       key, pos, M, run, runs, ranks, sorted + 2 * Mp, sorted + 3 * Mp, beside);
    if (const hipError_t e = hipGetLastError()) return e;
    key = sorted + 2 * Mp;
    pos = sorted + 3 * Mp;
  }
  const EmbedBwd a{dY, ldy, M, (int)D, scale, accumulate, dW, key, pos, list, part,
                   (int)((D + 7) / 8 * 8), embed_tile(M)};
  if (dy_bf16) return grad_bf16 ? sums<true, true>(a, st) : sums<true, false>(a, st);
  return grad_bf16 ? sums<false, true>(a, st) : sums<false, false>(a, st);
}

}  // namespace qlora
