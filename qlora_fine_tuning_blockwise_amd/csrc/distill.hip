// Distillation from a teacher's top logits on gfx950: the divergence of the
// student's distribution from the teacher's, and its gradient.
//
// For a row with student logits z[V], teacher entries (id_j, t_j), j < k, and
// temperature T, the entries with id_j in [0, V) and t_j > -inf are live, and
//   p_j  = exp(t_j / T) / sum over live entries       (0 for the others)
//   m    = max z,  L = log sum_v exp((z_v - m) / T)
//   loss = T^2 sum_j p_j (log p_j - ((z_{id_j} - m) / T - L))
//   dz_v = dloss T (exp((z_v - m) / T - L) - sum over j with id_j = v of p_j)
// A row with no live entry has loss 0 and a zero gradient, as has one with
// dloss = 0; their logits are not read. Entries that name the same id add.
//
// m and L are kept apart: their sum would absorb L where every logit is
// large. The difference z - m is formed before the scaling, so a row of
// the type's lowest values is a uniform distribution and not a NaN.
//
// The forward reads each logit once: a lane keeps a running maximum and the
// sum of exponentials taken from it, and joins 32 logits at a time. The
// backward streams the row and then rewrites the few entries the teacher
// names. Waves work alone (no barriers in the streams): each reads the
// teacher's entries itself and, in the backward, rewrites those whose logits it
// has written. The logits pass through once, so they are read and their
// gradients written with the nontemporal hint (a reader of the gradients that
// follows gains too from 131 MB on: call and reader 93 against 101 us; at 42 MB
// it loses, 36 against 33 us).
//
// Memory bounds both on long rows: the forward's pass over 2048 x 128000 bf16
// runs at 6.7 TB/s (7.0 TB/s is what reading alone reaches here). On short rows
// and few rows the chain of dependent loads does. Since every wave of every
// piece loads all of a row's entries, many of them cost time: with k = 64, 256
// and 1024 entries 512 x 32000 bf16 takes 10.4, 13.0 and 27.8 us forward and
// 16.8, 21.6 and 60 us backward, 2048 x 128000 89, 98 and 226 us and 175, 189 and
// 414 us.
#include "rows.h"

namespace qlora {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kFwdRound = 8192;  // logits a workgroup holds at once: 32 a thread
// Logits of a workgroup of the backward: 64 a thread of bf16, 16 where fp32
// takes part (2048 x 64000 fp32: 172 us, with 32 a thread 181 us, with 8 218 us).
constexpr int bwd_round(bool bf16) { return (bf16 ? 64 : 16) * kThreads; }
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// s exp(d / T), half = log2(e) / (2 T): the hardware's exponential flushes
// results below 2^-126 to zero, the square of the root keeps them. d = z - m is
// scaled by one product, whose rounding (|d / T| 2^-24 of the result) is all
// that grows with the exponent; the row's exp(-L) is part of s. (As exp(d / T -
// L) the rounding of the larger exponent doubled the error: 333 x 32003, root
// mean square, 8.3 against 3.8 times 2^-24 of a gradient.)
__device__ __forceinline__ float scaled_exp(float s, float d, float half) {
  const float h = exp2_fast(d * half);
  return s * h * h;
}

struct Teacher {
  const void* ids;
  const void* t;
  bool ids64, t_bf16;
  int k;
};

// Orders a wave's LDS accesses of different lanes (they are issued in program
// order; only the compiler must keep it).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The teacher's entries of one row in the wave's LDS: id[j] (-1 where entry j
// is not live) and t[j]. Returns whether any entry is live, the largest live
// t in `top`. With `logit` the student's logits at the live entries as well,
// requested before anything waits for the entries' values.
template <bool ZB>
__device__ __forceinline__ bool teacher_load(const Teacher& a, int64_t row, int64_t V, int lane,
                                             int32_t* id, float* t, float& top,
                                             const elem_t<ZB>* z = nullptr,
                                             float* logit = nullptr) {
  constexpr int kBatch = 4;  // entries of a lane whose loads are in flight together
  float m = -INFINITY;
  bool some = false;
  const int64_t first = row * a.k;
  for (int j0 = lane; j0 < a.k; j0 += 64 * kBatch) {
    int64_t i[kBatch];
    float v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) i[b] = -1, v[b] = 0.0f;
    if (a.ids64) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (j0 + 64 * b < a.k) i[b] = static_cast<const int64_t*>(a.ids)[first + j0 + 64 * b];
    } else {
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (j0 + 64 * b < a.k) i[b] = static_cast<const int32_t*>(a.ids)[first + j0 + 64 * b];
    }
    if (a.t_bf16) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (j0 + 64 * b < a.k) v[b] = load_any(a.t, true, first + j0 + 64 * b);
    } else {
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (j0 + 64 * b < a.k) v[b] = load_any(a.t, false, first + j0 + 64 * b);
    }
    float zb[kBatch];
    if (logit) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        zb[b] = i[b] >= 0 && i[b] < V ? load_any(z, ZB, i[b]) : 0.0f;
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const bool live = i[b] >= 0 && i[b] < V && !(v[b] == -INFINITY);  // a NaN is live and spreads
      if (j0 + 64 * b < a.k) {
        id[j0 + 64 * b] = live ? (int32_t)i[b] : -1;
        t[j0 + 64 * b] = v[b];
        if (logit) logit[j0 + 64 * b] = zb[b];
      }
      some |= live;
      if (live) m = fmaxf(m, v[b]);
    }
  }
  if (!__ballot(some)) return false;
  m = wave_reduce(m, OpMax());
  top = m == -INFINITY ? 0.0f : m;  // every live entry is a NaN
  return true;
}

// Sum over the live entries of exp((t - top) / T). The probabilities are these
// exponentials over it, not exponentials of their logarithms: they then sum to
// one but for their last roundings (2048 x 128000: the losses' error is 1.7
// times 2^-24 instead of 4.3, root mean square).
__device__ __forceinline__ float teacher_sum(int k, int lane, const int32_t* id, const float* t,
                                             float top, float invT) {
  float s = 0.0f;
  for (int j = lane; j < k; j += 64) s += id[j] < 0 ? 0.0f : expf((t[j] - top) * invT);
  return wave_reduce(s, OpSum());
}

// A maximum and the sum of exponentials taken from it; from 0 where the
// maximum is -inf, so that a part of -inf alone adds 0.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
  MaxSum r;
  r.m = fmaxf(a.m, b.m);
  const float base = finite_base(r.m);
  // an empty side has s = 0 and m = -inf: its factor is 0 or 1
  r.s = a.s * exp2_fast((a.m - base) * c) + b.s * exp2_fast((b.m - base) * c);
  return r;
}

__device__ __forceinline__ MaxSum wave_join(MaxSum a, float c) {
  MaxSum r;
  r.m = wave_reduce(a.m, OpMax());
  r.s = wave_reduce(a.s * exp2_fast((a.m - finite_base(r.m)) * c), OpSum());
  return r;
}

// U vectors of logits into the pair. -inf adds nothing: it fills the places
// of a vector that lie outside of the row.
template <bool ZB, int E, int U>
__device__ __forceinline__ void take(MaxSum& a, const Vec<ZB, E> (&q)[U], float c,
                                     float limit) {
  float v[U][E];
  float m = a.m;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    to_float<ZB, E>(q[u], v[u]);
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, v[u][e]);
  }
  const float base = finite_base(m);
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) s[u] = 0.0f;
  float fix = 1.0f;
  if (__builtin_fabsf(base) <= limit) {  // |base c| <= 2^20
    const float bc = base * c;
    // (v - base) c as one operation: v c - base c, whose second term is rounded
    // alike for all of them, by 2^-4 at most; the rounding is taken out of the
    // sum.
    fix = exp2_fast(-fmaf(base, c, -bc));
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) s[u] += exp2_fast(fmaf(v[u][e], c, -bc));
  } else {  // base c is large against its rounding, or not finite
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) s[u] += exp2_fast((v[u][e] - base) * c);
  }
#pragma unroll
  for (int u = 1; u < U; ++u) s[0] += s[u];
  a.s = fmaf(a.s, exp2_fast((a.m - base) * c), fix * s[0]);
  a.m = m;
}

// How a row is dealt out. Its logits are taken from `origin` <= 0 on, the
// place of the 128-byte line in which the row begins, so that every access of
// a wave but a row's first and last covers whole lines; a piece is a run of
// rounds, and in a round thread i of the workgroup holds the vectors at
// (u kThreads + i) E, u < U.
template <bool kBf16>
__device__ __forceinline__ int row_origin(const void* row) {
  constexpr uintptr_t kSize = kBf16 ? 2 : 4;
  return -(int)((reinterpret_cast<uintptr_t>(row) & 127) / kSize);
}

template <bool ZB, int E, int U>
__device__ __forceinline__ void load_round(const elem_t<ZB>* z, int64_t at, Vec<ZB, E> (&q)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) q[u] = load_vec<ZB, E, true>(z + at + u * kThreads * E);
}

// A round that leaves [0, V): the logits [first, n) of each vector.
template <bool ZB, int E, int U>
__device__ __forceinline__ void load_ends(const elem_t<ZB>* z, int64_t at, int64_t V,
                                          Vec<ZB, E> (&q)[U], int (&first)[U], int (&n)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t v = at + u * kThreads * E;
    n[u] = count_below<E>(v, V);
    first[u] = v >= 0 ? 0 : v <= -E ? E : (int)-v;
    q[u] = first[u] == 0 && n[u] == E ? load_vec<ZB, E, true>(z + v) : fill_vec<ZB, E, kNegInf>();
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (first[u] < n[u] && (first[u] > 0 || n[u] < E))
      q[u] = load_part<ZB, E, kNegInf>(z + at + u * kThreads * E, n[u], first[u]);
}

struct DistillFwd {
  const void* z;
  int64_t ldz, M, V;
  Teacher teacher;
  float T, invT;
  float c, limit;  // log2(e) / T; 2^20 / c
  float* loss;
  float* stats;
  MaxSum* part;  // [M][splits][kWaves]
  int splits;
  int rounds;  // of a split
};

// loss and statistics of a row from its joined pair, by one wave.
__device__ __forceinline__ void finish_row(const DistillFwd& a, int64_t row, int lane, MaxSum r,
                                           const int32_t* id, const float* t, const float* logit,
                                           float top) {
  const float L = logf(r.s);
  const float sum = teacher_sum(a.teacher.k, lane, id, t, top, a.invT);
  const float logsum = logf(sum);
  float s = 0.0f;
  for (int j = lane; j < a.teacher.k; j += 64) {
    if (id[j] < 0) continue;
    const float at = (t[j] - top) * a.invT;
    const float p = expf(at) / sum;
    if (p != 0.0f) s += p * (at - logsum - ((logit[j] - r.m) * a.invT - L));
  }
  s = wave_reduce(s, OpSum());
  if (lane == 0) {
    a.loss[row] = a.T * a.T * s;
    if (a.stats) {
      a.stats[row] = r.m;
      a.stats[a.M + row] = L;
    }
  }
}

__device__ __forceinline__ void empty_row(const DistillFwd& a, int64_t row) {
  a.loss[row] = 0.0f;
  if (a.stats) a.stats[row] = a.stats[a.M + row] = 0.0f;
}

// Workgroup (row, split): its part of the row. With one split its first wave
// also finishes the row; otherwise distill_finish_kernel does.
template <bool ZB>
__global__ __launch_bounds__(kThreads) void distill_fwd_kernel(DistillFwd a) {
  constexpr int E = ZB ? 8 : 4, U = kFwdRound / (kThreads * E);
  extern __shared__ float lds[];  // of each wave: id[k], t[k], the logits at the ids
  __shared__ MaxSum pair[kWaves];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  int32_t* id = reinterpret_cast<int32_t*>(lds) + wave * 3 * a.teacher.k;
  float* t = reinterpret_cast<float*>(id) + a.teacher.k;
  float* logit = t + a.teacher.k;
  const float c = a.c, limit = a.limit;
  for (int64_t item = blockIdx.x; item < a.M * a.splits; item += gridDim.x) {
    const int64_t row = item / a.splits;
    const int split = (int)(item - row * a.splits);
    float top = 0.0f;
    const elem_t<ZB>* z = static_cast<const elem_t<ZB>*>(a.z) + row * a.ldz;
    // every wave finds the same answer: the barriers below are reached by all
    if (!teacher_load<ZB>(a.teacher, row, a.V, lane, id, t, top, z,
                          a.splits == 1 && wave == 0 ? logit : nullptr)) {
      if (threadIdx.x == 0 && split == 0) empty_row(a, row);
      continue;
    }
    const int64_t base = row_origin<ZB>(z) + (int64_t)split * a.rounds * kFwdRound;
    MaxSum r{-INFINITY, 0.0f};
    const auto load = [&](int i, Vec<ZB, E>(&q)[U]) {
      const int64_t at = base + (int64_t)i * kFwdRound;
      if (at >= 0 && at + kFwdRound <= a.V) {
        load_round<ZB, E>(z, at + threadIdx.x * E, q);
      } else {
        int first[U], n[U];
        load_ends<ZB, E>(z, at + threadIdx.x * E, a.V, q, first, n);
      }
    };
    Vec<ZB, E> q[U];
    for (int i = 0; i < a.rounds; ++i) {
      load(i, q);
      take<ZB, E, U>(r, q, c, limit);
    }
    r = wave_join(r, c);
    if (a.splits > 1) {
      if (lane == 0) a.part[item * kWaves + wave] = r;
      continue;
    }
    if (lane == 0) pair[wave] = r;
    __syncthreads();
    if (wave == 0) {
      r = pair[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) r = join(r, pair[w], c);
      finish_row(a, row, lane, r, id, t, logit, top);
    }
    __syncthreads();  // `pair` is written anew for the next item
  }
}

template <bool ZB>
__global__ __launch_bounds__(64) void distill_finish_kernel(DistillFwd a) {
  extern __shared__ float lds[];
  const int lane = threadIdx.x;
  int32_t* id = reinterpret_cast<int32_t*>(lds);
  float *t = lds + a.teacher.k, *logit = t + a.teacher.k;
  const float c = a.c;
  const int parts = a.splits * kWaves;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const elem_t<ZB>* z = static_cast<const elem_t<ZB>*>(a.z) + row * a.ldz;
    // an empty row's parts were not written; they are not used
    MaxSum r = lane < parts ? a.part[row * parts + lane] : MaxSum{-INFINITY, 0.0f};
    float top = 0.0f;
    if (!teacher_load<ZB>(a.teacher, row, a.V, lane, id, t, top, z, logit)) continue;
    for (int i = lane + 64; i < parts; i += 64) r = join(r, a.part[row * parts + i], c);
    finish_row(a, row, lane, wave_join(r, c), id, t, logit, top);
  }
}

struct DistillBwd {
  const void* z;
  int64_t ldz, M, V;
  Teacher teacher;
  float T, invT, half;  // half: log2(e) / (2 T)
  const float* stats;
  const float* dloss;
  void* dz;
  int64_t ldg;
  int chunks;
};

// Workgroup (row, chunk): one round of the row. Rounds of 32 KB a workgroup,
// all of it in flight at once, measured best: 2048 x 128000 bf16 in 177 us
// (5.9 TB/s of the 6.5 TB/s that a copy in the same pattern reaches), 193 us
// with two rounds a workgroup, 190 us with rounds of half the size; without
// the nontemporal hint 200 us, and on rows that do not begin on a line (V =
// 128008) 208 us where the rounds begin with the row instead of its line.
template <bool ZB, bool GB>
__global__ __launch_bounds__(kThreads) void distill_bwd_kernel(DistillBwd a) {
  constexpr int E = ZB && GB ? 8 : 4, kRound = bwd_round(ZB && GB), U = kRound / (kThreads * E);
  extern __shared__ float lds[];  // of each wave: id[k], t[k], then its own entries' id and p
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int k = a.teacher.k;
  int32_t* id = reinterpret_cast<int32_t*>(lds) + wave * 2 * k;
  float* t = reinterpret_cast<float*>(id) + k;
  for (int64_t item = blockIdx.x; item < a.M * a.chunks; item += gridDim.x) {
    const int64_t row = item / a.chunks;
    const int chunk = (int)(item - row * a.chunks);
    const elem_t<ZB>* z = static_cast<const elem_t<ZB>*>(a.z) + row * a.ldz;
    elem_t<GB>* g = static_cast<elem_t<GB>*>(a.dz) + row * a.ldg;
    const float dl = a.dloss[row];
    float top = 0.0f;
    const int64_t begin = row_origin<GB>(g) + (int64_t)chunk * kRound;
    const int64_t at = begin + threadIdx.x * E;
    if (dl == 0.0f || !teacher_load<ZB>(a.teacher, row, a.V, lane, id, t, top)) {
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = at + u * kThreads * E;
        const int n = count_below<E>(i, a.V);
        if (i >= 0 && n == E)
          store_vec<GB, E, true>(g + i, v);
        else if (i > -E && n > 0)
          store_part<GB, E>(g + i, v, n, i < 0 ? (int)-i : 0);
      }
      continue;
    }
    const float scale = dl * a.T;
    const float m = a.stats[row], norm = expf(-a.stats[a.M + row]);
    const float factor = scale * norm;
    Vec<ZB, E> q[U];
    if (begin >= 0 && begin + kRound <= a.V) {
      load_round<ZB, E>(z, at, q);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[E];
        to_float<ZB, E>(q[u], v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = scaled_exp(factor, v[e] - m, a.half);
        store_vec<GB, E, true>(g + at + u * kThreads * E, v);
      }
    } else {
      int first[U], n[U];
      load_ends<ZB, E>(z, at, a.V, q, first, n);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[E];
        to_float<ZB, E>(q[u], v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = scaled_exp(factor, v[e] - m, a.half);
        if (first[u] == 0 && n[u] == E)
          store_vec<GB, E, true>(g + at + u * kThreads * E, v);
        else if (first[u] < n[u])
          store_part<GB, E>(g + at + u * kThreads * E, v, n[u], first[u]);
      }
    }
    const float sum = teacher_sum(k, lane, id, t, top, a.invT);
    // The entries whose logits this wave has written, moved to the front.
    int own = 0;
    for (int j0 = 0; j0 < k; j0 += 64) {
      const int j = j0 + lane;
      const int32_t v = j < k ? id[j] : -1;
      const float p = v < 0 ? 0.0f : expf((t[j] - top) * a.invT) / sum;
      const bool mine = v >= 0 && v >= begin && v < begin + kRound &&
                        ((v - begin) / (64 * E)) % kWaves == wave;
      const uint64_t all = __ballot(mine);
      wave_sync();  // the reads above come before the writes below, which are not past them
      if (mine) {
        const int at = own + __popcll(all & ((1ull << lane) - 1));
        id[at] = v;
        t[at] = p;
      }
      own += __popcll(all);
    }
    wave_sync();  // the list is whole, and the wave's gradients are written before its entries are
    for (int j = lane; j < own; j += 64) {
      const int32_t v = id[j];
      float given = 0.0f;
      bool again = false;
#pragma unroll 8
      for (int i = 0; i < own; ++i) {
        const bool same = id[i] == v;
        given += same ? t[i] : 0.0f;
        again |= same && i < j;
      }
      if (again) continue;  // the first entry of an id writes it
      const float e = scaled_exp(norm, load_any(z, ZB, v) - m, a.half);
      store1<GB>(g + v, scale * (e - given));
    }
    wave_sync();  // the lists are written anew for the next item
  }
}

// A row of V logits as pieces of `rounds` rounds of `round` logits. (A row
// may begin up to a line after its first piece's place.)
struct Pieces {
  int count, rounds;
};

// Forward: up to eight rounds (64K logits) a row is one workgroup's and the
// call is one launch; longer rows are cut into pieces of four rounds, which
// costs the finishing launch but keeps the workgroups short, so that rows
// without a live entry leave no hole at the end. Measured with bf16 logits,
// in one launch against pieces of four rounds: 1 x 64000 10.9 against 14.8 us,
// 2048 x 64000 (fp32) 84.3 against 87.4 us, but 64 x 128000 19.7 against
// 14.9 us; pieces of two, four and eight rounds on 2048 x 128000 with a
// quarter of the rows empty: 76, 69 and 71 us.
Pieces fwd_pieces(int64_t V) {
  const int64_t n = (V + 63 + kFwdRound - 1) / kFwdRound;
  if (n <= 8) return {1, (int)n};
  const int64_t p = (n + 3) / 4;
  return {(int)p, (int)((n + p - 1) / p)};
}

}  // namespace

int distill_parts(int64_t V) {
  const int s = fwd_pieces(V).count;
  return s > 1 ? s * kWaves : 0;
}

hipError_t launch_distill_fwd(const void* z, int64_t ldz, bool z_bf16, int64_t M, int64_t V,
                              const void* ids, bool ids64, const void* t, bool t_bf16, int k,
                              float T, float* loss, float* stats, float* part, hipStream_t st) {
  const Pieces p = fwd_pieces(V);
  const int splits = p.count;
  const float c = 1.0f / T * kLog2e;
  const DistillFwd a{z, ldz, M, V, {ids, t, ids64, t_bf16, k}, T, 1.0f / T, c, 0x1p20f / c, loss,
                     stats, reinterpret_cast<MaxSum*>(part), splits, p.rounds};
  const int64_t items = M * splits;
  const dim3 grid((unsigned)(items < 65536 ? items : 65536)), rows((unsigned)(M < 65536 ? M : 65536));
  const size_t lds = (size_t)k * 12;
  if (z_bf16)
    hipLaunchKernelGGL(distill_fwd_kernel<true>, grid, dim3(kThreads), lds * kWaves, st, a);
  else
    hipLaunchKernelGGL(distill_fwd_kernel<false>, grid, dim3(kThreads), lds * kWaves, st, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && splits > 1) {
    if (z_bf16)
      hipLaunchKernelGGL(distill_finish_kernel<true>, rows, dim3(64), lds, st, a);
    else
      hipLaunchKernelGGL(distill_finish_kernel<false>, rows, dim3(64), lds, st, a);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_distill_bwd(const void* z, int64_t ldz, bool z_bf16, int64_t M, int64_t V,
                              const void* ids, bool ids64, const void* t, bool t_bf16, int k,
                              float T, const float* stats, const float* dloss, void* dz,
                              int64_t ldg, bool g_bf16, hipStream_t st) {
  const int round = bwd_round(z_bf16 && g_bf16);
  const int chunks = (int)((V + 63 + round - 1) / round);
  const DistillBwd a{z, ldz, M, V, {ids, t, ids64, t_bf16, k}, T, 1.0f / T,
                     (float)(0.5 * 1.4426950408889634 / (double)T), stats, dloss, dz, ldg, chunks};
  const int64_t items = M * chunks;
  const dim3 grid((unsigned)(items < 65536 ? items : 65536)), block(kThreads);
  const size_t lds = (size_t)k * 8 * kWaves;
  if (z_bf16 && g_bf16)
    hipLaunchKernelGGL((distill_bwd_kernel<true, true>), grid, block, lds, st, a);
  else if (z_bf16)
    hipLaunchKernelGGL((distill_bwd_kernel<true, false>), grid, block, lds, st, a);
  else if (g_bf16)
    hipLaunchKernelGGL((distill_bwd_kernel<false, true>), grid, block, lds, st, a);
  else
    hipLaunchKernelGGL((distill_bwd_kernel<false, false>), grid, block, lds, st, a);
  return hipGetLastError();
}

}  // namespace qlora
