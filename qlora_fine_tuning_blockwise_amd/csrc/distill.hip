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
// The forward reads each logit once: a thread keeps a running maximum and the
// sum of exponentials taken from it, and joins eight or more logits at a
// time. The backward streams the row and then rewrites the few entries the
// teacher names.
#include <type_traits>

#include "rows.h"

namespace qlora {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

struct Teacher {
  const void* ids;
  const void* t;
  bool ids64, t_bf16;
  int k;
};

// The teacher's distribution of one row in LDS: id[j] (-1 where entry j is
// not live) and p[j]; every thread gets log sum exp((t - top) / T) in `logsum`
// and the top. Returns whether any entry is live. All threads call it; ends
// with a barrier.
__device__ __forceinline__ bool teacher_row(const Teacher& a, int64_t row, int64_t V, float invT,
                                            int32_t* id, float* p, float* red, int& par,
                                            float& top, float& logsum) {
  float m[1] = {-INFINITY};
  bool some = false;
  for (int j = threadIdx.x; j < a.k; j += kThreads) {
    const int64_t i = load_index(a.ids, a.ids64, row * a.k + j);
    const float t = load_any(a.t, a.t_bf16, row * a.k + j);
    const bool live = i >= 0 && i < V && !(t == -INFINITY);  // a NaN is live and spreads
    id[j] = live ? (int32_t)i : -1;
    p[j] = t;
    some |= live;
    if (live) m[0] = fmaxf(m[0], t);
  }
  if (!__syncthreads_or(some)) return false;
  group_reduce<kThreads, 1>(m, red, kWaves, par, OpMax());
  top = m[0] == -INFINITY ? 0.0f : m[0];  // every live entry is a NaN
  float s[1] = {0.0f};
  for (int j = threadIdx.x; j < a.k; j += kThreads) {
    const float e = id[j] < 0 ? 0.0f : expf((p[j] - top) * invT);
    s[0] += e;
  }
  group_reduce<kThreads, 1>(s, red, kWaves, par, OpSum());
  logsum = logf(s[0]);
  return true;
}

// Running maximum and sum of a thread joined with another pair: sums are
// taken from max(m, the lowest finite), so a part of -inf alone adds 0.
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

__device__ __forceinline__ void take(MaxSum& a, const float (&v)[8], int n, float c) {
  float m = a.m;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, e < n ? v[e] : -INFINITY);
  const float base = finite_base(m);
  float s = a.s * exp2_fast((a.m - base) * c);
#pragma unroll
  for (int e = 0; e < 8; ++e) s += e < n ? exp2_fast((v[e] - base) * c) : 0.0f;
  a.m = m;
  a.s = s;
}

// The pair of the whole workgroup, in every thread.
__device__ __forceinline__ MaxSum group_join(MaxSum a, float c, float* red, int& par) {
  float m[1] = {a.m};
  group_reduce<kThreads, 1>(m, red, kWaves, par, OpMax());
  const float base = finite_base(m[0]);
  float s[1] = {a.s * exp2_fast((a.m - base) * c)};
  group_reduce<kThreads, 1>(s, red, kWaves, par, OpSum());
  return MaxSum{m[0], s[0]};
}

struct DistillFwd {
  const void* z;
  int64_t ldz, M, V;
  Teacher teacher;
  float T, invT;
  float* loss;
  float* stats;
  MaxSum* part;  // [M][splits]
  int splits;
  int64_t per;  // logits of a split
};

// loss and statistics of a row from its joined pair.
template <bool ZB>
__device__ __forceinline__ void finish_row(const DistillFwd& a, int64_t row, MaxSum r,
                                           const int32_t* id, const float* t, float top,
                                           float logsum, float* red, int& par) {
  const float L = logf(r.s);
  float s[1] = {0.0f};
  for (int j = threadIdx.x; j < a.teacher.k; j += kThreads) {
    if (id[j] < 0) continue;
    const float logp = (t[j] - top) * a.invT - logsum;
    const float p = expf(logp);
    const float z = load_any(a.z, ZB, row * a.ldz + id[j]);
    if (p != 0.0f) s[0] += p * (logp - ((z - r.m) * a.invT - L));
  }
  group_reduce<kThreads, 1>(s, red, kWaves, par, OpSum());
  if (threadIdx.x == 0) {
    a.loss[row] = a.T * a.T * s[0];
    if (a.stats) {
      a.stats[row] = r.m;
      a.stats[a.M + row] = L;
    }
  }
}

// Workgroup (row, split): its part of the row. With one split it also
// finishes the row; otherwise distill_finish_kernel does.
template <bool ZB>
__global__ __launch_bounds__(kThreads) void distill_fwd_kernel(DistillFwd a) {
  extern __shared__ float lds[];  // id[k], t[k]
  __shared__ float red[2 * kWaves];
  int32_t* id = reinterpret_cast<int32_t*>(lds);
  float* t = lds + a.teacher.k;
  int par = 0;
  const float c = a.invT * kLog2e;
  for (int64_t item = blockIdx.x; item < a.M * a.splits; item += gridDim.x) {
    const int64_t row = item / a.splits;
    const int split = (int)(item % a.splits);
    float top = 0.0f, logsum = 0.0f;
    if (!teacher_row(a.teacher, row, a.V, a.invT, id, t, red, par, top, logsum)) {
      if (threadIdx.x == 0 && split == 0) {
        a.loss[row] = 0.0f;
        if (a.stats) a.stats[row] = a.stats[a.M + row] = 0.0f;
      }
      continue;
    }
    const elem_t<ZB>* z = static_cast<const elem_t<ZB>*>(a.z) + row * a.ldz;
    const int64_t from = split * a.per, to = from + a.per < a.V ? from + a.per : a.V;
    MaxSum r{-INFINITY, 0.0f};
    constexpr int U = 4;
    for (int64_t v0 = from + threadIdx.x * 8; v0 < to; v0 += U * kThreads * 8) {
      Row8<ZB> q[U];
      int n[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t left = to - (v0 + u * kThreads * 8);
        n[u] = left >= 8 ? 8 : left < 0 ? 0 : (int)left;
        q[u] = zero8<ZB>();
        if (n[u] == 8)
          q[u] = load8<ZB>(z + v0 + u * kThreads * 8);
        else if (n[u] > 0)
          q[u] = load8_part<ZB>(z + v0 + u * kThreads * 8, n[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[8];
        to_float<ZB>(q[u], v);
        if (n[u] > 0) take(r, v, n[u], c);
      }
    }
    r = group_join(r, c, red, par);
    if (a.splits == 1)
      finish_row<ZB>(a, row, r, id, t, top, logsum, red, par);
    else if (threadIdx.x == 0)
      a.part[item] = r;
    __syncthreads();  // id and t are written anew for the next item
  }
}

template <bool ZB>
__global__ __launch_bounds__(kThreads) void distill_finish_kernel(DistillFwd a) {
  extern __shared__ float lds[];
  __shared__ float red[2 * kWaves];
  int32_t* id = reinterpret_cast<int32_t*>(lds);
  float* t = lds + a.teacher.k;
  int par = 0;
  const float c = a.invT * kLog2e;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    float top = 0.0f, logsum = 0.0f;
    if (!teacher_row(a.teacher, row, a.V, a.invT, id, t, red, par, top, logsum)) continue;
    MaxSum r{-INFINITY, 0.0f};
    for (int i = threadIdx.x; i < a.splits; i += kThreads) r = join(r, a.part[row * a.splits + i], c);
    r = group_join(r, c, red, par);
    finish_row<ZB>(a, row, r, id, t, top, logsum, red, par);
    __syncthreads();
  }
}

struct DistillBwd {
  const void* z;
  int64_t ldz, M, V;
  Teacher teacher;
  float T, invT;
  const float* stats;
  const float* dloss;
  void* dz;
  int64_t ldg;
  int chunks;
  int64_t per;  // logits of a chunk, a multiple of eight
};

template <bool ZB, bool GB>
__global__ __launch_bounds__(kThreads) void distill_bwd_kernel(DistillBwd a) {
  extern __shared__ float lds[];
  __shared__ float red[2 * kWaves];
  int32_t* id = reinterpret_cast<int32_t*>(lds);
  float* p = lds + a.teacher.k;
  int par = 0;
  for (int64_t item = blockIdx.x; item < a.M * a.chunks; item += gridDim.x) {
    const int64_t row = item / a.chunks;
    const int chunk = (int)(item % a.chunks);
    const int64_t from = chunk * a.per, to = from + a.per < a.V ? from + a.per : a.V;
    const elem_t<ZB>* z = static_cast<const elem_t<ZB>*>(a.z) + row * a.ldz;
    elem_t<GB>* g = static_cast<elem_t<GB>*>(a.dz) + row * a.ldg;
    const float dl = a.dloss[row];
    float top = 0.0f, logsum = 0.0f;
    // dl is the row's: all threads take the same side
    if (dl == 0.0f || !teacher_row(a.teacher, row, a.V, a.invT, id, p, red, par, top, logsum)) {
      const float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      for (int64_t v0 = from + threadIdx.x * 8; v0 < to; v0 += kThreads * 8) {
        if (to - v0 >= 8)
          store8<GB>(g + v0, v);
        else
          store8_part<GB>(g + v0, v, (int)(to - v0));
      }
      __syncthreads();
      continue;
    }
    const float scale = dl * a.T;
    const float m = a.stats[row], L = a.stats[a.M + row];
    for (int j = threadIdx.x; j < a.teacher.k; j += kThreads)
      p[j] = id[j] < 0 ? 0.0f : expf((p[j] - top) * a.invT - logsum);
    constexpr int U = 4;
    for (int64_t v0 = from + threadIdx.x * 8; v0 < to; v0 += U * kThreads * 8) {
      Row8<ZB> q[U];
      int n[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t left = to - (v0 + u * kThreads * 8);
        n[u] = left >= 8 ? 8 : left < 0 ? 0 : (int)left;
        q[u] = zero8<ZB>();
        if (n[u] == 8)
          q[u] = load8<ZB>(z + v0 + u * kThreads * 8);
        else if (n[u] > 0)
          q[u] = load8_part<ZB>(z + v0 + u * kThreads * 8, n[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[8];
        to_float<ZB>(q[u], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = scale * exp2_fast(fmaf(v[e] - m, a.invT, -L) * kLog2e);
        if (n[u] == 8)
          store8<GB>(g + v0 + u * kThreads * 8, v);
        else if (n[u] > 0)
          store8_part<GB>(g + v0 + u * kThreads * 8, v, n[u]);
      }
    }
    __syncthreads();  // the row's values are written before the teacher's entries are, and p is whole
    for (int j = threadIdx.x; j < a.teacher.k; j += kThreads) {
      const int32_t v = id[j];
      if (v < from || v >= to) continue;
      float sum = 0.0f;
      bool again = false;
      for (int i = 0; i < a.teacher.k; ++i) {
        const bool same = id[i] == v;
        sum += same ? p[i] : 0.0f;
        again |= same && i < j;
      }
      if (again) continue;  // the first entry of an id writes it
      const float q = exp2_fast(fmaf(load_any(z, ZB, v) - m, a.invT, -L) * kLog2e);
      store1<GB>(g + v, scale * (q - sum));
    }
    __syncthreads();
  }
}

int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }

}  // namespace

int distill_splits(int64_t M, int64_t V) {
  const int64_t want = M > 0 ? 1024 / M : 1, most = (V + 8191) / 8192;
  const int64_t s = want < most ? want : most;
  return (int)(s < 1 ? 1 : s);
}

hipError_t launch_distill_fwd(const void* z, int64_t ldz, bool z_bf16, int64_t M, int64_t V,
                              const void* ids, bool ids64, const void* t, bool t_bf16, int k,
                              float T, float* loss, float* stats, float* part, hipStream_t st) {
  const int splits = distill_splits(M, V);
  const DistillFwd a{z, ldz, M, V, {ids, t, ids64, t_bf16, k}, T, 1.0f / T, loss, stats,
                     reinterpret_cast<MaxSum*>(part), splits, round8((V + splits - 1) / splits)};
  const int64_t items = M * splits;
  const dim3 grid((unsigned)(items < 65536 ? items : 65536)), rows((unsigned)(M < 65536 ? M : 65536));
  const size_t lds = (size_t)k * 8;
  if (z_bf16)
    hipLaunchKernelGGL(distill_fwd_kernel<true>, grid, dim3(kThreads), lds, st, a);
  else
    hipLaunchKernelGGL(distill_fwd_kernel<false>, grid, dim3(kThreads), lds, st, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && splits > 1) {
    if (z_bf16)
      hipLaunchKernelGGL(distill_finish_kernel<true>, rows, dim3(kThreads), lds, st, a);
    else
      hipLaunchKernelGGL(distill_finish_kernel<false>, rows, dim3(kThreads), lds, st, a);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_distill_bwd(const void* z, int64_t ldz, bool z_bf16, int64_t M, int64_t V,
                              const void* ids, bool ids64, const void* t, bool t_bf16, int k,
                              float T, const float* stats, const float* dloss, void* dz,
                              int64_t ldg, bool g_bf16, hipStream_t st) {
  const int chunks = (int)((V + 32767) / 32768);
  const DistillBwd a{z, ldz, M, V, {ids, t, ids64, t_bf16, k}, T, 1.0f / T, stats, dloss, dz, ldg,
                     chunks, round8((V + chunks - 1) / chunks)};
  const int64_t items = M * chunks;
  const dim3 grid((unsigned)(items < 65536 ? items : 65536)), block(kThreads);
  const size_t lds = (size_t)k * 8;
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
