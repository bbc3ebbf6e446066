// Norm of a row, forward and backward, on gfx950: layer norm, and the form
// without the mean (RMS).
//
//   mean = sum x / N (0 for RMS);  rstd = 1 / sqrt(sum (x - mean)^2 / N + eps)
//   y    = (x - mean) rstd gamma + beta
// and with xh = (x - mean) rstd, g = dY gamma:
//   dX     = rstd (g - c1 - xh c2),  c1 = sum g / N (0 for RMS), c2 = sum g xh / N
//   dgamma = sum_m dY xh,  dbeta = sum_m dY
//
// A row is read once and stays in registers, so the variance is taken around
// the mean in a second pass that costs no memory traffic (the one-pass form
// with sum x^2 cancels when the mean is large against the deviation). All
// statistics and sums are fp32.
//
// T threads hold a row (NV vectors of E elements each, T vectors apart, so that
// a wave's access is one run); a wave alone needs no barrier.
//
// Memory bounds the forward: 4096 x 4096 bf16 moves 67 MB in 11.3 us (5.9 TB/s;
// a copy of that size reaches 5.7 to 6.0). One row alone takes 2.9 us, of which
// a launch is 2.
//
// The deviations are squared at 2^-k of their size, 4^k >= N: the sum of N
// squares then leaves fp32 no sooner than one square does, and a row's values
// may come near 2^64 (unscaled, rows of 2^60 gave rstd = 0 from about 256
// columns on). Powers of two change no rounding, and the scaled difference is
// one fused operation, so it costs nothing; the smallest square that keeps its
// bits is of a deviation of 2^(k - 63), which counts only without eps.
#include "rows.h"

namespace qlora {
namespace {

// Where a thread's vectors lie in a row of N elements. A row that is no whole
// number of vectors ends in a vector that is moved back to end with it: its
// first `skip` elements are the neighbour's too. Both hold the same values and
// store the same results; in the row's sums they count once. (Rows shorter
// than a vector, kShort, are read and written element by element.)
template <int T, int NV, int E>
struct Place {
  int at[NV];    // first element
  int skip[NV];  // elements that do not count; E: no vector
  __device__ __forceinline__ Place(int t, int N) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int first = (t + i * T) * E;
      at[i] = first + E <= N || N < E ? first : N - E;
      skip[i] = first >= N ? E : N < E ? 0 : first - at[i];
    }
  }
  __device__ __forceinline__ bool any(int i) const { return skip[i] < E; }
};

template <bool kBf16, bool kShort, int T, int NV, int E>
__device__ __forceinline__ void load_row(const elem_t<kBf16>* row, int N, const Place<T, NV, E>& p,
                                         Vec<kBf16, E> (&r)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    r[i] = zero_vec<kBf16, E>();
    if (p.any(i)) r[i] = kShort ? load_part<kBf16, E>(row, N) : load_vec<kBf16, E>(row + p.at[i]);
  }
}

template <bool kBf16, bool kShort, int T, int NV, int E>
__device__ __forceinline__ void store_row(elem_t<kBf16>* row, int N, const Place<T, NV, E>& p,
                                          const float (&v)[NV][E]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!p.any(i)) continue;
    if (kShort)
      store_part<kBf16, E>(row, v[i], N);
    else
      store_vec<kBf16, E>(row + p.at[i], v[i]);
  }
}

// The affine vectors, whose type is a run-time value.
template <bool kShort, int T, int NV, int E>
__device__ __forceinline__ void load_affine(const void* w, bool bf16, int N,
                                            const Place<T, NV, E>& p, float other,
                                            float (&v)[NV][E]) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) v[i][e] = other;
  if (!w) return;
  if (bf16) {
    Vec<true, E> r[NV];
    load_row<true, kShort, T, NV, E>(static_cast<const uint16_t*>(w), N, p, r);
#pragma unroll
    for (int i = 0; i < NV; ++i) to_float<true, E>(r[i], v[i]);
  } else {
    Vec<false, E> r[NV];
    load_row<false, kShort, T, NV, E>(static_cast<const float*>(w), N, p, r);
#pragma unroll
    for (int i = 0; i < NV; ++i) to_float<false, E>(r[i], v[i]);
  }
}

// 1 / N, the 2^-k at which deviations are squared, and what the squares' sum is
// multiplied by, 4^k / N.
struct Width {
  float inv, scale, inv_squares;
};

// The statistics of the row in v.
template <bool kShort, int T, int NV, int E>
__device__ __forceinline__ void row_stats(const float (&v)[NV][E], const Place<T, NV, E>& p, int N,
                                          const Width& w, bool center, float eps, float* red,
                                          int waves, int& par, float& mean, float& rstd) {
  const auto counts = [&](int i, int e) { return e >= p.skip[i] && (!kShort || e < N); };
  mean = 0.0f;
  if (center) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) s[0] += counts(i, e) ? v[i][e] : 0.0f;
    group_reduce<T, 1>(s, red, waves, par, OpSum());
    mean = s[0] * w.inv;
  }
  const float shift = -mean * w.scale;
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float d = counts(i, e) ? fmaf(v[i][e], w.scale, shift) : 0.0f;
      s[0] = fmaf(d, d, s[0]);
    }
  group_reduce<T, 1>(s, red, waves, par, OpSum());
  rstd = 1.0f / __builtin_sqrtf(s[0] * w.inv_squares + eps);
}

// A workgroup is one row's threads, or four waves with a row each.
constexpr int fwd_threads(int T) { return T == 64 ? 256 : T; }

struct NormFwd {
  const void* x;
  int64_t ldx, M;
  int N;
  bool center, w_bf16;
  const void* gamma;
  const void* beta;
  float eps;
  Width width;
  void* y;
  int64_t ldy;
  float* stats;
};

template <bool XB, bool YB, int T, int N8, bool kShort>
__global__ __launch_bounds__(fwd_threads(T)) void norm_fwd_kernel(NormFwd a) {
  constexpr int kThreads = fwd_threads(T);
  constexpr int kGroups = kThreads / T, kWaves = kThreads / 64;
  constexpr int E = XB && YB ? 8 : 4, NV = N8 * 8 / E;
  __shared__ float red[2 * kMostReduced * kWaves];
  const int t = threadIdx.x % T;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / T;
  if (row >= a.M) return;  // of four waves with a row each: they have no barriers
  const elem_t<XB>* x = static_cast<const elem_t<XB>*>(a.x);
  const Place<T, NV, E> p(t, a.N);
  Vec<XB, E> next[NV];
  load_row<XB, kShort>(x + row * a.ldx, a.N, p, next);
  float g[NV][E], b[NV][E];
  load_affine<kShort>(a.gamma, a.w_bf16, a.N, p, 1.0f, g);
  load_affine<kShort>(a.beta, a.w_bf16, a.N, p, 0.0f, b);
  int par = 0;
  for (; row < a.M; row += step) {
    float v[NV][E];
#pragma unroll
    for (int i = 0; i < NV; ++i) to_float<XB, E>(next[i], v[i]);
    if (row + step < a.M) load_row<XB, kShort>(x + (row + step) * a.ldx, a.N, p, next);
    float mean, rstd;
    row_stats<kShort>(v, p, a.N, a.width, a.center, a.eps, red, kWaves, par, mean, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = fmaf((v[i][e] - mean) * rstd, g[i][e], b[i][e]);
    store_row<YB, kShort>(static_cast<elem_t<YB>*>(a.y) + row * a.ldy, a.N, p, v);
    if (a.stats && t == 0) {
      a.stats[row] = mean;
      a.stats[a.M + row] = rstd;
    }
  }
}

struct NormBwd {
  const void* dY;
  int64_t ldy;
  const void* x;
  int64_t ldx, M;
  int N;
  bool center, w_bf16;
  const void* gamma;
  float eps;
  Width width;
  const float* stats;
  void* dX;
  int64_t lddx;
  float* part;  // [workgroups][2][ldp] sums of dY xh and of dY; NULL: not wanted
  int ldp;
};

constexpr int kBwdThreads = 1024;

// Each workgroup, one a CU, walks rows and keeps its columns' sums for dgamma
// and dbeta in registers; its row groups are added in LDS in order and leave
// one pair of partial rows, which norm_grad_kernel adds in order.
//
// Memory bounds it: 2048 x 8192 bf16 moves 101 MB and 17 MB of partial rows in
// 21 us (5.6 TB/s); norm_grad_kernel and the gap before it take 6 us more.
// Loads of the next row in flight (16 more registers) changed nothing there,
// nor did a quarter fewer vector instructions; two workgroups a CU double the
// partial rows (37 us). Nontemporal stores of dX are 3 us faster alone and cost
// the kernel that reads dX next 4.5 us, so the stores are plain.
template <bool XB, bool YB, bool DB, int T, int N8, bool kShort>
__global__ __launch_bounds__(kBwdThreads) void norm_bwd_kernel(NormBwd a) {
  constexpr int kGroups = kBwdThreads / T, kWaves = kBwdThreads / 64;
  constexpr int E = XB && YB && DB ? 8 : 4, NV = N8 * 8 / E;
  __shared__ float red[2 * kMostReduced * kWaves];
  __shared__ float join[kGroups > 1 ? 2 * T * 8 * N8 : 1];
  const int t = threadIdx.x % T, group = threadIdx.x / T;
  const elem_t<XB>* x = static_cast<const elem_t<XB>*>(a.x);
  const elem_t<YB>* dY = static_cast<const elem_t<YB>*>(a.dY);
  const Place<T, NV, E> p(t, a.N);
  const int64_t step = (int64_t)gridDim.x * kGroups;
  float g[NV][E], ag[NV][E], ab[NV][E];
  load_affine<kShort>(a.gamma, a.w_bf16, a.N, p, 1.0f, g);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) ag[i][e] = ab[i][e] = 0.0f;
  const float invN = a.width.inv;
  int par = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kGroups; row0 < a.M; row0 += step) {
    const int64_t row = row0 + group;
    float mean = 0.0f, rstd = 0.0f;
    if (a.stats && row < a.M) {
      if (a.center) mean = a.stats[row];
      rstd = a.stats[a.M + row];
    }
    Vec<XB, E> rx[NV];
    Vec<YB, E> ry[NV];
    if (row < a.M) {
      load_row<XB, kShort>(x + row * a.ldx, a.N, p, rx);
      load_row<YB, kShort>(dY + row * a.ldy, a.N, p, ry);
    } else {  // zeros: the barriers are reached either way
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        rx[i] = zero_vec<XB, E>();
        ry[i] = zero_vec<YB, E>();
      }
    }
    float d[NV][E], dy[NV][E];  // x, from below x - mean
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      to_float<XB, E>(rx[i], d[i]);
      to_float<YB, E>(ry[i], dy[i]);
    }
    if (!a.stats)
      row_stats<kShort>(d, p, a.N, a.width, a.center, a.eps, red, kWaves, par, mean, rstd);
    if (row >= a.M) rstd = 0.0f;  // of zeros; with eps = 0 it was infinite
    // With xh = d rstd: dX = rstd (g - c1 - d (rstd c2)), c2 = rstd (sum g d) / N.
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        // Where there is no element or no row, dY is 0 and d finite (unless
        // the row's own mean is not): it adds nothing.
        d[i][e] -= mean;
        ag[i][e] = fmaf(dy[i][e] * rstd, d[i][e], ag[i][e]);
        ab[i][e] += dy[i][e];
        dy[i][e] *= g[i][e];
        const float once = e >= p.skip[i] ? dy[i][e] : 0.0f;
        s[0] += once;
        s[1] = fmaf(once, d[i][e], s[1]);
      }
    if (a.dX) {
      group_reduce<T, 2>(s, red, kWaves, par, OpSum());
      const float c1 = a.center ? s[0] * invN : 0.0f, k2 = s[1] * invN * rstd * rstd;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) dy[i][e] = fmaf(-d[i][e], k2, dy[i][e] - c1) * rstd;
      if (row < a.M)
        store_row<DB, kShort>(static_cast<elem_t<DB>*>(a.dX) + row * a.lddx, a.N, p, dy);
    }
  }
  if (!a.part) return;
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.ldp;
  if constexpr (kGroups > 1) {
#pragma unroll 1
    for (int k = 0; k < kGroups; ++k) {
      if (group == k) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            // a moved-back vector's first elements are the neighbour's to add
            if (e < p.skip[i] || (kShort && e >= a.N)) continue;
            const int at = p.at[i] + e;
            join[at] = k ? join[at] + ag[i][e] : ag[i][e];
            join[T * 8 * N8 + at] = k ? join[T * 8 * N8 + at] + ab[i][e] : ab[i][e];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.N; c += kBwdThreads) {
      out[c] = join[c];
      out[a.ldp + c] = join[T * 8 * N8 + c];
    }
  } else {
    store_row<false, kShort>(out, a.N, p, ag);
    store_row<false, kShort>(out + a.ldp, a.N, p, ab);
  }
}

// grad[c] = sum over the workgroups' partial rows: 64 columns a workgroup,
// 16 lanes of four columns by 16 ranges of rows, the ranges added in order.
__global__ __launch_bounds__(256) void norm_grad_kernel(const float* part, int rows, int ldp,
                                                        int N, void* dgamma, void* dbeta,
                                                        bool bf16) {
  __shared__ f32x4_t join[16][16];
  void* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const int lane = threadIdx.x % 16, range = threadIdx.x / 16;
  const int c = blockIdx.x * 64 + lane * 4;
  const int per = (rows + 15) / 16;
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < ldp) {
    const float* p = part + blockIdx.y * ldp + c;
    const int end = min(rows, (range + 1) * per);
#pragma unroll 8
    for (int r = range * per; r < end; ++r)
      s += *reinterpret_cast<const f32x4_t*>(p + (int64_t)r * 2 * ldp);
  }
  join[range][lane] = s;
  __syncthreads();
  if (threadIdx.x < 64) {
    const float* q = reinterpret_cast<const float*>(join);
    float v = q[threadIdx.x];
    for (int k = 1; k < 16; ++k) v += q[k * 64 + threadIdx.x];
    const int at = blockIdx.x * 64 + threadIdx.x;
    if (at < N) {
      if (bf16)
        store1<true>(static_cast<uint16_t*>(out) + at, v);
      else
        store1<false>(static_cast<float*>(out) + at, v);
    }
  }
}

template <bool XB, bool YB, int T, int N8, bool kShort = false>
hipError_t fwd(const NormFwd& a, hipStream_t st) {
  constexpr int kThreads = fwd_threads(T);
  const int64_t blocks = (a.M + kThreads / T - 1) / (kThreads / T);
  // As many workgroups as the GPU holds at once, six of 256 threads a CU or one
  // of 512, each with its share of rows (4096 x 4096 bf16: 11.3 us, one row a
  // workgroup 13.3 us; 1500 x 12000: 16.5 us, 20 us with a row or two each).
  const int64_t most = kThreads <= 256 ? 1536 * 256 / kThreads : 256;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  hipLaunchKernelGGL((norm_fwd_kernel<XB, YB, T, N8, kShort>), dim3(grid), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

// Threads of a row and elements of a thread (in eights): few threads with more
// elements each, as long as the registers hold them, since a row's reductions
// and barriers cost every wave the same. Measured on bf16 rows of 33.5 MB, us:
//   N =   512:  64 x 1 13.3, 128 x 1 19.6       N =  4096: 256 x 2 12.9, 512 x 1 18.8
//   N =  1024:  64 x 2 13.1, 128 x 1 14.4       N =  8192: 256 x 4 24.9, 512 x 2 25.1,
//   N =  2048: 128 x 2 12.8, 256 x 1 14.3,                 1024 x 1 34.0 (67 MB)
//               64 x 4 15.2                     N = 16384: 512 x 4 25.2, 1024 x 2 27.0 (67 MB)
template <bool XB, bool YB>
hipError_t fwd_width(const NormFwd& a, hipStream_t st) {
  if (a.N < (XB && YB ? 8 : 4)) return fwd<XB, YB, 64, 1, true>(a, st);
  if (a.N <= 512) return fwd<XB, YB, 64, 1>(a, st);
  if (a.N <= 1024) return fwd<XB, YB, 64, 2>(a, st);
  if (a.N <= 2048) return fwd<XB, YB, 128, 2>(a, st);
  if (a.N <= 4096) return fwd<XB, YB, 256, 2>(a, st);
  if (a.N <= 8192) return fwd<XB, YB, 256, 4>(a, st);
  return fwd<XB, YB, 512, 4>(a, st);
}

template <bool XB, bool YB, bool DB, int T, int N8, bool kShort = false>
hipError_t bwd(const NormBwd& a, unsigned grid, hipStream_t st) {
  hipLaunchKernelGGL((norm_bwd_kernel<XB, YB, DB, T, N8, kShort>), dim3(grid), dim3(kBwdThreads), 0,
                     st, a);
  return hipGetLastError();
}

// Threads of a row, eight elements each while 1024 threads hold the row; more
// elements a thread leave too few registers. Measured, us: 32768 x 512 64 x 1
// 31.9, 128 x 1 32.1, 256 x 1 46; 16384 x 1024 128 x 1 28.4, 64 x 2 50, 256 x 1
// 31.0; 8192 x 2048 256 x 1 26.3, 128 x 2 41, 512 x 1 29.9; 4096 x 4096 512 x 1
// 27.2, 256 x 2 40; 2048 x 8192 1024 x 1 27.6, 512 x 2 39. Rows past 8192 need 16
// elements a thread all the same: those builds sit at the limit of 128 registers
// and, but for the one that is bf16 throughout, keep 4 to 28 more in scratch
// (2048 x 16384 bf16 48 us for 201 MB, fp32 95 us for 403 MB).
template <bool XB, bool YB, bool DB>
hipError_t bwd_width(const NormBwd& a, unsigned grid, hipStream_t st) {
  if (a.N < (XB && YB && DB ? 8 : 4)) return bwd<XB, YB, DB, 64, 1, true>(a, grid, st);
  if (a.N <= 512) return bwd<XB, YB, DB, 64, 1>(a, grid, st);
  if (a.N <= 1024) return bwd<XB, YB, DB, 128, 1>(a, grid, st);
  if (a.N <= 2048) return bwd<XB, YB, DB, 256, 1>(a, grid, st);
  if (a.N <= 4096) return bwd<XB, YB, DB, 512, 1>(a, grid, st);
  if (a.N <= 8192) return bwd<XB, YB, DB, 1024, 1>(a, grid, st);
  return bwd<XB, YB, DB, 1024, 2>(a, grid, st);
}

// k is the least that has 4^k >= N.
Width width_of(int64_t N) {
  Width w{1.0f / (float)N, 1.0f, 1.0f / (float)N};
  for (int64_t n = 1; n < N; n *= 4) {
    w.scale *= 0.5f;
    w.inv_squares *= 4.0f;
  }
  return w;
}

int bwd_groups(int64_t N) {
  return N <= 512 ? 16 : N <= 1024 ? 8 : N <= 2048 ? 4 : N <= 4096 ? 2 : 1;
}

}  // namespace

int norm_bwd_parts(int64_t M, int64_t N) {
  const int g = bwd_groups(N);
  const int64_t need = (M + g - 1) / g;
  return (int)(need < 256 ? need : 256);
}

hipError_t launch_norm_fwd(const void* x, int64_t ldx, bool x_bf16, int64_t M, int64_t N,
                           bool center, const void* gamma, const void* beta, bool w_bf16,
                           float eps, void* y, int64_t ldy, bool y_bf16, float* stats,
                           hipStream_t st) {
  const NormFwd a{x, ldx, M, (int)N, center, w_bf16, gamma, beta, eps, width_of(N), y, ldy, stats};
  if (x_bf16) return y_bf16 ? fwd_width<true, true>(a, st) : fwd_width<true, false>(a, st);
  return y_bf16 ? fwd_width<false, true>(a, st) : fwd_width<false, false>(a, st);
}

hipError_t launch_norm_bwd(const void* dY, int64_t ldy, bool dy_bf16, const void* x, int64_t ldx,
                           bool x_bf16, int64_t M, int64_t N, bool center, const void* gamma,
                           bool w_bf16, float eps, const float* stats, void* dX, int64_t lddx,
                           bool dx_bf16, void* dgamma, void* dbeta, bool grad_bf16, float* part,
                           hipStream_t st) {
  const int ldp = (int)((N + 7) / 8 * 8);
  const bool grads = dgamma || dbeta;
  const NormBwd a{dY, ldy, x, ldx, M, (int)N, center, w_bf16, gamma, eps, width_of(N), stats, dX,
                  lddx, grads ? part : nullptr, ldp};
  const unsigned grid = (unsigned)norm_bwd_parts(M, N);
  hipError_t e = hipSuccess;
  if (M == 0) {
    // no rows: norm_grad_kernel writes zeros
  } else if (x_bf16 && dy_bf16)
    e = dx_bf16 ? bwd_width<true, true, true>(a, grid, st) : bwd_width<true, true, false>(a, grid, st);
  else if (x_bf16)
    e = dx_bf16 ? bwd_width<true, false, true>(a, grid, st) : bwd_width<true, false, false>(a, grid, st);
  else if (dy_bf16)
    e = dx_bf16 ? bwd_width<false, true, true>(a, grid, st) : bwd_width<false, true, false>(a, grid, st);
  else
    e = dx_bf16 ? bwd_width<false, false, true>(a, grid, st) : bwd_width<false, false, false>(a, grid, st);
  if (e == hipSuccess && grads) {
    hipLaunchKernelGGL(norm_grad_kernel, dim3((unsigned)((ldp + 63) / 64), 2), dim3(256), 0, st, part,
                       (int)grid, ldp, (int)N, dgamma, dbeta, grad_bf16);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace qlora
