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
// T threads hold a row, NV vectors of eight elements each; a wave alone needs
// no barrier.
#include <type_traits>

#include "rows.h"

namespace qlora {
namespace {

// The statistics of the rows in v (n elements of it count, from column 0 on
// in steps of T vectors).
template <int T, int NV>
__device__ __forceinline__ void row_stats(const float (&v)[NV][8], const int (&cnt)[NV], float invN,
                                          bool center, float eps, float* red, int waves, int& par,
                                          float& mean, float& rstd) {
  mean = 0.0f;
  if (center) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[i][e];
    group_reduce<T, 1>(s, red, waves, par, OpSum());
    mean = s[0] * invN;
  }
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = e < cnt[i] ? v[i][e] - mean : 0.0f;
      s[0] = fmaf(d, d, s[0]);
    }
  group_reduce<T, 1>(s, red, waves, par, OpSum());
  rstd = 1.0f / __builtin_sqrtf(s[0] * invN + eps);
}

template <bool kBf16, int NV, int T>
__device__ __forceinline__ void load_row(const elem_t<kBf16>* row, int t, int N,
                                         const int (&cnt)[NV], Vec<kBf16, 8> (&r)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) r[i] = cnt[i] == 8 ? load_vec<kBf16, 8>(row + (t + i * T) * 8) : zero_vec<kBf16, 8>();
  if (N % 8) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (cnt[i] > 0 && cnt[i] < 8) r[i] = load_part<kBf16, 8>(row + (t + i * T) * 8, cnt[i]);
  }
}

struct NormFwd {
  const void* x;
  int64_t ldx, M;
  int N;
  bool center, w_bf16;
  const void* gamma;
  const void* beta;
  float eps;
  void* y;
  int64_t ldy;
  float* stats;
};

template <bool XB, bool YB, int T, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_fwd_kernel(NormFwd a) {
  constexpr int kThreads = T < 256 ? 256 : T;
  constexpr int kGroups = kThreads / T, kWaves = kThreads / 64;
  __shared__ float red[2 * kWaves];
  const int t = threadIdx.x % T;
  int cnt[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int left = a.N - (t + i * T) * 8;
    cnt[i] = left < 0 ? 0 : left > 8 ? 8 : left;
  }
  float g[NV][8], b[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      g[i][e] = 1.0f;
      b[i][e] = 0.0f;
    }
    if (a.gamma && cnt[i]) load_any_vec<8>(a.gamma, a.w_bf16, (t + i * T) * 8, cnt[i], g[i]);
    if (a.beta && cnt[i]) load_any_vec<8>(a.beta, a.w_bf16, (t + i * T) * 8, cnt[i], b[i]);
  }
  const float invN = 1.0f / (float)a.N;
  int par = 0;
  for (int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / T; row < a.M;
       row += (int64_t)gridDim.x * kGroups) {
    Vec<XB, 8> raw[NV];
    load_row<XB, NV, T>(static_cast<const elem_t<XB>*>(a.x) + row * a.ldx, t, a.N, cnt, raw);
    float v[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) to_float<XB, 8>(raw[i], v[i]);
    float mean, rstd;
    row_stats<T, NV>(v, cnt, invN, a.center, a.eps, red, kWaves, par, mean, rstd);
    elem_t<YB>* out = static_cast<elem_t<YB>*>(a.y) + row * a.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = fmaf((v[i][e] - mean) * rstd, g[i][e], b[i][e]);
      if (cnt[i] == 8)
        store_vec<YB, 8>(out + (t + i * T) * 8, v[i]);
      else if (cnt[i] > 0)
        store_part<YB, 8>(out + (t + i * T) * 8, v[i], cnt[i]);
    }
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
  const float* stats;
  void* dX;
  int64_t lddx;
  float* part;  // [workgroups][2][ldp] sums of dY xh and of dY; NULL: not wanted
  int ldp;
};

constexpr int kBwdThreads = 1024;

// Each workgroup walks rows and keeps its columns' sums for dgamma and dbeta
// in registers; its row groups are added in LDS in order and leave one pair
// of partial rows, which norm_grad_kernel adds in order.
template <bool XB, bool YB, bool DB, int T, int NV>
__global__ __launch_bounds__(kBwdThreads) void norm_bwd_kernel(NormBwd a) {
  constexpr int kGroups = kBwdThreads / T, kWaves = kBwdThreads / 64;
  __shared__ float red[2 * 2 * kWaves];
  __shared__ float join[kGroups > 1 ? 2 * T * 8 * NV : 1];
  const int t = threadIdx.x % T, group = threadIdx.x / T;
  int cnt[NV];
  float g[NV][8], ag[NV][8], ab[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int left = a.N - (t + i * T) * 8;
    cnt[i] = left < 0 ? 0 : left > 8 ? 8 : left;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      g[i][e] = 1.0f;
      ag[i][e] = ab[i][e] = 0.0f;
    }
    if (a.gamma && cnt[i]) load_any_vec<8>(a.gamma, a.w_bf16, (t + i * T) * 8, cnt[i], g[i]);
  }
  const float invN = 1.0f / (float)a.N;
  int par = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kGroups; row0 < a.M;
       row0 += (int64_t)gridDim.x * kGroups) {
    const int64_t row = row0 + group;
    const bool live = row < a.M;  // the barriers below are reached either way
    Vec<XB, 8> rx[NV];
    Vec<YB, 8> ry[NV];
    float mean = 0.0f, rstd = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      rx[i] = zero_vec<XB, 8>();
      ry[i] = zero_vec<YB, 8>();
    }
    if (live) {
      load_row<XB, NV, T>(static_cast<const elem_t<XB>*>(a.x) + row * a.ldx, t, a.N, cnt, rx);
      load_row<YB, NV, T>(static_cast<const elem_t<YB>*>(a.dY) + row * a.ldy, t, a.N, cnt, ry);
      if (a.stats) {
        mean = a.center ? a.stats[row] : 0.0f;
        rstd = a.stats[a.M + row];
      }
    }
    float x[NV][8], dy[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      to_float<XB, 8>(rx[i], x[i]);
      to_float<YB, 8>(ry[i], dy[i]);
    }
    if (!a.stats) row_stats<T, NV>(x, cnt, invN, a.center, a.eps, red, kWaves, par, mean, rstd);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[i][e] = (x[i][e] - mean) * rstd;
        if (live) {
          // columns past N hold dY = 0 but x = -mean rstd: they add nothing
          ag[i][e] = fmaf(dy[i][e], x[i][e], ag[i][e]);
          ab[i][e] += dy[i][e];
        }
        dy[i][e] *= g[i][e];
        s[0] += dy[i][e];
        s[1] = fmaf(dy[i][e], x[i][e], s[1]);
      }
    if (a.dX) {
      group_reduce<T, 2>(s, red, kWaves, par, OpSum());
      const float c1 = a.center ? s[0] * invN : 0.0f, c2 = s[1] * invN;
      if (live) {
        elem_t<DB>* out = static_cast<elem_t<DB>*>(a.dX) + row * a.lddx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dy[i][e] = (dy[i][e] - c1 - x[i][e] * c2) * rstd;
          if (cnt[i] == 8)
            store_vec<DB, 8>(out + (t + i * T) * 8, dy[i]);
          else if (cnt[i] > 0)
            store_part<DB, 8>(out + (t + i * T) * 8, dy[i], cnt[i]);
        }
      }
    }
  }
  if (!a.part) return;
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.ldp;
  if constexpr (kGroups > 1) {
    for (int k = 0; k < kGroups; ++k) {
      if (group == k) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at = (t + i * T) * 8 + e;
            join[at] = k ? join[at] + ag[i][e] : ag[i][e];
            join[T * 8 * NV + at] = k ? join[T * 8 * NV + at] + ab[i][e] : ab[i][e];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.N; c += kBwdThreads) {
      out[c] = join[c];
      out[a.ldp + c] = join[T * 8 * NV + c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (cnt[i]) {  // ldp is a multiple of eight
        store_vec<false, 8>(out + (t + i * T) * 8, ag[i]);
        store_vec<false, 8>(out + a.ldp + (t + i * T) * 8, ab[i]);
      }
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

template <bool XB, bool YB, int T, int NV>
hipError_t fwd(const NormFwd& a, hipStream_t st) {
  constexpr int kThreads = T < 256 ? 256 : T;
  const int64_t blocks = (a.M + kThreads / T - 1) / (kThreads / T);
  const unsigned grid = (unsigned)(blocks < 4096 ? blocks : 4096);
  hipLaunchKernelGGL((norm_fwd_kernel<XB, YB, T, NV>), dim3(grid), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

template <bool XB, bool YB>
hipError_t fwd_width(const NormFwd& a, hipStream_t st) {
  if (a.N <= 512) return fwd<XB, YB, 64, 1>(a, st);
  if (a.N <= 1024) return fwd<XB, YB, 64, 2>(a, st);
  if (a.N <= 2048) return fwd<XB, YB, 256, 1>(a, st);
  if (a.N <= 4096) return fwd<XB, YB, 256, 2>(a, st);
  if (a.N <= 8192) return fwd<XB, YB, 256, 4>(a, st);
  return fwd<XB, YB, 1024, 2>(a, st);
}

template <bool XB, bool YB, bool DB>
hipError_t bwd_width(const NormBwd& a, unsigned grid, hipStream_t st) {
  const dim3 g(grid), b(kBwdThreads);
  if (a.N <= 512)
    hipLaunchKernelGGL((norm_bwd_kernel<XB, YB, DB, 64, 1>), g, b, 0, st, a);
  else if (a.N <= 1024)
    hipLaunchKernelGGL((norm_bwd_kernel<XB, YB, DB, 128, 1>), g, b, 0, st, a);
  else if (a.N <= 2048)
    hipLaunchKernelGGL((norm_bwd_kernel<XB, YB, DB, 256, 1>), g, b, 0, st, a);
  else if (a.N <= 4096)
    hipLaunchKernelGGL((norm_bwd_kernel<XB, YB, DB, 512, 1>), g, b, 0, st, a);
  else if (a.N <= 8192)
    hipLaunchKernelGGL((norm_bwd_kernel<XB, YB, DB, 1024, 1>), g, b, 0, st, a);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<XB, YB, DB, 1024, 2>), g, b, 0, st, a);
  return hipGetLastError();
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
  const NormFwd a{x, ldx, M, (int)N, center, w_bf16, gamma, beta, eps, y, ldy, stats};
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
  const NormBwd a{dY, ldy, x, ldx, M, (int)N, center, w_bf16, gamma, eps, stats, dX, lddx,
                  grads ? part : nullptr, ldp};
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
