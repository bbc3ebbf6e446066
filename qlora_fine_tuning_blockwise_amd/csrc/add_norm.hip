// The norm behind a residual addition on gfx950, forward and backward, with an
// output in 8 bits:
//   h = x + r, rounded to r's type;  y = norm(h) as in norm.hip
//   E4M3: scale = max |y| / 448 over the row, code = e4m3(y / scale)
// and with dY, and dH that reaches h by itself:
//   dX = norm's dX of (dY, h) + dH  (the gradient of x and of r alike)
//
// The norm is that of the rounded h, the value that the next layer's addition
// and this norm's backward read: statistics and gradients then belong to the
// same row. x and r are read once, h and y written once; the sum, the
// statistics and y stay in fp32 registers, y is rounded once, and its largest
// magnitude is known before any of it is stored, so 8 bits cost one more
// reduction and no more traffic.
//
// y / scale is formed as y (448 / max |y|), one product an element: it differs
// from the quotient by two roundings of fp32, 2^-23 of a value that E4M3 rounds
// at 2^-4. The largest magnitude is a maximum of bit patterns, in which a NaN is
// the largest: the scale of a row with a NaN is NaN, and so are its codes.
//
// Memory bounds it, as it does the norm: 4096 x 4096 bf16 to 8 bits, 117 MB, 20.5
// us (5.7 TB/s); the backward of 2048 x 8192 bf16, 134 MB and 17 MB of partial
// column sums, 25.5 us and 4.0 us for joining them. One row of 4096: 2.6 us.
#include "norm_rows.h"

namespace qlora {
namespace {

constexpr int kOutF32 = 0, kOutBf16 = 1, kOutE4m3 = 2;
constexpr float kE4m3Max = 448.0f;

struct OpMaxBits {
  __device__ __forceinline__ float operator()(float a, float b) const {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    return __uint_as_float(x > y ? x : y);
  }
};

// E consecutive codes, rounded to nearest even (|v| <= 464 or NaN).
template <int E>
__device__ __forceinline__ void to_e4m3(const float (&v)[E], uint32_t (&q)[E / 4]) {
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], w, true);
    q[i] = (uint32_t)w;
  }
}

typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));

template <bool kShort, int T, int NV, int E>
__device__ __forceinline__ void store_codes(uint8_t* row, int N, const Place<T, NV, E>& p,
                                            const float (&v)[NV][E]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!p.any(i)) continue;
    uint32_t q[E / 4];
    to_e4m3<E>(v[i], q);
    if (kShort) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e < N) row[e] = (uint8_t)(q[e / 4] >> 8 * (e % 4));
    } else if constexpr (E == 8) {
      *reinterpret_cast<u32x2_a1*>(row + p.at[i]) = u32x2_t{q[0], q[1]};
    } else {
      *reinterpret_cast<u32_a1*>(row + p.at[i]) = q[0];
    }
  }
}

constexpr int fwd_threads(int T) { return T == 64 ? 256 : T; }

struct AddNormFwd {
  const void* x;
  int64_t ldx;
  const void* r;  // NULL: h is x, and is not written
  int64_t ldr, M;
  int N;
  bool center, w_bf16;
  const void* gamma;
  const void* beta;
  float eps;
  Width width;
  void* h;
  int64_t ldh;
  void* y;
  int64_t ldy;
  float* scales;
  float* stats;
};

template <bool XB, bool HB, int kOut, int T, int N8, bool kShort>
__global__ __launch_bounds__(fwd_threads(T)) void add_norm_fwd_kernel(AddNormFwd a) {
  constexpr int kThreads = fwd_threads(T);
  constexpr int kGroups = kThreads / T, kWaves = kThreads / 64;
  constexpr int E = XB && HB && kOut != kOutF32 ? 8 : 4, NV = N8 * 8 / E;
  __shared__ float red[2 * kMostReduced * kWaves];
  const int t = threadIdx.x % T;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / T;
  if (row >= a.M) return;  // of four waves with a row each: they have no barriers
  const elem_t<XB>* x = static_cast<const elem_t<XB>*>(a.x);
  const elem_t<HB>* r = static_cast<const elem_t<HB>*>(a.r);
  const Place<T, NV, E> p(t, a.N);
  Vec<XB, E> nx[NV];
  Vec<HB, E> nr[NV];
  load_row<XB, kShort>(x + row * a.ldx, a.N, p, nx);
  if (r) load_row<HB, kShort>(r + row * a.ldr, a.N, p, nr);
  float g[NV][E], b[NV][E];
  load_affine<kShort>(a.gamma, a.w_bf16, a.N, p, 1.0f, g);
  load_affine<kShort>(a.beta, a.w_bf16, a.N, p, 0.0f, b);
  int par = 0;
  for (; row < a.M; row += step) {
    float v[NV][E];
#pragma unroll
    for (int i = 0; i < NV; ++i) to_float<XB, E>(nx[i], v[i]);
    if (r) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float o[E];
        to_float<HB, E>(nr[i], o);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          v[i][e] += o[e];
          if (HB) v[i][e] = bf16_lo(pack_bf16x2(v[i][e], 0.0f));
        }
      }
    }
    if (row + step < a.M) {
      load_row<XB, kShort>(x + (row + step) * a.ldx, a.N, p, nx);
      if (r) load_row<HB, kShort>(r + (row + step) * a.ldr, a.N, p, nr);
    }
    float mean, rstd;
    row_stats<kShort>(v, p, a.N, a.width, a.center, a.eps, red, kWaves, par, mean, rstd);
    // Behind the statistics' exchange every thread has its elements of the row:
    // h may lie on x or on r.
    if (r) store_row<HB, kShort>(static_cast<elem_t<HB>*>(a.h) + row * a.ldh, a.N, p, v);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = fmaf((v[i][e] - mean) * rstd, g[i][e], b[i][e]);
    if constexpr (kOut == kOutE4m3) {
      float most[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (p.any(i) && (!kShort || e < a.N))
            most[0] = OpMaxBits()(most[0], __uint_as_float(__float_as_uint(v[i][e]) & 0x7FFFFFFFu));
      group_reduce<T, 1>(most, red, kWaves, par, OpMaxBits());
      const float scale = most[0] / kE4m3Max;
      if (most[0] >= 0x1p-100f || most[0] != most[0]) {
        const float inv = kE4m3Max / most[0];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] *= inv;
      } else {  // 448 / max leaves fp32: quotients, which a rounded scale may put past 448
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e)
            v[i][e] = scale > 0.0f ? fminf(fmaxf(v[i][e] / scale, -kE4m3Max), kE4m3Max) : 0.0f;
      }
      store_codes<kShort>(static_cast<uint8_t*>(a.y) + row * a.ldy, a.N, p, v);
      if (t == 0) a.scales[row] = scale;
    } else {
      constexpr bool YB = kOut == kOutBf16;
      store_row<YB, kShort>(static_cast<elem_t<YB>*>(a.y) + row * a.ldy, a.N, p, v);
    }
    if (a.stats && t == 0) {
      a.stats[row] = mean;
      a.stats[a.M + row] = rstd;
    }
  }
}

template <bool XB, bool HB, int kOut, int T, int N8, bool kShort = false>
hipError_t fwd(const AddNormFwd& a, hipStream_t st) {
  constexpr int kThreads = fwd_threads(T);
  const int64_t blocks = (a.M + kThreads / T - 1) / (kThreads / T);
  const int64_t most = kThreads <= 256 ? 1536 * 256 / kThreads : 256;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  hipLaunchKernelGGL((add_norm_fwd_kernel<XB, HB, kOut, T, N8, kShort>), dim3(grid), dim3(kThreads),
                     0, st, a);
  return hipGetLastError();
}

template <bool XB, bool HB, int kOut>
hipError_t fwd_width(const AddNormFwd& a, hipStream_t st) {
  if (a.N < (XB && HB && kOut != kOutF32 ? 8 : 4)) return fwd<XB, HB, kOut, 64, 1, true>(a, st);
  if (a.N <= 512) return fwd<XB, HB, kOut, 64, 1>(a, st);
  if (a.N <= 1024) return fwd<XB, HB, kOut, 64, 2>(a, st);
  if (a.N <= 2048) return fwd<XB, HB, kOut, 128, 2>(a, st);
  if (a.N <= 4096) return fwd<XB, HB, kOut, 256, 2>(a, st);
  if (a.N <= 8192) return fwd<XB, HB, kOut, 512, 2>(a, st);
  return fwd<XB, HB, kOut, 1024, 2>(a, st);
}

template <bool XB, bool HB>
hipError_t fwd_out(const AddNormFwd& a, int y_kind, hipStream_t st) {
  if (y_kind == kOutE4m3) return fwd_width<XB, HB, kOutE4m3>(a, st);
  return y_kind == kOutBf16 ? fwd_width<XB, HB, kOutBf16>(a, st) : fwd_width<XB, HB, kOutF32>(a, st);
}

}  // namespace

hipError_t launch_add_norm_fwd(const void* x, int64_t ldx, bool x_bf16, const void* r, int64_t ldr,
                               bool r_bf16, int64_t M, int64_t N, bool center, const void* gamma,
                               const void* beta, bool w_bf16, float eps, void* h, int64_t ldh,
                               void* y, int64_t ldy, int y_kind, float* scales, float* stats,
                               hipStream_t st) {
  const AddNormFwd a{x,    ldx,   r,   ldr,         M, (int)N, center, w_bf16, gamma,
                     beta, eps,   width_of(N), h, ldh, y, ldy, scales, stats};
  if (x_bf16) return r_bf16 ? fwd_out<true, true>(a, y_kind, st) : fwd_out<true, false>(a, y_kind, st);
  return r_bf16 ? fwd_out<false, true>(a, y_kind, st) : fwd_out<false, false>(a, y_kind, st);
}

hipError_t launch_add_norm_bwd(const void* dY, int64_t ldy, bool dy_bf16, const void* dH,
                               int64_t lddh, const void* h, int64_t ldh, bool h_bf16, int64_t M,
                               int64_t N, bool center, const void* gamma, bool w_bf16, float eps,
                               const float* stats, void* dX, int64_t lddx, bool dx_bf16,
                               void* dgamma, void* dbeta, bool grad_bf16, float* part,
                               hipStream_t st) {
  const int ldp = (int)((N + 7) / 8 * 8);
  const bool grads = dgamma || dbeta;
  const NormBwd a{dY, ldy, dH, lddh, h, ldh, M, (int)N, center, w_bf16, gamma, eps, width_of(N),
                  stats, dX, lddx, grads ? part : nullptr, ldp};
  const unsigned grid = (unsigned)norm_bwd_parts(M, N);
  hipError_t e = hipSuccess;
  if (M == 0) {
    // no rows: the gradients become zeros
  } else if (h_bf16 && dy_bf16)
    e = dx_bf16 ? bwd_width<true, true, true, true>(a, grid, st)
                : bwd_width<true, true, false, true>(a, grid, st);
  else if (h_bf16)
    e = dx_bf16 ? bwd_width<true, false, true, true>(a, grid, st)
                : bwd_width<true, false, false, true>(a, grid, st);
  else if (dy_bf16)
    e = dx_bf16 ? bwd_width<false, true, true, true>(a, grid, st)
                : bwd_width<false, true, false, true>(a, grid, st);
  else
    e = dx_bf16 ? bwd_width<false, false, true, true>(a, grid, st)
                : bwd_width<false, false, false, true>(a, grid, st);
  if (e == hipSuccess && grads)
    e = launch_norm_grad(part, (int)grid, ldp, N, dgamma, dbeta, grad_bf16, st);
  return e;
}

}  // namespace qlora
