// The vocabulary head's logits of a few rows on gfx950 (scoring a token, the last
// tokens of some sequences): what head.hip's tile kernel does for whole tiles of
// rows, as one stream through W.
//
// Memory bounds it: every row of W is read once, and up to 64 rows of x take 4
// products of the matrix units for each of W's fragments. A wave takes 16 entries
// of the vocabulary and all rows: fragments of W come straight from memory into
// registers, two chunks ahead of the one that is multiplied; those of x are shared
// by the eight waves through LDS, two chunks in turn (from the caches, each wave
// for itself, they cost 16 rows a third and 64 rows twice the time). Unaligned
// rows and odd widths run the same loads; the last chunk of K is masked. The
// statistics read W with the nontemporal hint; the probabilities do not, since the
// product behind them reads W again and finds a part of it in the Infinity Cache
// (32 rows, 32000 x 4096: 98 instead of 109 us for the gradient; at most 16 rows have
// a pass of their own, head_few_dx.hip). 1 row of 32000 x 4096: 48 us, 5.4 TB/s; of
// 128000 x 4096: 5.3 TB/s.
#include "head_terms.h"

namespace qlora {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

constexpr int kFrags = 8, kChunk = 32 * kFrags;  // fragments and elements of a chunk of K

__device__ __forceinline__ u32x4_t words(const Vec<true, 8>& v) {
  return u32x4_t{v.w[0], v.w[1], v.w[2], v.w[3]};
}

__device__ __forceinline__ Vec<true, 8> load_upto(const uint16_t* p, int64_t k, int64_t K) {
  const int n = count_below<8>(k, K);
  return n == 8 ? load_vec<true, 8>(p + k) : load_part<true, 8>(p + k, n);
}

// NT groups of 16 rows, kWaves waves.
template <int NT, int kWaves, bool kProbs>
__global__ __launch_bounds__(64 * kWaves) void head_few_kernel(HeadFew p) {
  constexpr int kThreads = 64 * kWaves, kEntries = 16 * kWaves;  // of the vocabulary
  constexpr int kBring = NT * 16 * 32 / kThreads, kRows = kThreads / 32;  // parts of x a thread, rows apart
  // A row's chunk is 512 bytes, 16-byte part c of row r at c ^ (r & 7).
  __shared__ __attribute__((aligned(16))) uint16_t xs[2][16 * NT * kChunk];
  __shared__ float2 red[kProbs ? 1 : kWaves * 16 * NT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int rows = kProbs ? *p.count : (int)p.M;
  // Without a live row nothing is read of W.
  if constexpr (kProbs) {
    if (rows == 0) return;
  } else {
    const int64_t label = lane < rows ? load_index(p.labels, p.ids64, lane) : -1;
    if (!__ballot(label >= 0 && label < p.V)) return;
  }
  const int64_t v0 = (int64_t)blockIdx.x * kEntries + 16 * wave;  // in the piece
  const int64_t K = p.K;
  // This lane's row of W; past the piece the last one, whose results are not used.
  const uint16_t* wrow = p.W + (v0 + i < p.vocab ? v0 + i : p.vocab - 1) * p.ldw;
  // Parts of x's chunk that this thread brings: rows r, r + kRows, ... (past the
  // last row that one, whose results are not used).
  const int xr = threadIdx.x / 32, xc = threadIdx.x % 32;
  const uint16_t* xrow[kBring];
#pragma unroll
  for (int t = 0; t < kBring; ++t) {
    const int j = kRows * t + xr < rows ? kRows * t + xr : rows > 0 ? rows - 1 : 0;
    xrow[t] = p.x + (kProbs ? (int64_t)(rows > 0 ? p.map[j] : 0) : (int64_t)j) * p.ldx;
  }
  // Two chunks in flight: chunk c in set c % 2.
  Vec<true, 8> wv[2][kFrags], xv[2][kBring];
  const auto load = [&](int c, auto sc) {  // x first: it is waited for while W is in flight
    constexpr int S = decltype(sc)::value;
    const int64_t k0 = (int64_t)c * kChunk;
#pragma unroll
    for (int t = 0; t < kBring; ++t) xv[S][t] = load_vec<true, 8>(xrow[t] + k0 + 8 * xc);
#pragma unroll
    for (int f = 0; f < kFrags; ++f) wv[S][f] = load_vec<true, 8, !kProbs>(wrow + k0 + 32 * f + 8 * g);
  };
  const auto put_x = [&](auto sc) {
    constexpr int S = decltype(sc)::value;
#pragma unroll
    for (int t = 0; t < kBring; ++t) {
      const int r = kRows * t + xr;
      *reinterpret_cast<u32x4_t*>(&xs[S][r * kChunk + 8 * (xc ^ (r & 7))]) = words(xv[S][t]);
    }
  };
  // LDS written by every wave; loads from memory may still fly.
  const auto meet_waves = [] {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  f32x4_t acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const auto multiply = [&](auto sc) {
    constexpr int S = decltype(sc)::value;
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        acc[t] = mfma_16x16x32(
            words(wv[S][f]),
            *reinterpret_cast<const u32x4_t*>(&xs[S][(16 * t + i) * kChunk + 8 * ((4 * f + g) ^ (i & 7))]),
            acc[t]);
    __builtin_amdgcn_sched_barrier(0);
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  // Chunk c: multiplied, c + 2 requested in its place, c + 1 of x made ready
  // (its buffer was read before the last meeting).
  const auto chunk = [&](int c, auto more, auto sc, auto oc) {
    multiply(sc);
    if constexpr (decltype(more)::value > 1) load(c + 2, sc);
    if constexpr (decltype(more)::value > 0) {
      put_x(oc);
      meet_waves();
    }
  };
  using I2 = std::integral_constant<int, 2>;
  const int chunks = (int)(K / kChunk);  // whole ones
  if (chunks > 1) {
    load(0, I0());
    load(1, I1());
    put_x(I0());
    meet_waves();
    int c = 0;
    for (; c + 3 < chunks; c += 2) {
      chunk(c, I2(), I0(), I1());
      chunk(c + 1, I2(), I1(), I0());
    }
    if (c + 2 < chunks) {
      chunk(c, I2(), I0(), I1());
      chunk(c + 1, I1(), I1(), I0());
      chunk(c + 2, I0(), I0(), I1());
    } else {
      chunk(c, I1(), I0(), I1());
      chunk(c + 1, I0(), I1(), I0());
    }
  } else if (chunks == 1) {
    load(0, I0());
    put_x(I0());
    meet_waves();
    chunk(0, I0(), I0(), I1());
  }
  if (const int64_t k0 = (int64_t)chunks * kChunk; k0 < K) {  // the rest, masked
#pragma unroll
    for (int t = 0; t < kBring; ++t) xv[0][t] = load_upto(xrow[t], k0 + 8 * xc, K);
#pragma unroll
    for (int f = 0; f < kFrags; ++f) wv[0][f] = load_upto(wrow, k0 + 32 * f + 8 * g, K);
    meet_waves();  // the last chunk may have been read from this buffer
    put_x(I0());
    meet_waves();
    multiply(I0());
  }
  // Element e of acc[t] is entry v0 + 4g + e of the vocabulary, row 16t + i.
  const int64_t v = v0 + 4 * g;
  if constexpr (!kProbs) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t row = 16 * t + i;
      const int64_t label = row < rows ? load_index(p.labels, p.ids64, row) : -1;
      float m = -INFINITY, z[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[e] = v + e < p.vocab ? acc[t][e] * p.scale : -INFINITY;
        m = fmaxf(m, z[e]);
        if (v + e < p.vocab && p.v0 + v + e == label) p.at_label[row] = z[e];
      }
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float from = m == -INFINITY ? 0.0f : m;
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) s += exp2_fast((z[e] - from) * kLog2e);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (g == 0) red[wave * 16 * NT + 16 * t + i] = float2{m, s};
    }
    __syncthreads();
    const int row = threadIdx.x;
    if (row < 16 * NT && row < rows) {
      float m = -INFINITY, s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) m = fmaxf(m, red[w * 16 * NT + row].x);
      const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float2 r = red[w * 16 * NT + row];
        s += r.y * exp2_fast((r.x - from) * kLog2e);
      }
      p.part[(int64_t)row * p.parts + p.v0 / kEntries + blockIdx.x] = float2{m, s};
    }
  } else {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t row = 16 * t + i;
      const bool in = row < rows;
      const HeadColumn c = in ? p.cols[row] : HeadColumn{0.0f, 0.0f, 0.0f, -1};
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        pr[e] = in && v + e < p.vocab
                    ? exp2_fast(fmaf(acc[t][e], p.scale, -c.most) * kLog2e) * c.over
                    : 0.0f;
      // The label's probability is none of P's entries: p - 1 stays in fp32.
      const int64_t away = c.label - (p.v0 + v);
      const bool mine = in && away >= 0 && away < 4;
      const int hot = mine ? (int)away : -1;
      float rest = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (hot == e) {
          rest = pr[e] - 1.0f;
          pr[e] = 0.0f;
        }
      if (mine && p.rest) p.rest[row] = rest;
      if (p.P && in && v < p.p_plane) store_terms(p.P + row * p.ldp + v, p.p_plane, p.p_terms, pr);
      if (p.Q) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          pr[e] = (hot == e ? rest : pr[e]) * c.factor;
        store_terms(p.Q + row * p.ldq + v, p.q_plane, p.q_terms, pr);
      }
    }
    if (p.Q) {  // the product behind it reduces over two whole steps of rows
      const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = NT; t < 4; ++t)
        store_terms(p.Q + (16 * t + i) * p.ldq + v, p.q_plane, p.q_terms, none);
    }
  }
}

// A workgroup a row: its parts joined.
__global__ __launch_bounds__(256) void head_few_loss_kernel(const float2* part, int64_t parts,
                                                            const float* at_label,
                                                            const void* labels, bool ids64,
                                                            int64_t M, int64_t V, float* loss,
                                                            float* stats) {
  __shared__ float red[2 * kMostReduced * 4];
  const int64_t row = blockIdx.x;
  const int64_t label = load_index(labels, ids64, row);
  const bool live = label >= 0 && label < V;
  float m[1] = {-INFINITY}, s[1] = {0.0f};
  if (live) {
#pragma unroll 4
    for (int64_t k = threadIdx.x; k < parts; k += 256) {
      const float2 v = part[row * parts + k];
      const float to = fmaxf(m[0], v.x), from = to == -INFINITY ? 0.0f : to;
      s[0] = s[0] * exp2_fast((m[0] - from) * kLog2e) + v.y * exp2_fast((v.x - from) * kLog2e);
      m[0] = to;
    }
  }
  int par = 0;
  const float mine = m[0];
  group_reduce<256, 1>(m, red, 4, par, OpMax());
  const float from = m[0] == -INFINITY ? 0.0f : m[0];
  s[0] *= exp2_fast((mine - from) * kLog2e);
  group_reduce<256, 1>(s, red, 4, par, OpSum());
  if (threadIdx.x) return;
  const float L = logf(s[0]);
  loss[row] = live ? L + (m[0] - at_label[row]) : 0.0f;
  if (stats) {
    stats[row] = live ? m[0] : 0.0f;
    stats[M + row] = live ? L : 0.0f;
  }
}

// Eight waves, or two where those leave CUs idle: a workgroup's loads reach some
// 35 GB/s on a CU (2048 x 5696, 4 rows: 16 workgroups of eight waves 44 us).
template <int NT, bool kProbs>
hipError_t few_rows(const HeadFew& a, hipStream_t st) {
  // Probabilities are written up to two whole steps of the product behind them.
  const int64_t to = kProbs ? (a.vocab + 63) / 64 * 64 : a.vocab;
  const dim3 grid((unsigned)((to + a.entries - 1) / a.entries));
  if (a.entries == 128)
    hipLaunchKernelGGL((head_few_kernel<NT, 8, kProbs>), grid, dim3(512), 0, st, a);
  else
    hipLaunchKernelGGL((head_few_kernel<NT, 2, kProbs>), grid, dim3(128), 0, st, a);
  return hipGetLastError();
}

template <bool kProbs>
hipError_t few(const HeadFew& a, hipStream_t st) {
  if (a.M <= 16) return few_rows<1, kProbs>(a, st);
  return a.M <= 32 ? few_rows<2, kProbs>(a, st) : few_rows<4, kProbs>(a, st);
}

}  // namespace

hipError_t launch_head_few_stats(const HeadFew& a, hipStream_t st) { return few<false>(a, st); }
hipError_t launch_head_few_probs(const HeadFew& a, hipStream_t st) { return few<true>(a, st); }

hipError_t launch_head_few_loss(const float2* part, int64_t parts, const float* at_label,
                                const void* labels, bool ids64, int64_t M, int64_t V, float* loss,
                                float* stats, hipStream_t st) {
  hipLaunchKernelGGL(head_few_loss_kernel, dim3((unsigned)M), dim3(256), 0, st, part, parts, at_label,
                     labels, ids64, M, V, loss, stats);
  return hipGetLastError();
}

}  // namespace qlora
