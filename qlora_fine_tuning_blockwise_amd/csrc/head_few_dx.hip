// The gradient of a few rows through the vocabulary head on gfx950, one pass over
// W: with the statistics of the forward a probability is final as soon as its
// logit is, so that a row of W serves the logit and its part of the gradient while
// it is on the chip.
//   P = exp(scale x W' - m) exp(-L), but 0 at the label;  sum = P W
//   dX = dloss scale (sum + (p_label - 1) W_label), the latter in fp32
//
// Memory bounds it. A workgroup takes 16 entries of the vocabulary at a time, a
// wave a slice of the hidden size: its 16 rows of W come straight from memory into
// registers, where they lie as the logits' product needs them; the eight waves'
// parts of the logits are joined through LDS, and W goes through a few KB of LDS
// that only its wave uses, to be read down its rows (transposing reads) for the
// gradient's product. Logits leave the matrix units in the order in which that
// product takes the probabilities. A part of W is requested for the next 16
// entries as soon as it has left its registers. The sums stay in registers to the
// end; each workgroup writes them once, and a second kernel joins them in order.
// 8 rows, 32000 x 4096: 57 us and 7 us for the join (the logits in one pass over W
// and the product in another: 48 and 46 us); 1 row of 128000 x 4096: the call takes
// 190 us, 5.5 TB/s. The loop has no register to spare at 4096 columns: what it can
// form anew it does not keep, since a register that is spilled is read back behind
// W's loads and waits for them (16 rows 123 instead of 84 us).
#include <type_traits>

#include "head_terms.h"

namespace qlora {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

__device__ __forceinline__ u32x4_t words(const Vec<true, 8>& v) {
  return u32x4_t{v.w[0], v.w[1], v.w[2], v.w[3]};
}

constexpr int kWaves = 8, kEntries = 16;

// NR: rows of x that LDS holds. NF: fragments of 32 columns of a wave's slice.
template <int NR, int NF, int kTerms>
__global__ __launch_bounds__(64 * kWaves, 1) void head_few_dx_kernel(HeadFewDx p) {
  constexpr int kSlice = 32 * NF, kWidth = kWaves * kSlice;
  // Fragments that go through LDS at a time (of 8 all at once: 8 rows, 32000 x 2048 48
  // instead of 41.5 us).
  constexpr int kStage = NR * NF > 128 ? 2 : NF < 16 ? 4 : 8;
  // The first of them as soon as the logits' product has read them: the waves' meeting
  // then finds the next loads in flight (8 rows, 32000 x 4096: 5 us). Of 2 fragments that is no
  // gain (16 rows: 3 us slower).
  constexpr bool kEarly = kStage > 2;
  // 16-byte part c of a row r lies at c ^ (r & 7), in both.
  __shared__ __attribute__((aligned(16))) uint16_t xs[NR * kWidth];
  __shared__ __attribute__((aligned(16))) uint16_t stages[kWaves][kEntries * 32 * kStage];
  __shared__ f32x4_t logits[2][kWaves][64];
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int live = __builtin_amdgcn_readfirstlane(*p.count);
  if (live == 0) return;
  const int K = (int)p.K, k0 = wave * kSlice;
  const int chunks = (int)((p.V + kEntries - 1) / kEntries);
  Vec<true, 8> w[NF];
  const bool whole = k0 + kSlice <= K;
  const auto load = [&](int c, int f0, auto count) __attribute__((always_inline)) {
    constexpr int kCount = decltype(count)::value;
    const int64_t v = (int64_t)c * kEntries + i;
    const uint16_t* from = p.W + (v < p.V ? v : p.V - 1) * p.ldw;
    from += k0 + 8 * g;
    if (whole) {
#pragma unroll
      for (int f = 0; f < kCount; ++f) w[f0 + f] = load_vec<true, 8, true>(from + 32 * (f0 + f));
    } else {  // behind the hidden size its last columns, which x has zeros for
      int last = K - 8 - (k0 + 8 * g);
      asm volatile("" : "+v"(last));  // the places are formed here, not kept through the loop
#pragma unroll
      for (int f = 0; f < kCount; ++f) w[f0 + f] = load_vec<true, 8, true>(from + min(32 * (f0 + f), last));
    }
  };
  // Of this lane's row, the label counted from its four entries.
  float most = 0.0f, over = 0.0f, at_label = 0.0f;
  int label = -kEntries;
  if (i < live) {
    const HeadColumn col = p.cols[i];
    most = col.most, over = col.over, label = col.label - 4 * g;
  }
  bool found = false;  // at_label is the label's probability
  int c = blockIdx.x;
  load(c, 0, std::integral_constant<int, NF>());
  // This wave's slice of the live rows, which no other wave reads.
#pragma unroll 4
  for (int at = lane; at < NR * 4 * NF; at += 64) {
    const int r = at / (4 * NF), part = at % (4 * NF), k = k0 + 8 * part;
    const Vec<true, 8> v = r < live && k < K ? load_vec<true, 8>(p.x + (int64_t)p.map[r] * p.ldx + k)
                                             : zero_vec<true, 8>();
    *reinterpret_cast<u32x4_t*>(&xs[r * kWidth + k0 + 8 * (part ^ (r & 7))]) = words(v);
  }
  // Of what is read and written, the places in the first parts; 64 elements on, the
  // swizzle is the same.
  const uint16_t* const xrow[2] = {&xs[(i % NR) * kWidth + k0 + 8 * (g ^ (i & 7))],
                                   &xs[(i % NR) * kWidth + k0 + 8 * ((4 + g) ^ (i & 7))]};
  uint16_t* const stage = stages[wave];
  uint16_t* const put[2] = {stage + i * (32 * kStage) + 8 * (g ^ (i & 7)),
                            stage + i * (32 * kStage) + 8 * ((4 + g) ^ (i & 7))};
  const int row = 4 * g + (i >> 2);
  const uint16_t* get[4];
#pragma unroll
  for (int t = 0; t < 4; ++t)
    get[t] = stage + row * (32 * kStage) + 4 * (i & 1) + 8 * ((2 * t + ((i >> 1) & 1)) ^ (row & 7));
  f32x4_t acc[2 * NF];  // of 16 columns each: element e is column 4g + e, live row i
#pragma unroll
  for (int t = 0; t < 2 * NF; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  // Waited for here: in the loop their wait would be one for the next part of W too.
  asm volatile("" : "+v"(most), "+v"(over), "+v"(label));
  for (int turn = 0; c < chunks; turn ^= 1) {
    f32x4_t s[2] = {f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}};
    const int next = c + gridDim.x;
    const auto into_stage = [&](int f0) __attribute__((always_inline)) {
#pragma unroll
      for (int f = 0; f < kStage; ++f)
        *reinterpret_cast<u32x4_t*>(put[f & 1] + 64 * (f >> 1)) = words(w[f0 + f]);
      if (next < chunks) load(next, f0, std::integral_constant<int, kStage>());
    };
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      s[f & 1] = mfma_16x16x32(words(w[f]), *reinterpret_cast<const u32x4_t*>(xrow[f & 1] + 64 * (f >> 1)),
                               s[f & 1]);
      if (kEarly && f == kStage - 1) into_stage(0);
    }
    // Two buffers in turn: one is written again two meetings after it was read.
    logits[turn][wave][lane] = s[0] + s[1];
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    f32x4_t z = logits[turn][0][lane];
#pragma unroll
    for (int o = 1; o < kWaves; ++o) z += logits[turn][o][lane];
    // Element e is entry 4g + e, live row i (past the live rows anything: what becomes
    // of it stays in its column, which is not stored).
    const int first = c * kEntries, left = (int)min(p.V - first, (int64_t)kEntries) - 4 * g;
    float pr[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      pr[e] = exp2_fast(fmaf(z[e], p.scale, -most) * kLog2e) * over;
      pr[e] = e < left ? pr[e] : 0.0f;
      const bool hot = label == first + e;
      at_label = hot ? pr[e] : at_label;
      found |= hot;
      pr[e] = hot ? 0.0f : pr[e];
    }
    s16x4_t prob[kTerms];
    prob[0] = __builtin_bit_cast(s16x4_t, term_of<0>(pr[0], pr[1], pr[2], pr[3]));
    if constexpr (kTerms > 1) {
      prob[1] = __builtin_bit_cast(s16x4_t, term_of<1>(pr[0], pr[1], pr[2], pr[3]));
      prob[2] = __builtin_bit_cast(s16x4_t, term_of<2>(pr[0], pr[1], pr[2], pr[3]));
    }
    c = next;
#pragma unroll
    for (int f0 = 0; f0 < NF; f0 += kStage) {
      if (f0 || !kEarly) into_stage(f0);
#pragma unroll
      for (int t = 0; t < 2 * kStage; ++t) {
        const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)(get[t & 3] + 64 * (t >> 2)));
#pragma unroll
        for (int n = 0; n < kTerms; ++n)
          acc[2 * f0 + t] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a, prob[n], acc[2 * f0 + t], 0, 0, 0);
      }
    }
  }
  if (wave == 0 && found) p.rest[i] = at_label - 1.0f;  // all waves have the same
  // [workgroup][16 columns][row][column of 16]
  if (i >= live) return;
  const int all = (K + 15) / 16;
  float* to = p.part + (((int64_t)blockIdx.x * all + k0 / 16) * p.M + i) * 16 + 4 * g;
#pragma unroll
  for (int t = 0; t < 2 * NF; ++t)
    if (k0 / 16 + t < all) *reinterpret_cast<f32x4_t*>(to + (int64_t)t * p.M * 16) = acc[t];
}

// 32 groups of four columns of a row a workgroup, each in eight ranges of the
// workgroups' sums; rows without loss are zero.
template <bool kBf16>
__global__ __launch_bounds__(256) void head_few_dx_join_kernel(HeadFewDx p) {
  __shared__ f32x4_t red[8][32];
  const int range = threadIdx.x / 32;
  const int live = *p.count, M = (int)p.M, all = ((int)p.K + 15) / 16 * M * 4;
  const int u = (int)blockIdx.x * 32 + (int)(threadIdx.x % 32);
  const int m = u / 4 % M, k = u / (4 * M) * 16 + u % 4 * 4;
  f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
  if (u < all && m < live) {
    const float* from = p.part + ((int64_t)range * all + u) * 4;
#pragma unroll 8
    for (int b = range; b < p.groups; b += 8, from += (int64_t)all * 32)
      sum += *reinterpret_cast<const f32x4_t*>(from);
  }
  red[range][threadIdx.x % 32] = sum;
  __syncthreads();
  if (range || u >= all || k >= p.K) return;
  const auto store = [&](int64_t to, const float (&v)[4]) {
    store_vec<kBf16, 4>(static_cast<elem_t<kBf16>*>(p.dX) + to * p.lddx + k, v);
  };
  if (p.inv[m] < 0) {
    const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    store(m, none);
  }
  if (m >= live) return;
#pragma unroll
  for (int r = 1; r < 8; ++r) sum += red[r][threadIdx.x];
  const HeadColumn col = p.cols[m];
  const float rest = p.rest[m];
  float at_label[4], v[4];
  to_float<true, 4>(load_vec<true, 4>(p.W + (int64_t)col.label * p.ldw + k), at_label);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = fmaf(rest, at_label[e], sum[e]) * col.factor;
  store(p.map[m], v);
}

template <int NR, int kTerms>
hipError_t rows_of(const HeadFewDx& a, hipStream_t st) {
  const dim3 grid((unsigned)a.groups), block(64 * kWaves);
  if (a.K <= 1024)
    hipLaunchKernelGGL((head_few_dx_kernel<NR, 4, kTerms>), grid, block, 0, st, a);
  else if (a.K <= 2048)
    hipLaunchKernelGGL((head_few_dx_kernel<NR, 8, kTerms>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((head_few_dx_kernel<NR, 16, kTerms>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_head_few_dx(const HeadFewDx& a, bool bf16, hipStream_t st) {
  hipError_t e;
  if (a.M <= 8)
    e = bf16 ? rows_of<8, 1>(a, st) : rows_of<8, 3>(a, st);
  else
    e = bf16 ? rows_of<16, 1>(a, st) : rows_of<16, 3>(a, st);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)(((a.K + 15) / 16 * a.M * 4 + 31) / 32));
  if (bf16)
    hipLaunchKernelGGL(head_few_dx_join_kernel<true>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(head_few_dx_join_kernel<false>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace qlora
