// The loss of the vocabulary head on gfx950, without keeping the logits.
//
// For a row x[K], a head W[V, K], a label and a scale s:
//   z_v  = s sum_k x_k W_vk,  m = max z,  L = log sum_v exp(z_v - m)
//   loss = L + (m - z_label)
//   p_v  = exp(z_v - m) exp(-L)
//   dX   = dloss s (sum over v != label of p_v W_v + (p_label - 1) W_label)
//   dW_v = sum over the rows of dloss s (p_v - [v = label]) x
// A row whose label lies outside of the vocabulary carries no loss.
//
// The rows that carry loss are gathered first (in a padded or masked batch a
// half of the rows and more carry none), so that the products run over live
// rows only; how many there are is known on the device alone, and every kernel
// reads it there.
//
// Forward: one product of the matrix units. A tile of 256 entries of the
// vocabulary by 256 rows keeps its logits in registers and leaves each row's
// largest one and the sum of exponentials taken from it, 8 bytes for 256 logits.
// Backward, in pieces of the vocabulary: the logits are formed again tile by
// tile and leave as probabilities in bf16, then the piece's part of the rows'
// gradients and of W's is a product each.
//
// Roundings to bf16: the products' operands have to be bf16. The label's
// probability never is one: its entry of dX's product is 0, p_label - 1 is formed
// in fp32 and multiplied by the label's row of W in fp32 at the end. What is
// rounded (2^-8 of a probability at most) are the other entries, which add up to
// 1 - p_label: dX is as near for a label of probability 0.999 as for one of 0.5
// (where p_label was rounded with the others and 1 subtracted afterwards, 0.9965
// cost a fourth of dX and 0.9986 all of it). dW takes p_label - 1 itself, rounded
// once. For fp32 gradients a value is split into three bf16 numbers (24 bits, as
// fp32 has) and the products have three times the terms.
//
// The tile loop is the dense stage's of the linear layer (gemm_nt.hip has its
// description): 256 x 256 tiles, four waves of 128 x 128 on
// v_mfma_f32_32x32x16_bf16, operands by direct-to-LDS loads, a in a ring of three
// pairs of steps, b in a ring of four steps. The matrix units bound it: 1536 rows,
// 128000 x 4096, forward 1250 us (1290 TFLOP/s), dX 2740 us (1175 TFLOP/s of two
// products); 1500 rows, 32003 x 2048: logits 202, dX 165, dW 206 us. A step of a
// tile takes 0.55 us, its first loads and its end 9 us (statistics) to 11 us. The
// build for dX keeps 16 registers in scratch, outside of the steps.
#include <type_traits>

#include "head_terms.h"

namespace qlora {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

__device__ __forceinline__ int ceil_tile(int64_t n) { return (int)((n + kTile - 1) / kTile); }

// Splits of the live rows' gradient along its reduction of `pairs` pairs of steps:
// those with the least rounds of 256 workgroups, where a workgroup takes its
// share of the reduction and the time of 50 pairs besides (first loads, 256 KB of
// sums read and written, and the clock, which falls as more CUs multiply: 1536 x
// 4096 in pieces of 500 pairs takes as long in 192 workgroups of two splits as in
// 480 of five, and 3% longer in 768 of eight), and a split's sums half a pair to be
// joined. One tile of 1542 pairs is best in many (127 rows, 32896 x 64, fp32: 106 us of
// 16 splits, 69 of 47, 65 of 64), four of 313 pairs in fewer (20 rows, 20000 x 1024:
// 42 us of 16, 40 of 21, 46 of 64). A wave weighs all of them at once.
__device__ __forceinline__ int dx_splits(int tiles, int pairs) {
  const int s = (threadIdx.x & 63) + 1;
  int best = 0x7FFFFFFF;  // the cost, then the number of splits
  if (s == 1 || (s <= kMostSplits && tiles * s <= kMostSums && s <= pairs)) {
    const int64_t cost = (int64_t)((tiles * s + 255) / 256) * ((pairs + s - 1) / s + 50) + s / 2;
    best = (int)(cost < (1 << 24) ? cost : (1 << 24) - 1) * kMostSplits + (s - 1);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) best = min(best, __shfl_xor(best, d));
  return best % kMostSplits + 1;
}
static_assert(kMostSplits <= 64, "a lane each");

// ------------------------------------------------------------- live rows
constexpr int kRowThreads = 1024;

// One workgroup: a thread counts the live rows of its run of rows, the counts
// are summed over the threads, and it writes its own.
__global__ __launch_bounds__(kRowThreads) void head_rows_kernel(HeadRows a) {
  __shared__ int32_t sums[kRowThreads / 64];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t per = (a.M + kRowThreads - 1) / kRowThreads;
  const int64_t first = t * per < a.M ? t * per : a.M;
  const int64_t last = first + per < a.M ? first + per : a.M;
  const auto live = [&](int64_t m, int64_t& label) {
    label = load_index(a.labels, a.ids64, m);
    return label >= 0 && label < a.V && (!a.dloss || a.dloss[m] != 0.0f);
  };
  int32_t n = 0;
  int64_t label;
  for (int64_t m = first; m < last; ++m) n += live(m, label);
  int32_t upto = n;  // inclusive over the wave
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  int32_t before = 0, all = 0;
  for (int w = 0; w < kRowThreads / 64; ++w) {
    if (w < wave) before += sums[w];
    all += sums[w];
  }
  int32_t j = before + upto - n;
  for (int64_t m = first; m < last; ++m) {
    const bool is = live(m, label);
    a.inv[m] = is ? j : -1;
    if (!is) continue;
    a.map[j] = (int32_t)m;
    HeadColumn c{0.0f, 0.0f, 0.0f, (int32_t)label};
    if (a.stats) {
      c.most = a.stats[m];
      c.over = exp2_fast(-a.stats[a.M + m] * kLog2e);
      c.factor = a.dloss[m] * a.scale;
    }
    a.cols[j++] = c;
  }
  const int32_t end = (all + kTile - 1) / kTile * kTile;
  for (int32_t k = all + t; k < end; k += kRowThreads) a.cols[k] = HeadColumn{0.0f, 0.0f, 0.0f, -1};
  if (t >= 64) return;
  const int splits = a.pairs ? dx_splits(max(ceil_tile(all) * ceil_tile(a.K), 1), a.pairs) : 1;
  if (t == 0) {
    a.count[0] = all;
    a.count[1] = splits;
  }
}

// ------------------------------------------------------------- b operands
// A thread takes 8 columns of a row: 16 bytes of a step.
__global__ __launch_bounds__(256) void head_pack_rows_kernel(const uint16_t* src, int64_t ld,
                                                             const int32_t* map,
                                                             const int32_t* count, int64_t rows,
                                                             int64_t K, uint16_t* out) {
  const int64_t steps = (K + kStep - 1) / kStep, vecs = steps * 4;
  const int64_t n = count ? *count : rows;
  const int64_t end = (n + kTile - 1) / kTile * kTile;
  const int64_t at = linear_thread();
  const int64_t j = at / vecs, c = at - j * vecs;
  if (j >= end) return;
  Vec<true, 8> v = zero_vec<true, 8>();
  if (j < n) {
    const uint16_t* p = src + (map ? (int64_t)map[j] : j) * ld + 8 * c;
    const int have = count_below<8>(8 * c, K);
    v = have == 8 ? load_vec<true, 8>(p) : load_part<true, 8>(p, have);
  }
  uint16_t* to = out + ((j / kTile) * steps + c / 4) * (kTile * kStep) + (j % kTile) * kStep + (c % 4) * 8;
  *reinterpret_cast<u32x4_t*>(to) = u32x4_t{v.w[0], v.w[1], v.w[2], v.w[3]};
}

// A thread copies 8 columns of a row with zeros behind its K columns: rows map[j] of
// src for the live ones, *count, and whole rows of zeros up to two whole steps; or
// all rows, where any is live.
__global__ __launch_bounds__(256) void head_copy_kernel(const uint16_t* src, int64_t ld,
                                                        const int32_t* map, const int32_t* count,
                                                        int64_t rows, int64_t K, int64_t Kp,
                                                        uint16_t* out) {
  const int64_t live = *count, n = map ? live : live ? rows : 0;
  const int64_t end = map ? (n + 2 * kStep - 1) / (2 * kStep) * (2 * kStep) : n;
  const int64_t vecs = Kp / 8, at = linear_thread();
  const int64_t r = at / vecs, c = (at - r * vecs) * 8;
  if (r >= end) return;
  Vec<true, 8> v = zero_vec<true, 8>();
  if (r < n) {
    const int have = count_below<8>(c, K);
    const uint16_t* p = src + (map ? (int64_t)map[r] : r) * ld + c;
    v = have == 8 ? load_vec<true, 8>(p) : load_part<true, 8>(p, have);
  }
  *reinterpret_cast<u32x4_t*>(out + at * 8) = u32x4_t{v.w[0], v.w[1], v.w[2], v.w[3]};
}

// Zeros, two elements of 16 bits a thread; an odd number of them ends in one.
__global__ __launch_bounds__(256) void head_zero_kernel(uint32_t* p, int64_t halves) {
  const int64_t i = linear_thread();
  if (2 * i + 1 < halves)
    p[i] = 0u;
  else if (2 * i < halves)
    reinterpret_cast<uint16_t*>(p)[2 * i] = 0;
}

// ------------------------------------------------------------------ tiles
constexpr int kOp = kTile * kStep;  // bf16 elements of one step of an operand (16 KB)
constexpr int kPair = 2 * kOp;      // of two steps
constexpr int kGroup = 4;           // tile rows per group in the tile order

// Place of workgroup `wg` in an order of T: workgroups are dealt to the eight
// XCDs round robin, and each XCD gets a contiguous range of the order.
__device__ __forceinline__ int xcd_order(int wg, int T) {
  const int xcd = wg & 7, per = T >> 3, extra = T & 7;
  return xcd * per + (xcd < extra ? xcd : extra) + (wg >> 3);
}

// The order walks groups of kGroup tile rows column by column: the tiles that run
// together on an XCD share row panels of a and column panels of b.
__device__ __forceinline__ void tile_of(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int group = t / (kGroup * tiles_n);
  const int first = group * kGroup;
  const int rows = tiles_m - first < kGroup ? tiles_m - first : kGroup;
  const int in = t - group * kGroup * tiles_n;
  tm = first + in % rows;
  tn = in / rows;
}

// At most n vector-memory operations in flight, no LDS operation.
template <int n>
__device__ __forceinline__ void wait_vmem_lgkm0() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (0x7 << 4));
  __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ const void* uniform_ptr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const void*>(((uint64_t)hi << 32) | lo);
}

template <int S, int N, typename T>
__device__ __forceinline__ T* pick(T* const (&arr)[N]) {
  static_assert(S >= 0 && S < N, "stage index");
  return arr[S];
}

// kTerms: of kProbs those that are written at most; of kDw 1 where bf16 sums are all
// that is written.
constexpr int kStats = 0, kProbs = 1, kDx = 2, kDw = 3;

__device__ __forceinline__ int64_t whole_pairs(int64_t n) { return (n + 2 * kStep - 1) / (2 * kStep) * (2 * kStep); }

// Rows of a matrix from one of its columns on: their first byte, and the bytes up
// to the matrix's end.
struct Window {
  const void* p;
  int size;
};

typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// A fragment of 8 reduction elements of one column from a tile that lies with
// its reduction along the rows: in each group of 16 lanes the transposing read
// takes 4 rows of 16 columns and gives each lane a column. p: the lane's 8 bytes
// of the first four rows; the other four lie 4 rows on.
__device__ __forceinline__ u32x4_t read_columns(const uint16_t* p) {
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * kTile));
  const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
  return u32x4_t{a[0], a[1], b[0], b[1]};
}

// A wave's 128 x 128 block of dW (rows of the block are columns of dW) by way of
// its 16 KB of LDS: 16-byte part c of row i at c ^ i. In LDS the sums are bf16
// where that is all that is written, 64 rows of dW at a time; fp32 (kWide) where dW
// is, or where they are added to it, 32 rows at a time.
template <bool kBf16, bool kWide>
__device__ __forceinline__ void put_dw(const f32x16_t (&acc)[4][4], uint16_t* own,
                                       const HeadTiles& p, int64_t k0, int64_t v0, int lane) {
  constexpr int E = kWide ? 4 : 8, kParts = 128 / E;
  constexpr int kPasses = kWide ? 4 : 2, kRows = 128 / kPasses;
  const int i = lane & 31, h = lane >> 5;
  const int part = lane % kParts, have = count_below<E>(k0 + E * part, p.K);
  const int rows = have <= 0 ? 0 : (int)min(p.vocab - v0, (int64_t)128);
  const int row0 = lane / kParts;
  elem_t<kBf16>* to = static_cast<elem_t<kBf16>*>(p.dW) + (p.v0 + v0 + row0) * p.K + k0 + E * part;
  char* const lds = reinterpret_cast<char*>(own);
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
#pragma unroll
    for (int n = 0; n < 4 / kPasses; ++n) {
      char* const at = lds + (32 * n + i) * (kParts * 16);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16_t& v = acc[mt][4 / kPasses * pass + n];
          if constexpr (kWide)
            *reinterpret_cast<f32x4_t*>(at + 16 * ((8 * mt + 2 * g + h) ^ i)) =
                f32x4_t{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
          else
            *reinterpret_cast<u32x2_t*>(at + 16 * ((4 * mt + g) ^ (i & 15)) + 8 * h) =
                u32x2_t{pack_bf16x2(v[4 * g], v[4 * g + 1]), pack_bf16x2(v[4 * g + 2], v[4 * g + 3])};
        }
    }
#pragma unroll 2
    for (int r = row0; r < kRows; r += 64 / kParts, to += (64 / kParts) * p.K) {
      const u32x4_t q = *reinterpret_cast<const u32x4_t*>(lds + (r * kParts + (part ^ (r & (kParts - 1)))) * 16);
      if (kRows * pass + r >= rows) continue;
      float v[E];
      if constexpr (kWide) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(q[e]);
        if (p.accumulate) {
          float old[E];
          to_float<kBf16, E>(have == E ? load_vec<kBf16, E>(to) : load_part<kBf16, E>(to, have), old);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] += old[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e & 1 ? bf16_hi(q[e / 2]) : bf16_lo(q[e / 2]);
      }
      if (have == E)
        store_vec<kBf16, E>(to, v);
      else
        store_part<kBf16, E>(to, v, have);
    }
  }
}

// The tile loop. Operands come in three forms:
//   rows    (a of kStats, kProbs, kDx): row-major, the reduction along a row. LDS
//           has three slots of a 256 x 64 tile (a pair of steps), 16-byte chunk c
//           of row r at c ^ ((r >> 1) & 7).
//   steps   (b of kStats, kProbs): [tile][step][256][32]. Four stages of a 256 x
//           32 tile, chunk c of row r at c ^ ((r >> 2) & 3).
//   columns (b of kDx, both of kDw): row-major, the reduction down the rows, as
//           W, the live rows and the logits' gradients lie: no transposed copy is
//           made. Four stages of a 32 x 256 tile, chunk c of row r at c ^ 2 g(r)
//           with g = 0, 5, 2, 7 for r % 4: the 4 rows by 32 bytes that 16 lanes
//           read lie in different banks, as do the 64 bytes of 32 lanes.
// A pair of slots is loaded two pairs ahead, a stage three steps.
template <int kMode, int kTerms = 1>
__global__ __launch_bounds__(256, 1) void head_tile_kernel(HeadTiles p) {
  constexpr bool kACols = kMode == kDw, kBCols = kMode == kDx || kMode == kDw;
  __shared__ __attribute__((aligned(1024))) uint16_t sa0[kPair];
  __shared__ __attribute__((aligned(1024))) uint16_t sa1[kPair];
  __shared__ __attribute__((aligned(1024))) uint16_t sa2[kACols ? kOp : kPair];
  __shared__ __attribute__((aligned(1024))) uint16_t sa3[kACols ? kOp : 8];
  __shared__ __attribute__((aligned(1024))) uint16_t sb0[kOp];
  __shared__ __attribute__((aligned(1024))) uint16_t sb1[kOp];
  __shared__ __attribute__((aligned(1024))) uint16_t sb2[kOp];
  __shared__ __attribute__((aligned(1024))) uint16_t sb3[kOp];
  uint16_t* const sa[4] = {sa0, sa1, sa2, sa3};  // columns: four stages in the first 16 KB of each
  uint16_t* const sb[4] = {sb0, sb1, sb2, sb3};
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // wave-uniform
  const int wm = w >> 1, wn = w & 1;
  const int live = __builtin_amdgcn_readfirstlane(*p.count);
  // Rows, columns and steps of this product; half: steps of one term.
  const int64_t M = kMode == kDx ? live : kMode == kDw ? p.K : p.vocab;
  const int64_t N = kMode == kStats || kMode == kProbs ? live : kMode == kDx ? p.K : p.vocab;
  const int half = kMode == kDx   ? (int)(whole_pairs(p.vocab) / kStep)
                   : kMode == kDw ? (int)(whole_pairs(live) / kStep)
                                  : (int)p.steps;
  const int all = kMode == kDx ? half * p.p_terms : kMode == kDw ? half * p.q_terms : half;
  const int tiles_m = ceil_tile(M), tiles_n = ceil_tile(N), tiles = tiles_m * tiles_n;
  const int splits = kMode == kDx ? __builtin_amdgcn_readfirstlane(p.count[1]) : 1;
  if ((int)blockIdx.x >= tiles * splits) return;
  // Each XCD (blockIdx.x % 8) gets a contiguous range of the splits' tiles.
  int order = xcd_order((int)blockIdx.x, tiles * splits), tm, tn;
  const int split = kMode == kDx ? order / tiles : 0;
  tile_of(order - split * tiles, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * kTile, n0 = (int64_t)tn * kTile;
  // A split has a whole number of pairs of steps.
  const int per = kMode == kDx ? (all / 2 + splits - 1) / splits * 2 : all;
  const int ks0 = split * per;
  const int nsteps = kMode == kDx ? min(per, all - ks0) : all;

  // Where the fragments of this wave lie in the tile. A wave takes 128 x 128; along the
  // live rows that is every other 32 of them, so that a tile that ends early is
  // less work for all waves.
  const auto a_at = [&](int mt) { return kMode == kDx ? 64 * mt + 32 * wm : 32 * mt + 128 * wm; };
  const auto b_at = [&](int nt) { return kMode == kStats || kMode == kProbs ? 64 * nt + 32 * wn : 32 * nt + 128 * wn; };
  f32x16_t acc[4][4];
#pragma unroll
  for (int mt = 0; mt < 4; ++mt)
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[mt][nt][e] = 0.0f;

  if (nsteps > 0) {
    const int lane = threadIdx.x & 63, i = lane & 31, h = lane >> 5;
    const int npairs = (nsteps + 1) / 2;
    const int64_t k0 = (int64_t)ks0 * kStep;
    typedef __attribute__((address_space(3))) void lds_void;
    // Direct-to-LDS roles. rows: wave w loads rows 64w + 8q + L/8 (q = 0..7) of
    // each pair, lane L at LDS position L%8. steps: wave w loads windows 4w .. 4w+3 (16 rows each) of each step.
    // Of both, rows past the matrix lie past the buffer and read zeros. columns: wave w loads rows 8w + 2q + L/32 (q = 0..3)
    // of each step, lane L at position L%32.
    constexpr uint32_t kNoRow = 0x80000000u;
    uint32_t aoff[8], boff[4];
    const int crow = 8 * w + (lane >> 5);  // of the first load; the others 2 rows on each
    const auto chunk_of = [&](int row) { return (lane & 31) ^ (2 * ((row & 3) ^ ((row & 1) << 2))); };
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = 64 * w + 8 * q + (lane >> 3);
      const int c = (lane & 7) ^ ((row >> 1) & 7);
      if constexpr (!kACols)
        aoff[q] = m0 + row < M ? (uint32_t)(row * p.lda * 2 + 16 * c) : kNoRow;
      else if (q < 4)
        aoff[q] = (uint32_t)((crow + 2 * q) * p.lda * 2 + 16 * chunk_of(crow + 2 * q));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 16 * (4 * w + j) + (lane >> 2);
      const int c = (lane & 3) ^ ((row >> 2) & 3);
      if constexpr (kBCols)
        boff[j] = (uint32_t)((crow + 2 * j) * p.ldb * 2 + 16 * chunk_of(crow + 2 * j));
      else
        boff[j] = n0 + row < N ? (uint32_t)(row * 64 + 16 * c) : kNoRow;
    }
    // rows: a ends with its last row's last step; what a final odd pair has past
    // it in that row reads zeros (in other rows the next row; it is not used).
    const int64_t a_bytes = min(((M - 1 - m0) * p.lda + (int64_t)(all - ks0) * kStep) * 2, (int64_t)0x7FFFFFFF);
    const __amdgpu_buffer_rsrc_t ares = __builtin_amdgcn_make_buffer_rsrc(
        (void*)uniform_ptr(p.a + m0 * p.lda + k0), (short)0, (int)a_bytes, 0x00020000);
    const __amdgpu_buffer_rsrc_t bres = __builtin_amdgcn_make_buffer_rsrc(
        (void*)uniform_ptr(p.b + (int64_t)tn * p.b_steps * kOp), (short)0, (int)0x7FFFFFFF, 0x00020000);
    // columns: the rows of step ks, 32 of them, as a buffer that ends with the
    // matrix (a step may pass its last row: zeros).
    const auto rows_of = [&](const uint16_t* m, int64_t ld, int64_t col, int64_t rows, int64_t width, int ks) {
      const int64_t r = (int64_t)ks * kStep;
      const int64_t left = ((rows - 1 - r) * ld + width - col) * 2;
      const int size = left < 0 || r >= rows ? 0 : left > 0x7FFFFFFF ? 0x7FFFFFFF : (int)left;
      return Window{uniform_ptr(m + r * ld + col), size};
    };
    const auto dma_cols = [&](const Window& from, uint32_t off, int q, uint16_t* stage) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          __builtin_amdgcn_make_buffer_rsrc((void*)from.p, (short)0, from.size, 0x00020000),
          (lds_void*)(stage + (8 * w + 2 * q) * kTile), 16, off, 0, 0, 0);
    };
    const auto step_at = [&](int kb) {  // the step of the whole product
      return ks0 + (kb < nsteps ? kb : nsteps - 1);
    };
    const auto dma_a_rows = [&](int q, int pair, uint16_t* slot) {
      const int ps = pair < npairs ? pair : npairs - 1;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ares, (lds_void*)(slot + (64 * w + 8 * q) * 64), 16,
                                               aoff[q], 128 * ps, 0, 0);
    };
    const auto from_a = [&](int kb) {
      const int ks = step_at(kb);
      return rows_of(p.a, p.lda, m0, p.rows_pad, p.lda, ks - ((ks >= half) + (ks >= 2 * half)) * half);
    };
    const auto dma_b_steps = [&](int j, int kb, uint16_t* stage) {
      const int ks = step_at(kb);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(bres, (lds_void*)(stage + 512 * (4 * w + j)), 16,
                                               boff[j], kOp * 2 * ks, 0, 0);
    };
    const int64_t b_rows = kMode == kDx ? p.vocab_left : p.rows_pad;
    const auto from_b = [&](int kb) {  // of Q the terms lie a plane apart
      const int ks = step_at(kb), term = (ks >= half) + (ks >= 2 * half);
      return rows_of(p.b + term * (kMode == kDw ? p.q_plane : 0), p.ldb, n0, b_rows, p.b_width,
                     ks - term * half);
    };
    // Fragment reads. rows: fragment (mt, step half par, substep s) is tile row
    // a_at(mt) + i, chunk 4par + 2s + h, at position chunk ^ ((i >> 1) & 7).
    // steps: (nt, s) is tile row b_at(nt) + i, chunk 2s + h at (2s + h) ^
    // ((i >> 2) & 3). columns: lane 16q + l reads rows 16s + 8(q/2) + l/4 (and 4
    // on), 8 bytes at columns b_at(nt) + 16(q%2) + 4(l%4).
    const int swa = (i >> 1) & 7, swb = (i >> 2) & 3;
    int fa[2][2];
#pragma unroll
    for (int par = 0; par < 2; ++par)
#pragma unroll
      for (int ss = 0; ss < 2; ++ss)
        fa[par][ss] = (a_at(0) + i) * 64 + 8 * ((4 * par + 2 * ss + h) ^ swa);
    const int fb0 = (b_at(0) + i) * 32 + 8 * (h ^ swb);
    const int fb1 = (b_at(0) + i) * 32 + 8 * ((2 + h) ^ swb);
    const int trow = 8 * h + ((lane >> 2) & 3), tg = 2 * ((trow & 3) ^ ((trow & 1) << 2));
    int ca[4], cb[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int c = 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
      ca[t] = trow * kTile + 8 * ((a_at(t) / 8 + c) ^ tg) + 4 * (lane & 1);
      cb[t] = trow * kTile + 8 * ((b_at(t) / 8 + c) ^ tg) + 4 * (lane & 1);
    }
    const auto frag_a = [&](const uint16_t* s, int t, int par, int ss) {
      if constexpr (kACols)
        return read_columns(s + ca[t] + 16 * ss * kTile);
      else
        return *reinterpret_cast<const u32x4_t*>(s + fa[par][ss] + (a_at(1) - a_at(0)) * 64 * t);
    };
    const auto frag_b = [&](const uint16_t* s, int t, int ss) {
      if constexpr (kBCols)
        return read_columns(s + cb[t] + 16 * ss * kTile);
      else
        return *reinterpret_cast<const u32x4_t*>(s + (ss ? fb1 : fb0) + (b_at(1) - b_at(0)) * 32 * t);
    };

    // Prologue: what steps 0 and 1 read, then a's pair 1 or step 2 and b's step
    // 2; wait for the former.
    const auto load_a = [&](int n, uint16_t* s) {  // pair or step n
      if constexpr (kACols) {
        const Window from = from_a(n);
#pragma unroll
        for (int q = 0; q < 4; ++q) dma_cols(from, aoff[q], q, s);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) dma_a_rows(q, n, s);
      }
    };
    const auto load_b = [&](int kb, uint16_t* stage) {
      if constexpr (kBCols) {
        const Window from = from_b(kb);
#pragma unroll
        for (int j = 0; j < 4; ++j) dma_cols(from, boff[j], j, stage);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) dma_b_steps(j, kb, stage);
      }
    };
    load_a(0, sa0);
    if constexpr (kACols) load_a(1, sa1);
    load_b(0, sb0);
    load_b(1, sb1);
    load_a(kACols ? 2 : 1, kACols ? sa2 : sa1);
    load_b(2, sb2);
    wait_vmem_lgkm0<kACols ? 8 : 12>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    constexpr int kAReads = kACols ? 2 : 1, kBReads = kBCols ? 2 : 1;
    const auto product = [&](auto mfc, auto nfc) __attribute__((always_inline)) {
      constexpr int MF = decltype(mfc)::value, NF = decltype(nfc)::value;
      constexpr int kMfmas = MF * NF, kBoth = MF < NF ? MF : NF, kReads = MF + NF;
      static_assert(kMfmas % 4 == 0 && kReads <= kMfmas, "a read and a load after some MFMA each");
      u32x4_t a0[MF], b0[NF], a1[MF], b1[NF];
#pragma unroll
      for (int t = 0; t < MF; ++t) a0[t] = frag_a(sa0, t, 0, 0);
#pragma unroll
      for (int t = 0; t < NF; ++t) b0[t] = frag_b(sb0, t, 0);
      // One step kb (stage kb % 4 = SB, pair slot (kb / 2) % 3 = SA, half PAR):
      // substep 0 computes on (a0, b0) while (kb, 1) is read into (a1, b1);
      // substep 1 computes on (a1, b1) while (kb+1, 0) is read into (a0, b0). One
      // load after every quarter of the MFMAs: b of step kb+3 in substep 0, a of pair kb/2 + 2
      // or of step kb+3 in substep 1.
      auto step = [&](int kb, auto sbc, auto sac, auto parc) __attribute__((always_inline)) {
        constexpr int SB = decltype(sbc)::value, SA = decltype(sac)::value;
        constexpr int PAR = decltype(parc)::value;
        constexpr int SA1 = PAR ? (SA + 1) % 3 : SA;  // slot of step kb+1
        constexpr int PAR1 = PAR ^ 1;
        constexpr int kACur = kACols ? SB : SA, kANxt = kACols ? (SB + 1) % 4 : SA1;
        constexpr int kALd = kACols ? (SB + 3) % 4 : (SA + 2) % 3;
        uint16_t* const acur = pick<kACur>(sa);
        uint16_t* const anxt = pick<kANxt>(sa);
        uint16_t* const ald = pick<kALd>(sa);
        uint16_t* const bcur = pick<SB>(sb);
        uint16_t* const bnxt = pick<(SB + 1) % 4>(sb);
        uint16_t* const bld = pick<(SB + 3) % 4>(sb);
        Window bnew{nullptr, 0}, anew{nullptr, 0};
        if constexpr (kBCols) bnew = from_b(kb + 3);
        if constexpr (kACols) anew = from_a(kb + 3);
#pragma unroll
        for (int g = 0; g < kMfmas; ++g) {
          const int mt = g / NF, nt = g % NF;
          acc[mt][nt] = mfma_32x32x16(a0[mt], b0[nt], acc[mt][nt]);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          if (g < kReads) {
            const int t = g < 2 * kBoth ? g >> 1 : g - kBoth;
            if (g < 2 * kBoth ? g & 1 : NF > MF) {
              b1[t] = frag_b(bcur, t, 1);
              __builtin_amdgcn_sched_group_barrier(0x100, kBReads, 0);
            } else {
              a1[t] = frag_a(acur, t, PAR, 1);
              __builtin_amdgcn_sched_group_barrier(0x100, kAReads, 0);
            }
          }
          if ((g + 1) % (kMfmas / 4) == 0) {
            const int q = g / (kMfmas / 4);
            if constexpr (kBCols)
              dma_cols(bnew, boff[q], q, bld);
            else
              dma_b_steps(q, kb + 3, bld);
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int g = 0; g < kMfmas; ++g) {
          const int mt = g / NF, nt = g % NF;
          acc[mt][nt] = mfma_32x32x16(a1[mt], b1[nt], acc[mt][nt]);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          if (g < kReads) {
            const int t = g < 2 * kBoth ? g >> 1 : g - kBoth;
            if (g < 2 * kBoth ? g & 1 : NF > MF) {
              b0[t] = frag_b(bnxt, t, 0);
              __builtin_amdgcn_sched_group_barrier(0x100, kBReads, 0);
            } else {
              a0[t] = frag_a(anxt, t, PAR1, 0);
              __builtin_amdgcn_sched_group_barrier(0x100, kAReads, 0);
            }
          }
          if ((g + 1) % (kMfmas / 4) == 0) {
            const int q = g / (kMfmas / 4);
            if constexpr (kACols)
              dma_cols(anew, aoff[q], q, ald);
            else
              dma_a_rows(4 * PAR + q, kb / 2 + 2, ald);
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        // This step's eight loads may still fly; everything earlier has landed.
        wait_vmem_lgkm0<8>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
      };
      using I0 = std::integral_constant<int, 0>;
      using I1 = std::integral_constant<int, 1>;
      using I2 = std::integral_constant<int, 2>;
      using I3 = std::integral_constant<int, 3>;
      // Twelve steps bring all rings back to their first stage and slot.
      int kb = 0;
      for (; kb + 12 <= nsteps; kb += 12) {
        step(kb + 0, I0(), I0(), I0());
        step(kb + 1, I1(), I0(), I1());
        step(kb + 2, I2(), I1(), I0());
        step(kb + 3, I3(), I1(), I1());
        step(kb + 4, I0(), I2(), I0());
        step(kb + 5, I1(), I2(), I1());
        step(kb + 6, I2(), I0(), I0());
        step(kb + 7, I3(), I0(), I1());
        step(kb + 8, I0(), I1(), I0());
        step(kb + 9, I1(), I1(), I1());
        step(kb + 10, I2(), I2(), I0());
        step(kb + 11, I3(), I2(), I1());
      }
      if (kb + 0 < nsteps) step(kb + 0, I0(), I0(), I0());
      if (kb + 1 < nsteps) step(kb + 1, I1(), I0(), I1());
      if (kb + 2 < nsteps) step(kb + 2, I2(), I1(), I0());
      if (kb + 3 < nsteps) step(kb + 3, I3(), I1(), I1());
      if (kb + 4 < nsteps) step(kb + 4, I0(), I2(), I0());
      if (kb + 5 < nsteps) step(kb + 5, I1(), I2(), I1());
      if (kb + 6 < nsteps) step(kb + 6, I2(), I0(), I0());
      if (kb + 7 < nsteps) step(kb + 7, I3(), I0(), I1());
      if (kb + 8 < nsteps) step(kb + 8, I0(), I1(), I0());
      if (kb + 9 < nsteps) step(kb + 9, I1(), I1(), I1());
      if (kb + 10 < nsteps) step(kb + 10, I2(), I2(), I0());
    };
    using I2f = std::integral_constant<int, 2>;
    using I4f = std::integral_constant<int, 4>;
    // Half the fragments where half a tile has no live rows (dX of 8 rows, 32000 x
    // 4096: 46 against 57 us; 100 rows, 32000 x 2048: forward 47 against 56 us; the
    // last of several tiles hardly gains, 300 rows of 128000 x 4096: 390 against 407).
    if (kMode == kDx && M - m0 <= kTile / 2)
      product(I2f(), I4f());
    else if (kMode != kDx && kMode != kDw && N - n0 <= kTile / 2)
      product(I4f(), I2f());
    else
      product(I4f(), I4f());
    // Direct-to-LDS loads still in flight must land before LDS is used again or
    // the workgroup ends.
    wait_vmem_lgkm0<0>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }

  // What follows starts from a thread id of its own: derived from the one above, its
  // values were kept in registers through the loop, which has none to spare.
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, i = lane & 31, h = lane >> 5;
  // Accumulator element e of (mt, nt) is tile row a_at(mt) + 8(e/4) + 4h + e%4, column
  // b_at(nt) + i.
  const int64_t mw = m0 + a_at(0) + 4 * h;
  uint16_t* const own = w == 0 ? sb0 : w == 1 ? sb1 : w == 2 ? sb2 : sb3;  // a wave's 16 KB of LDS
  if constexpr (kMode == kStats) {
    // A lane has 64 entries of the vocabulary of each of its four rows; the
    // other half of the wave and the other wave of the rows have the rest.
    float2* red = reinterpret_cast<float2*>(sa0);
    const bool whole = m0 + kTile <= M;  // all of the tile's entries exist
    const int left = (int)min(M - mw, (int64_t)kTile);
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      float m = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[mt][nt][e] *= p.scale;
      if (!whole) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (32 * mt + 8 * (e >> 2) + (e & 3) >= left) acc[mt][nt][e] = -INFINITY;
      }
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 16; ++e) m = fmaxf(m, acc[mt][nt][e]);
      m = fmaxf(m, __shfl_xor(m, 32));
      const float from = m == -INFINITY ? 0.0f : m;  // none of the vocabulary, or none above it
      float s = 0.0f;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 16; ++e) s += exp2_fast((acc[mt][nt][e] - from) * kLog2e);
      s += __shfl_xor(s, 32);
      if (h == 0) red[wm * kTile + b_at(nt) + i] = float2{m, s};
      // The label's logit, where this wave has it.
      const int64_t n = n0 + b_at(nt) + i;
      const int label = n < N ? p.cols[n].label : -1;
      const int64_t away = label - (p.v0 + mw);
      const bool mine = label >= 0 && away >= 0 && away < 128 && !(away & 4);
      const int d = (int)away;
      if (__ballot(mine)) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (mine && d == 32 * mt + 8 * (e >> 2) + (e & 3)) p.at_label[n] = acc[mt][nt][e];
      }
    }
    __syncthreads();
    if (n0 + tid < N) {
      const float2 x = red[tid], y = red[kTile + tid];
      const float m = fmaxf(x.x, y.x), from = m == -INFINITY ? 0.0f : m;
      const float s = x.y * exp2_fast((x.x - from) * kLog2e) + y.y * exp2_fast((y.x - from) * kLog2e);
      p.part[(p.v0 / kTile + tm) * p.rows_pad + n0 + tid] = float2{m, s};
    }
  } else if constexpr (kMode == kProbs) {
    // Whole pairs of steps of what the products reduce over are written: along
    // the vocabulary for P, along the live rows for Q. The wave's block goes through
    // its own LDS, a term at a time, so that a store is 256 bytes of four rows.
    const int64_t phalf = whole_pairs(p.vocab), qhalf = whole_pairs(live);
    const int64_t mwave = m0 + 128 * wm, nwave = n0 + 32 * wn;
    const bool whole = m0 + kTile <= M;
    const int left = (int)min(M - mw, (int64_t)kTile);
    int hot[4];  // the label's place among this lane's entries
    float rest[4], factor[4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const HeadColumn c = p.cols[n0 + b_at(nt) + i];  // whole tiles: zeros behind the live rows
      const int64_t away = c.label - (p.v0 + mw);
      hot[nt] = c.label < 0 || away < 0 || away >= kTile ? -1 : (int)away;
      factor[nt] = c.factor;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float v = exp2_fast(fmaf(acc[mt][nt][e], p.scale, -c.most) * kLog2e) * c.over;
          acc[mt][nt][e] = c.label >= 0 ? v : 0.0f;
        }
    }
    if (!whole) {
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (32 * mt + 8 * (e >> 2) + (e & 3) >= left) acc[mt][nt][e] = 0.0f;
    }
    // p - 1 at a label, which leaves the others; few waves have one.
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      rest[nt] = 0.0f;
      const bool mine = hot[nt] >= 0 && hot[nt] < 128 && !(hot[nt] & 4);
      if (!__ballot(mine)) continue;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (hot[nt] == 32 * mt + 8 * (e >> 2) + (e & 3)) {
            rest[nt] = acc[mt][nt][e];
            acc[mt][nt][e] = 0.0f;
          }
      rest[nt] -= 1.0f;
      if (mine && p.rest) p.rest[n0 + b_at(nt) + i] = rest[nt];
    }
    const int part = lane & 15, row0 = lane >> 4;
    // One term: bf16 in LDS, 64 rows at a time.
    const auto put_one = [&](uint16_t* at, int64_t ld, int rows, bool in) __attribute__((always_inline)) {
      at += (nwave + row0) * ld + mwave + 8 * part;
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          uint16_t* const to = own + (32 * n + i) * 128 + 4 * h;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const f32x16_t& v = acc[mt][2 * pass + n];
              *reinterpret_cast<u32x2_t*>(to + 8 * ((4 * mt + g) ^ (i & 15))) =
                  term_of<0>(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
            }
        }
#pragma unroll 4
        for (int r = 0; r < 16; ++r) {
          const int row = row0 + 4 * r;
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(own + row * 128 + 8 * (part ^ (row & 15)));
          if (in && 128 * pass + row + (r < 8 ? 0 : 32) < rows) *reinterpret_cast<u32x4_t*>(at) = v;
          at += (r % 8 == 7 ? 36 : 4) * ld;
        }
      }
    };
    // Three terms: fp32 in LDS, 32 rows at a time, split when they are read back.
    const auto put_three = [&](uint16_t* at, int64_t plane, int64_t ld, int rows, bool in) __attribute__((always_inline)) {
      f32x4_t* const lds = reinterpret_cast<f32x4_t*>(own);
      at += (nwave + row0) * ld + mwave + 8 * part;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x16_t& v = acc[mt][nt];
            lds[i * 32 + ((8 * mt + 2 * g + h) ^ i)] =
                f32x4_t{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
          }
#pragma unroll 2
        for (int r = 0; r < 8; ++r) {
          const int row = row0 + 4 * r;
          const f32x4_t x = lds[row * 32 + ((2 * part) ^ row)], y = lds[row * 32 + ((2 * part + 1) ^ row)];
          if (in && 64 * nt + row < rows) {
            const auto store = [&](uint16_t* to, u32x2_t a, u32x2_t b) {
              *reinterpret_cast<u32x4_t*>(to) = u32x4_t{a[0], a[1], b[0], b[1]};
            };
            store(at, term_of<0>(x[0], x[1], x[2], x[3]), term_of<0>(y[0], y[1], y[2], y[3]));
            store(at + plane, term_of<1>(x[0], x[1], x[2], x[3]), term_of<1>(y[0], y[1], y[2], y[3]));
            store(at + 2 * plane, term_of<2>(x[0], x[1], x[2], x[3]), term_of<2>(y[0], y[1], y[2], y[3]));
          }
          at += 4 * ld;
        }
        at += 32 * ld;
      }
    };
    const auto put = [&](uint16_t* to, int64_t plane, int terms, int64_t ld, int rows, bool in) __attribute__((always_inline)) {
      if (kTerms > 1 && terms > 1)
        put_three(to, plane, ld, rows, in);
      else
        put_one(to, ld, rows, in);
    };
    if (p.P)
      put(p.P, phalf, p.p_terms, p.ldp, (int)min(N - nwave, (int64_t)kTile), mwave + 8 * part < phalf);
    if (p.Q) {
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            acc[mt][nt][e] = (hot[nt] == 32 * mt + 8 * (e >> 2) + (e & 3) ? rest[nt] : acc[mt][nt][e]) *
                             factor[nt];
      put(p.Q, p.q_plane, p.q_terms, p.ldq, (int)min(qhalf - nwave, (int64_t)kTile),
          mwave + 8 * part < p.ldq);
    }
  } else if constexpr (kMode == kDx) {
    // The sums in the order of the registers, 16 bytes a thread: tile by tile,
    // split by split.
    float* to = p.acc + ((int64_t)split * tiles + tm * tiles_n + tn) * (kTile * kTile) + 4 * tid;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      if (m0 + a_at(mt) >= M) continue;  // no live row in these 32
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          f32x4_t* o = reinterpret_cast<f32x4_t*>(to + ((mt * 4 + nt) * 4 + g) * 1024);
          f32x4_t v = {acc[mt][nt][4 * g], acc[mt][nt][4 * g + 1], acc[mt][nt][4 * g + 2],
                       acc[mt][nt][4 * g + 3]};
          if (p.add) v += *o;
          *o = v;
        }
    }
  } else {
    const int64_t mwave = m0 + 128 * wm, nwave = n0 + 128 * wn;
    if constexpr (kTerms == 1) {  // bf16, not added to anything
      put_dw<true, false>(acc, own, p, mwave, nwave, lane);
    } else {
      if (p.dw_bf16)
        put_dw<true, true>(acc, own, p, mwave, nwave, lane);
      else
        put_dw<false, true>(acc, own, p, mwave, nwave, lane);
    }
  }
}

// -------------------------------------------------------------- the results
// 16 rows a workgroup, the tiles of the vocabulary in 16 ranges.
__global__ __launch_bounds__(256) void head_loss_kernel(const float2* part, int64_t tiles,
                                                        int64_t rows_pad, const float* at_label,
                                                        const int32_t* inv, int64_t M, float* loss,
                                                        float* stats) {
  __shared__ float2 red[16][16];
  const int r = threadIdx.x % 16, range = threadIdx.x / 16;
  const int64_t row = (int64_t)blockIdx.x * 16 + r;
  const int32_t j = row < M ? inv[row] : -1;
  const int64_t per = (tiles + 15) / 16;
  float m = -INFINITY, s = 0.0f;
  if (j >= 0) {
    const int64_t end = (range + 1) * per < tiles ? (range + 1) * per : tiles;
#pragma unroll 4
    for (int64_t t = range * per; t < end; ++t) {
      const float2 v = part[t * rows_pad + j];
      const float to = fmaxf(m, v.x), from = to == -INFINITY ? 0.0f : to;
      s = s * exp2_fast((m - from) * kLog2e) + v.y * exp2_fast((v.x - from) * kLog2e);
      m = to;
    }
  }
  red[range][r] = float2{m, s};
  __syncthreads();
  if (threadIdx.x >= 16 || row >= M) return;
  for (int k = 1; k < 16; ++k) {
    const float2 v = red[k][r];
    const float to = fmaxf(m, v.x), from = to == -INFINITY ? 0.0f : to;
    s = s * exp2_fast((m - from) * kLog2e) + v.y * exp2_fast((v.x - from) * kLog2e);
    m = to;
  }
  const float L = logf(s);
  loss[row] = j >= 0 ? L + (m - at_label[j]) : 0.0f;
  if (stats) {
    stats[row] = j >= 0 ? m : 0.0f;
    stats[M + row] = j >= 0 ? L : 0.0f;
  }
}

// Four rows a workgroup, four columns a thread: of live rows 4x .. 4x + 3 in the
// first half of the grid, whose sums lie as head_tile_kernel's registers had
// them, and of rows that carry no loss in the second half.
template <bool kBf16>
__global__ __launch_bounds__(256) void head_dx_finish_kernel(HeadDx a) {
  constexpr int E = 4;
  const int64_t k = ((int64_t)blockIdx.y * 256 + threadIdx.x) * E;
  if (k >= a.K) return;
  const int n = count_below<E>(k, a.K);
  const auto put = [&](int64_t row, const float (&v)[E]) {
    elem_t<kBf16>* to = static_cast<elem_t<kBf16>*>(a.dX) + row * a.lddx + k;
    if (n == E)
      store_vec<kBf16, E>(to, v);
    else
      store_part<kBf16, E>(to, v, n);
  };
  const int64_t groups = (a.M + 3) / 4;
  if ((int64_t)blockIdx.x >= groups) {
    const int64_t m = ((int64_t)blockIdx.x - groups) * 4;
    const float none[E] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int e = 0; e < 4; ++e)
      if (m + e < a.M && a.inv[m + e] < 0) put(m + e, none);
    return;
  }
  const int live = *a.count;
  const int j = (int)blockIdx.x * 4;
  if (j >= live) return;
  // The labels' rows of W, requested before the sums.
  HeadColumn col[4];
  float rest[4];
  Vec<true, E> w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    col[e] = a.cols[j + e < live ? j + e : j];
    rest[e] = a.rest[j + e < live ? j + e : j];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint16_t* from = a.W + (int64_t)col[e].label * a.ldw + k;
    w[e] = n == E ? load_vec<true, E>(from) : load_part<true, E>(from, n);
  }
  const int tiles_n = ceil_tile(a.K), tiles = ceil_tile(live) * tiles_n;
  const int splits = a.count[1];
  const int r = j % kTile, c = (int)(k % kTile);
  const int tid = ((r / 32) % 2 * 2 + c / 128) * 64 + ((r / 4) % 2) * 32 + c % 32;
  const int reg = ((r / 64) * 4 + c % 128 / 32) * 4 + r % 32 / 8;
  const float* from = a.acc + ((int64_t)(j / kTile) * tiles_n + k / kTile) * (kTile * kTile) + reg * 1024 + 4 * tid;
  f32x4_t sum[E];  // of a column, its four rows
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = 0; s < splits; ++s, from += (int64_t)tiles * (kTile * kTile)) {
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] += *reinterpret_cast<const f32x4_t*>(from + 4 * e);
  }
#pragma unroll
  for (int row = 0; row < 4; ++row) {
    if (j + row >= live) break;
    float o[E], v[E];
    to_float<true, E>(w[row], o);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = fmaf(rest[row], o[e], sum[e][row]) * col[row].factor;
    put(a.map[j + row], v);
  }
}

unsigned blocks_of(int64_t n) { return (unsigned)((n + 255) / 256); }
int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }

template <int kMode, int kTerms = 1>
hipError_t tiles(const HeadTiles& a, int64_t grid, hipStream_t st) {
  hipLaunchKernelGGL((head_tile_kernel<kMode, kTerms>), dim3((unsigned)grid), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_head_rows(const HeadRows& a, hipStream_t st) {
  hipLaunchKernelGGL(head_rows_kernel, dim3(1), dim3(kRowThreads), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_head_pack_rows(const uint16_t* src, int64_t ld, const int32_t* map,
                                 const int32_t* count, int64_t rows, int64_t K, uint16_t* out,
                                 hipStream_t st) {
  const int64_t vecs = (K + kStep - 1) / kStep * 4;
  hipLaunchKernelGGL(head_pack_rows_kernel, linear_grid(tiles_of(rows) * kTile * vecs), dim3(256), 0,
                     st, src, ld, map, count, rows, K, out);
  return hipGetLastError();
}

hipError_t launch_head_copy(const uint16_t* src, int64_t ld, const int32_t* map,
                            const int32_t* count, int64_t rows, int64_t K, int64_t Kp, uint16_t* out,
                            hipStream_t st) {
  const int64_t most = map ? (rows + 2 * kStep - 1) / (2 * kStep) * (2 * kStep) : rows;
  hipLaunchKernelGGL(head_copy_kernel, linear_grid(most * (Kp / 8)), dim3(256), 0, st, src, ld, map,
                     count, rows, K, Kp, out);
  return hipGetLastError();
}

hipError_t launch_head_zero(void* p, int64_t bytes, hipStream_t st) {
  hipLaunchKernelGGL(head_zero_kernel, linear_grid((bytes / 2 + 1) / 2), dim3(256), 0, st,
                     static_cast<uint32_t*>(p), bytes / 2);
  return hipGetLastError();
}

hipError_t launch_head_stats(const HeadTiles& a, hipStream_t st) {
  return tiles<kStats>(a, tiles_of(a.vocab) * tiles_of(a.rows_most), st);
}

hipError_t launch_head_probs(const HeadTiles& a, hipStream_t st) {
  const int64_t grid = tiles_of(a.vocab) * tiles_of(a.rows_most);
  return a.p_terms > 1 || a.q_terms > 1 ? tiles<kProbs, 3>(a, grid, st) : tiles<kProbs>(a, grid, st);
}

hipError_t launch_head_dx(const HeadTiles& a, hipStream_t st) {
  return tiles<kDx>(a, head_sums(a.rows_most, a.K), st);
}

hipError_t launch_head_dw(const HeadTiles& a, hipStream_t st) {
  const int64_t grid = tiles_of(a.vocab) * tiles_of(a.K);
  return a.accumulate || !a.dw_bf16 ? tiles<kDw, 3>(a, grid, st) : tiles<kDw>(a, grid, st);
}

hipError_t launch_head_loss(const float2* part, int64_t tiles, int64_t rows_pad,
                            const float* at_label, const int32_t* inv, int64_t M, float* loss,
                            float* stats, hipStream_t st) {
  hipLaunchKernelGGL(head_loss_kernel, dim3((unsigned)((M + 15) / 16)), dim3(256), 0, st, part, tiles,
                     rows_pad, at_label, inv, M, loss, stats);
  return hipGetLastError();
}

hipError_t launch_head_dx_finish(const HeadDx& a, bool bf16, hipStream_t st) {
  const dim3 grid((unsigned)((a.M + 3) / 4 * 2), blocks_of((a.K + 3) / 4));  // rows past the second dimension's 65535
  if (bf16)
    hipLaunchKernelGGL(head_dx_finish_kernel<true>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(head_dx_finish_kernel<false>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace qlora
