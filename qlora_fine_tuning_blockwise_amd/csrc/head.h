// Internal declarations of the vocabulary head's loss: what its entry points
// lay out and launch.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace qlora {

constexpr int kTile = 256;  // rows and columns of a product's tile
constexpr int kStep = 32;   // reduction elements of a step

// A live row as the tile kernels see it: its largest logit, exp(-log of its
// sum), the factor of its gradient, its label. Behind the live rows, up to a
// whole tile: zeros and no label.
struct HeadColumn {
  float most, over, factor;
  int32_t label;
};

// The rows that carry loss, in order: map[j] is the row of live row j, inv[m]
// the live row of row m or -1, count[0] how many there are, count[1] the splits of
// their gradient's product.
struct HeadRows {
  const void* labels;
  bool ids64;
  const float* dloss;  // rows with 0 carry nothing either; NULL in the forward
  const float* stats;  // [2, M]; NULL in the forward
  float scale;
  int64_t M, V, K;
  int pairs;  // of launch_head_dx; 0 without it
  int32_t* map;
  int32_t* inv;
  int32_t* count;
  HeadColumn* cols;
};
hipError_t launch_head_rows(const HeadRows& a, hipStream_t st);

// b operands lie in tiles of 256 of their rows, a tile's steps one behind
// another, 16 KB each: [tile][step][256][32].
// out = rows map[j] of src (rows j themselves without a map), j < *count (or
// `rows` without), reduction over the K columns; zero up to a whole tile of rows
// and a whole step.
hipError_t launch_head_pack_rows(const uint16_t* src, int64_t ld, const int32_t* map,
                                 const int32_t* count, int64_t rows, int64_t K, uint16_t* out,
                                 hipStream_t st);
// out[j] = row map[j] of src (row j without a map) with zeros behind its K columns
// up to Kp; for j < rows, nothing where *count is 0; with a map for j < *count, and
// rows of zeros up to two whole steps.
hipError_t launch_head_copy(const uint16_t* src, int64_t ld, const int32_t* map,
                            const int32_t* count, int64_t rows, int64_t K, int64_t Kp, uint16_t* out,
                            hipStream_t st);

// Zeros in 4-byte aligned memory, a multiple of two bytes (dW without rows).
hipError_t launch_head_zero(void* p, int64_t bytes, hipStream_t st);

// A product's tiles; what a and b are depends on the launch.
struct HeadTiles {
  const uint16_t* a;  // 16-byte aligned rows
  int64_t lda;        // a multiple of 8
  const uint16_t* b;
  int64_t b_steps;    // steps that a tile of b has room for (logits)
  int64_t ldb, b_width, vocab_left;  // gradients: b's rows, columns; entries of the vocabulary from v0 on
  const int32_t* count;
  int64_t v0, vocab;  // the piece's first entry of the vocabulary, its entries
  int64_t rows_most;  // the most live rows there can be
  int64_t K;          // the hidden size
  int64_t steps;      // of the logits' reduction
  float scale;
  // logits: partial statistics [tile of the vocabulary][rows_pad]
  const HeadColumn* cols;
  float2* part;
  int64_t rows_pad;
  float* at_label;  // statistics: the labels' logits
  // probabilities P (0 at the row's label) and the logits' gradients Q, live rows by
  // vocabulary; the terms of P lie one behind another in a row, those of Q a plane
  // apart
  float* rest;  // the labels' probabilities less 1, of live rows; NULL without P
  uint16_t* P;
  int64_t ldp;
  int p_terms;
  uint16_t* Q;
  int64_t ldq, q_plane;
  int q_terms;
  // gradients
  float* acc;  // sums of the live rows' gradient, [split][tile][256 x 256]
  bool add;    // to what acc holds
  void* dW;
  bool dw_bf16, accumulate;
};
// Partial statistics and the labels' logits; probabilities; the gradient of the
// live rows; the gradient of the piece's rows of W.
hipError_t launch_head_stats(const HeadTiles& a, hipStream_t st);
hipError_t launch_head_probs(const HeadTiles& a, hipStream_t st);
hipError_t launch_head_dx(const HeadTiles& a, hipStream_t st);
hipError_t launch_head_dw(const HeadTiles& a, hipStream_t st);
// Splits of the live rows' gradient at most, and tiles times splits at most
// where there is more than one.
constexpr int kMostSplits = 64, kMostSums = 512;
// Sums of 256 x 256 that acc holds: tiles times splits, at most, for any count of
// live rows.
inline int64_t head_sums(int64_t rows_most, int64_t K) {
  const int64_t tiles = (rows_most + kTile - 1) / kTile * ((K + kTile - 1) / kTile);
  const int64_t split = tiles * kMostSplits < kMostSums ? tiles * kMostSplits : kMostSums;
  return tiles > split ? tiles : split;
}

// The logits of at most kFewRows rows, one pass over W at any row stride and
// alignment. Statistics: of rows j themselves, joined over `entries`
// entries of the vocabulary (few_entries): part[row][parts]. Probabilities: of live rows, as
// launch_head_probs leaves them; p_plane: elements between P's terms.
constexpr int64_t kFewRows = 64;
// Entries of the vocabulary that a workgroup takes: 128, or 32 where those leave CUs
// idle. More than 32 rows of x are worth sharing sooner (64 rows, 20000 x 1024: 20.7
// against 26.5 us, 12000 x 2048: 33 against 25; 32 rows, 20000 x 1024: level).
inline int64_t few_entries(int64_t V, int64_t M) { return V >= (M > 32 ? 128 : 192) * 128 ? 128 : 32; }
struct HeadFew {
  const uint16_t* W;  // the piece's rows
  int64_t ldw;
  const uint16_t* x;
  int64_t ldx, M, K, V, v0, vocab, entries;  // v0, vocab: the piece
  float scale;
  const void* labels;
  bool ids64;
  float2* part;
  int64_t parts;
  float* at_label;
  const int32_t* map;
  const int32_t* count;
  const HeadColumn* cols;
  float* rest;
  uint16_t* P;
  int64_t ldp, p_plane;
  int p_terms;
  uint16_t* Q;
  int64_t ldq, q_plane;
  int q_terms;
};
hipError_t launch_head_few_stats(const HeadFew& a, hipStream_t st);
hipError_t launch_head_few_probs(const HeadFew& a, hipStream_t st);
hipError_t launch_head_few_loss(const float2* part, int64_t parts, const float* at_label,
                                const void* labels, bool ids64, int64_t M, int64_t V, float* loss,
                                float* stats, hipStream_t st);

// loss and stats (may be NULL) of all M rows from the partial statistics.
hipError_t launch_head_loss(const float2* part, int64_t tiles, int64_t rows_pad,
                            const float* at_label, const int32_t* inv, int64_t M, float* loss,
                            float* stats, hipStream_t st);
// dX of all M rows: factor (sum of the splits + rest times the label's row of W),
// or 0.
struct HeadDx {
  const float* acc;
  const float* rest;
  const int32_t* map;
  const int32_t* inv;
  const int32_t* count;
  const HeadColumn* cols;
  const uint16_t* W;
  int64_t ldw, M, K;
  void* dX;
  int64_t lddx;
};
hipError_t launch_head_dx_finish(const HeadDx& a, bool bf16, hipStream_t st);

// dX of at most kFewDxRows rows in one pass over W, at any row stride and
// alignment, for hidden sizes of whole 16 bytes that a workgroup's waves hold
// (32000 x 4096: 8 rows 68 us where logits and product apart take 109, 16 rows 84
// against 98; 32000 x 2048: 42 and 48 against 63).
constexpr int64_t kFewDxRows = 16, kFewDxWidth = 4096;
inline bool few_dx(int64_t M, int64_t K) { return M <= kFewDxRows && K <= kFewDxWidth && K % 8 == 0; }
// Workgroups, one a CU: each leaves a sum of every live row.
inline int few_dx_groups(int64_t V) { return V < 256 * 16 ? (int)((V + 15) / 16) : 256; }
inline int64_t few_dx_sums(int64_t M, int64_t V, int64_t K) { return few_dx_groups(V) * ((K + 15) / 16) * 16 * M; }
struct HeadFewDx {
  const uint16_t* W;
  int64_t ldw;
  const uint16_t* x;
  int64_t ldx, M, V, K;
  float scale;
  const int32_t* map;
  const int32_t* inv;
  const int32_t* count;
  const HeadColumn* cols;
  float* part;  // few_dx_sums of them
  float* rest;  // the live rows' p - 1 at their labels
  int groups;
  void* dX;
  int64_t lddx;
};
hipError_t launch_head_few_dx(const HeadFewDx& a, bool bf16, hipStream_t st);

}  // namespace qlora
