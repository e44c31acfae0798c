// Layouts of the block-scaled FP8 operands (host and device).
//
// A value is e4m3(code) * 2^(byte - 127): e4m3 codes under one power-of-two
// scale (a ue8m0 byte) per row and block of 128 elements along K, the unit
// both the activations' rows and the weights' output columns use.
//
//   KS = ceil(K / 128)   k-stages: 128 codes are a 128-byte operand row
//   KW = ceil(KS / 4)    scale words: the bytes of 4 consecutive blocks
//
// Operand rows are stored as the shared-memory image a K-major tcgen05
// operand with the 128-byte swizzle has: 16-byte chunk c of row r at
// (c ^ (r % 8)) * 16 of the row, and stage by stage, so that a run of rows of
// one stage that starts on a multiple of 8 is one contiguous copy - whatever
// its length, and without padding around a ragged group of rows:
//
//   activations  codes  [KS][Mp][128], Mp = M rounded up to 8
//                scales [KW][Mp] words
//   weights      codes  [experts][KS][N][128]   (N % 8 == 0)
//                scales [experts][NT][KW][512 bytes], NT = ceil(N / 128): an
//                       atom holds the words of 128 columns as a tcgen05.cp
//                       32x128b.warpx4 copy reads them, column c's word at
//                       (c % 32) * 16 + (c / 32) * 4
// Codes past K are zero in both; activation rows past M and words of columns
// past N are never written and never reach an output.
#pragma once

#include <cstddef>
#include <cstdint>

namespace svdq {
namespace fp8 {

constexpr int kBlock = 128;
constexpr int kScaleAtom = 512;

inline int k_stages(int K) { return (K + kBlock - 1) / kBlock; }
inline int k_words(int K) { return (k_stages(K) + 3) / 4; }
inline int padded_rows(int M) { return (M + 7) & ~7; }
// The rows of a token tile of the kernel for few rows, or 0 for more rows than
// that (an average share above 128 an expert).  Experts are liked unevenly, and
// one whose rows fill several tiles reads its weights as often, so theirs hold
// twice the average share (64 experts, 1001 rows: 35.7 us in tiles of 32, 40.5
// in tiles of 16).  The smallest tiles quantize X on the way in and need no
// workspace.
constexpr bool few_fused(int tile_rows) { return tile_rows <= 16; }
inline int few_tile(int M, int experts) {
  const long long share = (static_cast<long long>(M) + experts - 1) / experts, rows = experts > 1 ? 2 * share : share;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : share <= 128 ? 128 : 0;
}
inline bool needs_workspace(int M, int experts) {
  const int tile = few_tile(M, experts);
  return tile == 0 || !few_fused(tile);
}
inline size_t act_code_bytes(int M, int K) {
  return static_cast<size_t>(k_stages(K)) * static_cast<size_t>(padded_rows(M)) * kBlock;
}
inline size_t act_bytes(int M, int K) {
  return act_code_bytes(M, K) + static_cast<size_t>(k_words(K)) * static_cast<size_t>(padded_rows(M)) * 4u;
}
inline size_t weight_code_bytes(int K, int N, int experts) {
  return static_cast<size_t>(experts) * static_cast<size_t>(k_stages(K)) * static_cast<size_t>(N) * kBlock;
}
inline size_t weight_bytes(int K, int N, int experts) {
  return weight_code_bytes(K, N, experts) +
         static_cast<size_t>(experts) * static_cast<size_t>((N + 127) / 128) * static_cast<size_t>(k_words(K)) * kScaleAtom;
}

}  // namespace fp8
}  // namespace svdq
