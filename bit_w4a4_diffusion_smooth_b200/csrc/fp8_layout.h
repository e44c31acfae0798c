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
// (c ^ (r % 8)) * 16 of the row.  A run of rows that starts on a multiple of 8
// is therefore one contiguous copy.
//
//   activations  codes  [KS][Mp][128], Mp = M rounded up to 8: any 8-aligned
//                       run of rows of one stage is contiguous, so a ragged
//                       group of rows needs no padding of its own
//                scales [KW][Mp] words
//   weights      codes  [experts][NT][KS][128 rows][128], NT = ceil(N / 128)
//                scales [experts][NT][KW][512 bytes]: the word of row r at
//                       (r % 32) * 16 + (r / 32) * 4, the image of a
//                       tcgen05.cp 32x128b.warpx4 copy
// Codes past K are zero in both; weight rows past N hold zero codes;
// activation rows past M are never written and never reach an output.
#pragma once

#include <cstddef>
#include <cstdint>

namespace svdq {
namespace fp8 {

constexpr int kBlock = 128;
constexpr int kTileN = 128;          // weight rows per tile
constexpr int kTileBytes = kTileN * kBlock;
constexpr int kScaleAtom = 512;

inline int k_stages(int K) { return (K + kBlock - 1) / kBlock; }
inline int k_words(int K) { return (k_stages(K) + 3) / 4; }
inline int n_tiles(int N) { return (N + kTileN - 1) / kTileN; }
inline int padded_rows(int M) { return (M + 7) & ~7; }
inline size_t act_code_bytes(int M, int K) {
  return static_cast<size_t>(k_stages(K)) * static_cast<size_t>(padded_rows(M)) * kBlock;
}
inline size_t act_bytes(int M, int K) {
  return act_code_bytes(M, K) + static_cast<size_t>(k_words(K)) * static_cast<size_t>(padded_rows(M)) * 4u;
}
inline size_t weight_code_bytes(int K, int N, int experts) {
  return static_cast<size_t>(experts) * static_cast<size_t>(n_tiles(N)) * static_cast<size_t>(k_stages(K)) * kTileBytes;
}
inline size_t weight_bytes(int K, int N, int experts) {
  return weight_code_bytes(K, N, experts) +
         static_cast<size_t>(experts) * static_cast<size_t>(n_tiles(N)) * static_cast<size_t>(k_words(K)) * kScaleAtom;
}

#ifdef __CUDACC__
// Scale byte of a block from the bits of its largest finite magnitude (a bf16
// value widened to float): e the smallest exponent >= -127 with
// amax <= 448 * 2^e.  448 = 1.75 * 2^8, so e is amax's own exponent minus 8,
// one more when its fraction is above 1.75 (0x600000); the carry of the
// addition is that comparison.  amax 0 and magnitudes below 2^-119 take
// e = -127.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const int e = static_cast<int>((amax_bits + 0x1FFFFFu) >> 23) - 8;
  return static_cast<uint32_t>(e < 0 ? 0 : e);
}
// 2^(127 - byte) as a float: exact, normal for the bytes scale_byte returns (0..247).
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
#endif

}  // namespace fp8
}  // namespace svdq
