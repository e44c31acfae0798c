// The block-scaled FP8 quantizer of one block of 128 elements, device side.
//
// Per row and 128 elements along K:
//   amax = largest finite |x|,  s = 2^e with the smallest e >= -127 such that
//   amax <= 448 * 2^e,          code = e4m3(x / s), round to nearest even.
// s is a power of two, so x / s is exact and the code carries the only
// rounding (relative 2^-4 of a normal code); nothing saturates.  A power of
// two instead of amax / 448 costs no precision (e4m3 codes keep their relative
// step over 2^-6..448) and is what the tensor cores take as a block scale, so
// the GEMM needs no rescaling pass.  Infinities and NaN become the NaN code: an
// e4m3 has no infinity, and the row's products are NaN either way.
#pragma once

#include <cuda_runtime.h>

#include "device_common.cuh"

namespace svdq {
namespace fp8 {

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

// e4m3 codes of two values, the first in the low byte (RNE, satfinite; NaN gives the NaN code).
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float nan_if_infinite(float v) {
  return fabsf(v) == __uint_as_float(0x7F800000u) ? __uint_as_float(0x7FC00000u) : v;
}
// |x| of both bf16 halves of a word as integers; non-finite halves become 0.
__device__ __forceinline__ uint32_t finite_abs2(uint32_t w) {
  uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
  lo = lo >= 0x7F80u ? 0u : lo;
  hi = hi >= 0x7F80u ? 0u : hi;
  return lo | (hi << 16);
}

// Called by a full warp: each 8 consecutive lanes hold one block of 128, 16
// elements (8 words of bf16 pairs) a lane.  Returns the block's scale byte and
// the lane's 16 codes.
__device__ __forceinline__ uint32_t quantize16(const uint32_t (&w)[8], uint32_t (&out)[4]) {
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
  uint32_t top = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const bool odd = top >= 0x7F80u;          // a non-finite element in this block
  if (__any_sync(0xFFFFFFFFu, odd)) {       // rare: the maximum again, over the finite elements
    uint32_t f2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) f2 = __vmaxu2(f2, finite_abs2(w[i]));
    top = max(f2 & 0xFFFFu, f2 >> 16);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  }
  const uint32_t byte = scale_byte(top << 16);
  const float inv = inverse_scale(byte);
  const float2 inv2 = make_float2(inv, inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f[j] = make_float2(__uint_as_float(w[2 * i + j] << 16), __uint_as_float(w[2 * i + j] & 0xFFFF0000u));
      if (odd) f[j] = make_float2(nan_if_infinite(f[j].x), nan_if_infinite(f[j].y));
      f[j] = dev::mul2_rn(f[j], inv2);
    }
    out[i] = cvt_e4m3x2(f[0].x, f[0].y) | (cvt_e4m3x2(f[1].x, f[1].y) << 16);
  }
  return byte;
}

}  // namespace fp8
}  // namespace svdq
