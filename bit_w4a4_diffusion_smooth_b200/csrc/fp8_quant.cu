// Block-scaled FP8 operands: the activation quantizer and the weight pack.
//
// Both quantize blocks of 128 elements along K (fp8_quant.cuh): of an
// activation row, and of an output column of the weight.
#include <cuda_runtime.h>

#include <string>

#include "device_common.cuh"
#include "fp8_layout.h"
#include "fp8_quant.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace fp8 {
namespace {

// One warp per (row, scale word): 512 elements, 16 per lane, so 8 lanes hold a
// block of 128.  Two 16-byte loads and one 16-byte store per lane.  The place
// in the sequence moves by increments: its division had been half of the
// kernel's instructions (4608 x 2560: 7.7 us, 68% of issue slots).
constexpr int QUANT_THREADS = 256;

__global__ void __launch_bounds__(QUANT_THREADS)
    quantize_act_kernel(const uint16_t *X, int M, int K, size_t ldx, int KS, int KW, int Mp, uint8_t *codes,
                        uint32_t *scales) {
  dev::grid_dependency_wait();
  dev::grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int warps = static_cast<int>(gridDim.x) * (QUANT_THREADS / 32);
  const int at = static_cast<int>(blockIdx.x) * (QUANT_THREADS / 32) + static_cast<int>(threadIdx.x >> 5);
  const int rows_on = warps / KW, words_on = warps % KW;
  int row = at / KW, kw = at % KW;
  for (; row < M; row += rows_on, kw += words_on) {
    if (kw >= KW) {
      kw -= KW;
      if (++row >= M) break;
    }
    const int k0 = kw * 512 + lane * 16;
    const uint16_t *src = X + static_cast<size_t>(row) * ldx + k0;
    uint4 v[2];
    v[0] = k0 < K ? __ldcg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0, 0, 0, 0);
    v[1] = k0 + 8 < K ? __ldcg(reinterpret_cast<const uint4 *>(src + 8)) : make_uint4(0, 0, 0, 0);
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t out[4];
    const uint32_t byte = quantize16(w, out);
    const int ks = kw * 4 + (lane >> 3), chunk = lane & 7;
    if (ks < KS)
      *reinterpret_cast<uint4 *>(codes + (static_cast<size_t>(ks) * Mp + row) * kBlock + ((chunk ^ (row & 7)) << 4)) =
          make_uint4(out[0], out[1], out[2], out[3]);
    uint32_t word = byte << (8 * (lane >> 3));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 16);
    if (lane == 0) scales[static_cast<size_t>(kw) * Mp + row] = word;
  }
}

// Weight pack: one block per (k-stage, 128 output columns, expert), a thread
// per output column, which reads its 128 elements down K (a warp's reads of one
// k are 64 contiguous bytes) and keeps them in registers between the maximum
// and the codes.  Run once per layer.
constexpr int PACK_COLS = 128;

__global__ void __launch_bounds__(PACK_COLS)
    pack_weights_kernel(const uint16_t *W, int K, int N, size_t ldw, size_t stride_e, int KS, int KW, uint8_t *codes,
                        uint8_t *scales) {
  const int ks = blockIdx.x, e = blockIdx.z;
  const int n = blockIdx.y * PACK_COLS + threadIdx.x;
  if (n >= N) return;
  const uint16_t *src = W + static_cast<size_t>(e) * stride_e + n;
  uint32_t w[64];
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const int k = ks * kBlock + 2 * i;           // K % 8 == 0: both or neither
    const uint32_t lo = k < K ? __ldg(src + static_cast<size_t>(k) * ldw) : 0u;
    const uint32_t hi = k < K ? __ldg(src + static_cast<size_t>(k + 1) * ldw) : 0u;
    w[i] = lo | (hi << 16);
    m2 = __vmaxu2(m2, finite_abs2(w[i]));
  }
  const uint32_t byte = scale_byte(max(m2 & 0xFFFFu, m2 >> 16) << 16);
  const float inv = inverse_scale(byte);
  uint8_t *dst = codes + ((static_cast<size_t>(e) * KS + ks) * N + n) * kBlock;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = w[8 * c + 2 * i], b = w[8 * c + 2 * i + 1];
      out[i] = cvt_e4m3x2(__fmul_rn(nan_if_infinite(__uint_as_float(a << 16)), inv),
                          __fmul_rn(nan_if_infinite(__uint_as_float(a & 0xFFFF0000u)), inv)) |
               (cvt_e4m3x2(__fmul_rn(nan_if_infinite(__uint_as_float(b << 16)), inv),
                           __fmul_rn(nan_if_infinite(__uint_as_float(b & 0xFFFF0000u)), inv))
                << 16);
    }
    *reinterpret_cast<uint4 *>(dst + ((c ^ (n & 7)) << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
  }
  uint8_t *word = scales + ((static_cast<size_t>(e) * gridDim.y + blockIdx.y) * KW + ks / 4) * kScaleAtom +
                  (threadIdx.x & 31) * 16 + (threadIdx.x >> 5) * 4;
  word[ks & 3] = static_cast<uint8_t>(byte);
  if (ks == KS - 1)                              // the blocks past K of the last word
    for (int j = (ks & 3) + 1; j < 4; ++j) word[j] = 127;
}

}  // namespace

int launch_quantize_act(const char *fn, const void *X, int M, int K, int ldx, void *workspace, int sm_count,
                        cudaStream_t stream) {
  const int KS = k_stages(K), KW = k_words(K), Mp = padded_rows(M);
  const long long total = static_cast<long long>(M) * KW;
  const long long blocks = (total + QUANT_THREADS / 32 - 1) / (QUANT_THREADS / 32);
  const long long most = 8ll * sm_count;       // 64 warps an SM, the rest in turn
  DependentLaunch dl(dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(QUANT_THREADS), 0, stream);
  uint8_t *codes = static_cast<uint8_t *>(workspace);
  cudaError_t e = cudaLaunchKernelEx(&dl.cfg, quantize_act_kernel, static_cast<const uint16_t *>(X), M, K,
                                     static_cast<size_t>(ldx), KS, KW, Mp, codes,
                                     reinterpret_cast<uint32_t *>(codes + act_code_bytes(M, K)));
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string(fn) + " launch: " + cudaGetErrorString(e));
  return SVDQ_OK;
}

}  // namespace fp8
}  // namespace svdq

using namespace svdq;

extern "C" int fp8_weight_size(int K, int N, int experts, size_t *bytes) {
  if (!bytes) return fail(SVDQ_ERR_INVALID_ARG, "fp8_weight_size: null pointer");
  if (K < 8 || K % 8 || N < 8 || N % 8 || experts < 1 || experts > FP8_MAX_EXPERTS)
    return fail(SVDQ_ERR_SHAPE, "fp8_weight_size: need K % 8 == 0, N % 8 == 0, 1 <= experts <= 512");
  *bytes = fp8::weight_bytes(K, N, experts);
  return ok();
}

extern "C" int fp8_workspace_size(int M, int K, int experts, size_t *bytes) {
  if (!bytes) return fail(SVDQ_ERR_INVALID_ARG, "fp8_workspace_size: null pointer");
  if (M < 1 || M > FP8_MAX_ROWS || K < 8 || K % 8 || experts < 1 || experts > FP8_MAX_EXPERTS)
    return fail(SVDQ_ERR_SHAPE, "fp8_workspace_size: need 1 <= M <= 2^30, K % 8 == 0, 1 <= experts <= 512");
  *bytes = fp8::needs_workspace(M, experts) ? fp8::act_bytes(M, K) : 0;
  return ok();
}

extern "C" int fp8_pack_weights(const void *W, int K, int N, int ldw, int64_t expert_stride, int experts, void *packed,
                                svdq_stream_t stream) {
  if (!W || !packed) return fail(SVDQ_ERR_INVALID_ARG, "fp8_pack_weights: null pointer");
  if (K < 8 || K % 8 || N < 8 || N % 8 || experts < 1 || experts > FP8_MAX_EXPERTS || ldw < N ||
      (experts > 1 && expert_stride < 0) || N > 8388480)
    return fail(SVDQ_ERR_SHAPE,
                "fp8_pack_weights: need K % 8 == 0, N % 8 == 0, N <= 8388480, ldw >= N, 1 <= experts <= 512");
  if (!aligned16(packed)) return fail(SVDQ_ERR_ALIGNMENT, "fp8_pack_weights: packed must be 16-byte aligned");
  if (!current_device_state()) return SVDQ_ERR_NOT_INITIALIZED;
  const int KS = fp8::k_stages(K), KW = fp8::k_words(K);
  const int blocks_n = (N + fp8::PACK_COLS - 1) / fp8::PACK_COLS;
  uint8_t *codes = static_cast<uint8_t *>(packed);
  fp8::pack_weights_kernel<<<dim3(KS, blocks_n, experts), fp8::PACK_COLS, 0, stream>>>(
      static_cast<const uint16_t *>(W), K, N, static_cast<size_t>(ldw), static_cast<size_t>(expert_stride), KS, KW,
      codes, codes + fp8::weight_code_bytes(K, N, experts));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string("fp8_pack_weights launch: ") + cudaGetErrorString(e));
  return ok();
}
