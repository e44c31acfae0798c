// Block-scaled FP8 linear layer: the entry points.  Few rows (an average share
// of at most 128 an expert, more where its tiles fill the SMs better) run in the
// kernel of weight-bound calls, which quantizes X itself if they are very few;
// otherwise a quantizer runs in front, and many rows go through 256-row tiles
// on SM pairs.
#include <cuda_runtime.h>

#include <string>

#include "fp8_gemm.cuh"

namespace svdq {
namespace fp8 {

int launch_quantize_act(const char *fn, const void *X, int M, int K, int ldx, void *workspace, int sm_count,
                        cudaStream_t stream);
int launch_gemm_few(const char *fn, const Params &p, int tile, int epilogue, int sm_count, cudaStream_t stream);
int launch_gemm_pair(const char *fn, const Params &p, int epilogue, int sm_count, cudaStream_t stream);

namespace {

// Whether 128-row tiles of the few-row kernel beat 256-row tiles on SM pairs for more rows than 128.  Per stage of
// 128 along K a round of theirs takes about 0.285 us (a unit an SM) against 0.365 us (a unit a pair), and the pairs'
// start and end take 4 us more.  Measured, K = 2560, few rows / pairs: 256 rows -> 7680 11.7 / 15.5 us, 768 rows ->
// 7680 22.6 / 22.9 us, 512 rows -> 15360 28.2 / 24.1 us; 4096 -> 2560: 512 rows 14.5 / 18.5 us.
bool few_is_faster(const Params &p, int sm_count) {
  const long long half = p.offsets ? p.experts / 2 : 0;      // what ragged experts leave unfilled on average
  const long long few_tiles = p.offsets ? p.M / 128 + half + 1 : (p.M + 127) / 128;
  const long long pair_tiles = p.offsets ? p.M / 256 + half + 1 : (p.M + 255) / 256;
  const long long few_rounds = (few_tiles * ((p.N + 127) / 128) + sm_count - 1) / sm_count;
  const long long pairs = sm_count / 2, pair_rounds = (pair_tiles * ((p.N + 239) / 240) + pairs - 1) / pairs;
  return 57 * p.KS * few_rounds < 73 * p.KS * pair_rounds + 800;
}

// Whether an element of X [M][ldx], K columns, is one of Y [M][ldy], N columns.  Interleaved rows (one stride, columns
// apart) are not; with two strides, what lies inside the other's range counts as shared.
bool overlap(const void *X, int K, int ldx, const void *Y, int N, int ldy, int M) {
  const int64_t x = static_cast<int64_t>(reinterpret_cast<uintptr_t>(X)) / 2;
  const int64_t y = static_cast<int64_t>(reinterpret_cast<uintptr_t>(Y)) / 2;
  if (y >= x + static_cast<int64_t>(M - 1) * ldx + K || x >= y + static_cast<int64_t>(M - 1) * ldy + N) return false;
  if (M == 1 || ldx != ldy) return true;
  const int64_t at = ((y - x) % ldx + ldx) % ldx;            // Y's first column in X's rows
  return at < K || at + N > ldx;
}

int run(const char *fn, const void *X, int M, int K, int ldx, const int *offsets, int experts, const void *packed,
        const void *bias, int N, int epilogue, int gelu_col_begin, void *Y, int ldy, void *workspace,
        cudaStream_t stream) {
  const std::string name(fn);
  if (!X || !packed || !Y) return fail(SVDQ_ERR_INVALID_ARG, name + ": null pointer");
  if (epilogue < SVDQ_EPILOGUE_NONE || epilogue > SVDQ_EPILOGUE_GELU_TANH)
    return fail(SVDQ_ERR_INVALID_ARG, name + ": unknown epilogue");
  if (M < 1 || M > FP8_MAX_ROWS || K < 8 || K % 8 || N < 8 || N % 8 || ldx < K || ldx % 8 || ldy < N || ldy % 8)
    return fail(SVDQ_ERR_SHAPE, name + ": need 1 <= M <= 2^30, K % 8 == 0, N % 8 == 0, ldx >= K, ldy >= N, ldx % 8 == 0, "
                                       "ldy % 8 == 0");
  if (experts < 1 || experts > FP8_MAX_EXPERTS) return fail(SVDQ_ERR_SHAPE, name + ": need 1 <= experts <= 512");
  if (gelu_col_begin < 0 || gelu_col_begin > N) return fail(SVDQ_ERR_SHAPE, name + ": gelu_col_begin outside [0, N]");
  // units of work are counted in int, with room for the tiles that ragged experts add
  if ((static_cast<long long>(M) / 16 + 2ll * experts) * (N / 128 + 1) > 0x3FFFFFFFll)
    return fail(SVDQ_ERR_SHAPE, name + ": M x N is too large");
  const bool ws = needs_workspace(M, experts);
  if (ws && !workspace) return fail(SVDQ_ERR_INVALID_ARG, name + ": null pointer");
  if (!aligned16(X) || !aligned16(packed) || !aligned16(Y) || (ws && !aligned16(workspace)) ||
      (bias && !aligned16(bias)))
    return fail(SVDQ_ERR_ALIGNMENT, name + ": pointers must be 16-byte aligned");
  if (offsets && (reinterpret_cast<uintptr_t>(offsets) & 3u))
    return fail(SVDQ_ERR_ALIGNMENT, name + ": offsets must be 4-byte aligned");
  if (overlap(X, K, ldx, Y, N, ldy, M)) return fail(SVDQ_ERR_INVALID_ARG, name + ": Y overlaps X");
  DeviceState *st = current_device_state();
  if (!st) return SVDQ_ERR_NOT_INITIALIZED;

  Params p{};
  p.X = static_cast<const uint16_t *>(X);
  p.ldx = static_cast<size_t>(ldx);
  p.w = static_cast<const uint8_t *>(packed);
  p.sw = reinterpret_cast<const uint32_t *>(p.w + weight_code_bytes(K, N, experts));
  p.bias = static_cast<const uint16_t *>(bias);
  p.Y = static_cast<uint16_t *>(Y);
  p.ldy = static_cast<size_t>(ldy);
  p.offsets = offsets;
  p.experts = experts;
  p.M = M;
  p.Mp = padded_rows(M);
  p.N = N;
  p.K = K;
  p.KS = k_stages(K);
  p.KW = k_words(K);
  p.gelu_col_begin = gelu_col_begin;
  p.status = st->status_word;
  p.limit_ns = kWaitLimitNs;
  int rc = SVDQ_OK;
  if (ws) {
    p.x = static_cast<const uint8_t *>(workspace);
    p.sx = reinterpret_cast<const uint32_t *>(p.x + act_code_bytes(M, K));
    rc = launch_quantize_act(fn, X, M, K, ldx, workspace, st->sm_count, stream);
  }
  int tile = few_tile(M, experts);
  if (tile == 0 && few_is_faster(p, st->sm_count)) tile = 128;
  if (rc == SVDQ_OK)
    rc = tile ? launch_gemm_few(fn, p, tile, epilogue, st->sm_count, stream)
              : launch_gemm_pair(fn, p, epilogue, st->sm_count, stream);
  return rc == SVDQ_OK ? ok() : rc;
}

}  // namespace
}  // namespace fp8
}  // namespace svdq

using namespace svdq;

extern "C" int fp8_linear(const void *X, int M, int K, int ldx, const void *packed, const void *bias, int N,
                          int epilogue, int gelu_col_begin, void *Y, int ldy, void *workspace, svdq_stream_t stream) {
  return fp8::run("fp8_linear", X, M, K, ldx, nullptr, 1, packed, bias, N, epilogue, gelu_col_begin, Y, ldy, workspace,
                  stream);
}

extern "C" int fp8_linear_grouped(const void *X, int M, int K, int ldx, const int32_t *offsets, int experts,
                                  const void *packed, const void *bias, int N, int epilogue, int gelu_col_begin,
                                  void *Y, int ldy, void *workspace, svdq_stream_t stream) {
  if (!offsets) return fail(SVDQ_ERR_INVALID_ARG, "fp8_linear_grouped: null pointer");
  return fp8::run("fp8_linear_grouped", X, M, K, ldx, offsets, experts, packed, bias, N, epilogue, gelu_col_begin, Y,
                  ldy, workspace, stream);
}
