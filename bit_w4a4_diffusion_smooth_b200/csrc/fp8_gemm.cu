// Block-scaled FP8 GEMM: entry points and the kernel.
//
// One CTA computes 128 output columns (the MMA's M: lanes of tensor memory)
// by TOK rows of X (the MMA's N: columns of tensor memory).  With the weight on
// the M side a call of a few rows multiplies few rows: TOK goes down to 16, and
// such a call is bound by one pass over the weight, not by MMAs on padding.
//
// Roles (one CTA per SM, persistent over units of work, 8 warps):
//   warp 0     producer: per k-stage the 16 KB weight tile and TOK x 128 bytes
//              of activation codes, one bulk copy each (both are stored as
//              their shared-memory images)
//   warp 1     owns TMEM; one thread copies the scale words into TMEM
//              (tcgen05.cp, every fourth stage) and issues the MMAs
//   warp 2     brings the scale words of the next four stages into shared
//              memory in the copy's layout
//   warps 4-7  epilogue: drain the accumulator (two of them in TMEM, so the
//              next unit's MMAs run meanwhile), bias, GELU, bf16, and turn
//              the tile through shared memory into 16-byte row segments
// Every wait is bounded; one that runs out records SVDQ_ERR_TIMEOUT, raises
// the abort flag, and the CTA drains its copies and MMAs, frees TMEM and ends.
#include <cuda_runtime.h>

#include <string>

#include "fp8_gemm.cuh"

namespace svdq {
namespace fp8 {

int launch_quantize_act(const char *fn, const void *X, int M, int K, int ldx, void *workspace, int sm_count,
                        cudaStream_t stream);
int launch_gemm_pair(const char *fn, const Params &p, int epilogue, int sm_count, cudaStream_t stream);

namespace {

constexpr int THREADS = 256;
constexpr int EPI_WARPS = 4;
constexpr int SF_BUFS = 4;                     // scale words of 4 x 4 k-stages
constexpr int SF_BYTES = 2 * kScaleAtom;       // weight atom, activation atom
constexpr int EPI_STAGE = 32 * 64;             // a warp's 32 rows x 32 columns of bf16

template <int TOK>
struct Shape {
  static constexpr int STAGE = kTileBytes + TOK * kBlock;
  // as many stages as 196 KB holds: each is one 16 KB weight tile in flight
  static constexpr int STAGES = (196 * 1024) / STAGE;
  static constexpr int SF_OFF = STAGES * STAGE;
  static constexpr int EPI_OFF = SF_OFF + SF_BUFS * SF_BYTES;
  static constexpr int TAB_OFF = EPI_OFF + EPI_WARPS * EPI_STAGE;
  static constexpr int BAR_OFF = (TAB_OFF + static_cast<int>(sizeof(ExpertTable)) + 15) & ~15;
  static constexpr int BYTES = 1024 + BAR_OFF + 512;
  static constexpr uint32_t SF_COL = 2 * TOK;  // behind the two accumulators; 8 columns a buffer
  static constexpr uint32_t TMEM_COLS = TOK <= 16 ? 64 : TOK == 32 ? 128 : TOK == 64 ? 256 : 512;
  static_assert(STAGE % 1024 == 0, "operand tiles start on 1024-byte boundaries");
  static_assert(SF_COL + 8 * SF_BUFS <= TMEM_COLS, "accumulators and scales fit in TMEM");
  static_assert(BYTES <= 232448, "fits in shared memory");
};

template <int TOK, int EPI>
__global__ void __launch_bounds__(THREADS, 1) fp8_gemm_kernel(const __grid_constant__ Params p) {
  using S = Shape<TOK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::BAR_OFF);
  uint64_t *empty = full + S::STAGES;
  uint64_t *sf_full = empty + S::STAGES;
  uint64_t *sf_empty = sf_full + SF_BUFS;
  uint64_t *tmem_full = sf_empty + SF_BUFS;
  uint64_t *tmem_empty = tmem_full + 2;
  uint64_t *drain = tmem_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  ExpertTable *tab = reinterpret_cast<ExpertTable *>(smem + S::TAB_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      dev::mbar_init(&full[s], 1);
      dev::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < SF_BUFS; ++b) {
      dev::mbar_init(&sf_full[b], 1);
      dev::mbar_init(&sf_empty[b], 1);
    }
    for (int a = 0; a < 2; ++a) {
      dev::mbar_init(&tmem_full[a], 1);
      dev::mbar_init(&tmem_empty[a], EPI_WARPS);
    }
    dev::mbar_init(drain, 1);
    *abort_flag = 0;
    dev::fence_mbar_init();
  }
  if (warp == 1) {
    dev::tmem_alloc(tmem_slot, S::TMEM_COLS);
    dev::tmem_relinquish();
  }
  dev::grid_dependency_wait();
  dev::grid_launch_dependents();
  if (warp == 2) fill_expert_table(p, TOK, tab);
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int items = tab->tiles[p.experts] * p.ntn;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      int it = 0;
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const Item u = find_item(p, tab, TOK, p.ntn, item);
        const uint8_t *wsrc = p.w + (static_cast<size_t>(u.expert) * p.ntn + u.nt) * p.KS * kTileBytes;
        const uint8_t *xsrc = p.x + static_cast<size_t>(u.row0) * kBlock;
        // rows past the end of the buffer are not copied: what the stage holds there reaches no output
        const uint32_t xbytes = static_cast<uint32_t>(min(TOK, p.Mp - u.row0)) * kBlock;
        for (int ks = 0; ks < p.KS; ++ks, ++it) {
          const int s = it % S::STAGES;
          if (!dev::mbar_wait(&empty[s], ((it / S::STAGES) & 1) ^ 1, p.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t *dst = smem + s * S::STAGE;
          dev::mbar_arrive_expect_tx(&full[s], kTileBytes + xbytes);
          dev::bulk_load(dst, wsrc + static_cast<size_t>(ks) * kTileBytes, kTileBytes, &full[s]);
          dev::bulk_load(dst + kTileBytes, xsrc + static_cast<size_t>(ks) * p.Mp * kBlock, xbytes, &full[s]);
        }
      }
      if (!ok) {
        *abort_flag = 1;
        dev::report(p.status, SVDQ_ERR_TIMEOUT);
      }
      for (int j = max(0, it - S::STAGES); j < it; ++j)   // every copy in flight lands before the CTA ends
        dev::mbar_wait(&full[j % S::STAGES], (j / S::STAGES) & 1, p.limit_ns, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ scales into TMEM, MMAs
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_mxf8(kTileN, TOK);
      int it = 0, quad = 0, n = 0;
      bool ok = true, issued = false;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x, ++n) {
        const int a = n & 1;
        if (!dev::mbar_wait(&tmem_empty[a], ((n >> 1) & 1) ^ 1, p.limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        dev::tc_fence_after();
        const uint32_t acc = tmem + a * TOK;
        uint32_t sfa = 0, sfb = 0;
        for (int ks = 0; ks < p.KS; ++ks, ++it) {
          const int s = it % S::STAGES, b = quad % SF_BUFS;
          if ((ks & 3) == 0) {
            if (!dev::mbar_wait(&sf_full[b], (quad / SF_BUFS) & 1, p.limit_ns, abort_flag)) {
              ok = false;
              break;
            }
            dev::tc_fence_after();
            const uint32_t src = dev::smem_u32(smem + S::SF_OFF + b * SF_BYTES);
            sfa = tmem + S::SF_COL + 8 * b;
            sfb = sfa + 4;
            dev::tmem_cp_32x128b_x4(sfa, dev::desc_sf(src));
            dev::tmem_cp_32x128b_x4(sfb, dev::desc_sf(src + kScaleAtom));
            issued = true;
          }
          if (!dev::mbar_wait(&full[s], (it / S::STAGES) & 1, p.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          dev::tc_fence_after();
          const uint32_t sw = dev::smem_u32(smem + s * S::STAGE), sx = sw + kTileBytes;
          const uint32_t id = with_scale_byte(idesc, static_cast<uint32_t>(ks & 3));
#pragma unroll
          for (int j = 0; j < 4; ++j)                     // K = 32 codes = 32 bytes per MMA
            umma_mxf8(acc, dev::desc_sw128(sw + 32 * j), dev::desc_sw128(sx + 32 * j), id, sfa, sfb,
                      ks > 0 || j > 0 ? 1u : 0u);
          dev::tc_commit(&empty[s]);
          if ((ks & 3) == 3 || ks == p.KS - 1) {
            dev::tc_commit(&sf_empty[b]);
            ++quad;
          }
        }
        if (!ok) break;
        dev::tc_commit(&tmem_full[a]);
      }
      if (!ok) {
        *abort_flag = 1;
        dev::report(p.status, SVDQ_ERR_TIMEOUT);
      }
      if (issued) {                                       // the tensor core is idle before TMEM is freed
        dev::tc_commit(drain);
        dev::mbar_wait(drain, 0, p.limit_ns, nullptr);
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ scale words
    int quad = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const Item u = find_item(p, tab, TOK, p.ntn, item);
      const uint8_t *wsrc = p.sw + (static_cast<size_t>(u.expert) * p.ntn + u.nt) * p.KW * kScaleAtom;
      for (int kw = 0; kw < p.KW; ++kw, ++quad) {
        const int b = quad % SF_BUFS;
        const uint4 wa = __ldg(reinterpret_cast<const uint4 *>(wsrc + static_cast<size_t>(kw) * kScaleAtom) + lane);
        const uint32_t *xs = p.sx + static_cast<size_t>(kw) * p.Mp;
        uint32_t xw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = u.row0 + 32 * i + lane;
          xw[i] = 32 * i + lane < TOK && row < p.Mp ? xs[row] : 0u;
        }
        if (!dev::mbar_wait_warp(&sf_empty[b], ((quad / SF_BUFS) & 1) ^ 1, p.limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t *dst = smem + S::SF_OFF + b * SF_BYTES;
        reinterpret_cast<uint4 *>(dst)[lane] = wa;
        reinterpret_cast<uint4 *>(dst + kScaleAtom)[lane] = make_uint4(xw[0], xw[1], xw[2], xw[3]);
        dev::fence_proxy_async();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&sf_full[b]);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      dev::report(p.status, SVDQ_ERR_TIMEOUT);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                               // TMEM lane quarter this warp may access
    uint8_t *stage = smem + S::EPI_OFF + q * EPI_STAGE;
    int n = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x, ++n) {
      const Item u = find_item(p, tab, TOK, p.ntn, item);
      const int a = n & 1, col0 = u.nt * kTileN + 32 * q, col = col0 + lane;
      float bias = 0.0f;
      if (p.bias && col < p.N)
        bias = __uint_as_float(static_cast<uint32_t>(__ldg(p.bias + static_cast<size_t>(u.expert) * p.N + col)) << 16);
      const bool act = col >= p.gelu_col_begin;
      if (!dev::mbar_wait_warp(&tmem_full[a], (n >> 1) & 1, p.limit_ns, abort_flag)) {
        if (lane == 0) {
          *abort_flag = 1;
          dev::report(p.status, SVDQ_ERR_TIMEOUT);
        }
        break;
      }
      dev::tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(a * TOK);
      constexpr int CH = TOK < 32 ? TOK : 32;             // rows per chunk
#pragma unroll 1
      for (int c = 0; c < TOK; c += CH) {
        if (u.row0 + c >= u.end) break;                   // no row of this expert from here on
        uint32_t v[CH];
        if constexpr (CH == 32) dev::tmem_ld_32x32b_x32(taddr + c, v);
        else tmem_ld_32x32b_x16(taddr + c, v);
        dev::tmem_wait_ld();
#pragma unroll
        for (int t = 0; t < CH; t += 2) {
          const float2 y = make_float2(__uint_as_float(v[t]) + bias, __uint_as_float(v[t + 1]) + bias);
          float2 g = activate2<EPI>(y);
          if constexpr (EPI != SVDQ_EPILOGUE_NONE) {
            g.x = act ? g.x : y.x;
            g.y = act ? g.y : y.y;
          }
          reinterpret_cast<__nv_bfloat16 *>(stage + t * 64)[lane] = __float2bfloat16_rn(g.x);
          reinterpret_cast<__nv_bfloat16 *>(stage + (t + 1) * 64)[lane] = __float2bfloat16_rn(g.y);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < CH / 8; ++i) {                // 8 rows x 4 segments of 16 bytes
          const int t = 8 * i + (lane >> 2), seg = lane & 3, row = u.row0 + c + t;
          if (row >= u.begin && row < u.end && col0 + 8 * seg < p.N)
            *reinterpret_cast<uint4 *>(p.Y + static_cast<size_t>(row) * p.ldy + col0 + 8 * seg) =
                *reinterpret_cast<const uint4 *>(stage + t * 64 + seg * 16);
        }
        __syncwarp();
      }
      dev::tc_fence_before();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&tmem_empty[a]);
    }
  }

  dev::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    dev::tc_fence_after();
    dev::tmem_dealloc(tmem, S::TMEM_COLS);
  }
}

template <int TOK, int EPI>
int launch(const char *fn, const Params &p, long long units, int sm_count, cudaStream_t stream) {
  int rc = smem_optin_once<fp8_gemm_kernel<TOK, EPI>>(Shape<TOK>::BYTES, fn);
  if (rc != SVDQ_OK) return rc;
  const int grid = units < sm_count ? static_cast<int>(units) : sm_count;
  DependentLaunch dl(dim3(grid), dim3(THREADS), Shape<TOK>::BYTES, stream);
  cudaError_t e = cudaLaunchKernelEx(&dl.cfg, fp8_gemm_kernel<TOK, EPI>, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string(fn) + " launch: " + cudaGetErrorString(e));
  return SVDQ_OK;
}
template <int TOK>
int launch(const char *fn, const Params &p, int epilogue, long long units, int sm_count, cudaStream_t stream) {
  return epilogue == SVDQ_EPILOGUE_GELU_ERF    ? launch<TOK, SVDQ_EPILOGUE_GELU_ERF>(fn, p, units, sm_count, stream)
         : epilogue == SVDQ_EPILOGUE_GELU_TANH ? launch<TOK, SVDQ_EPILOGUE_GELU_TANH>(fn, p, units, sm_count, stream)
                                               : launch<TOK, SVDQ_EPILOGUE_NONE>(fn, p, units, sm_count, stream);
}

int run(const char *fn, const void *X, int M, int K, int ldx, const int *offsets, int experts, const void *packed,
        const void *bias, int N, int epilogue, int gelu_col_begin, void *Y, int ldy, void *workspace,
        cudaStream_t stream) {
  const std::string name(fn);
  if (!X || !packed || !Y || !workspace) return fail(SVDQ_ERR_INVALID_ARG, name + ": null pointer");
  if (epilogue < SVDQ_EPILOGUE_NONE || epilogue > SVDQ_EPILOGUE_GELU_TANH)
    return fail(SVDQ_ERR_INVALID_ARG, name + ": unknown epilogue");
  if (M < 1 || K < 8 || K % 8 || N < 8 || N % 8 || ldx < K || ldx % 8 || ldy < N || ldy % 8)
    return fail(SVDQ_ERR_SHAPE, name + ": need M >= 1, K % 8 == 0, N % 8 == 0, ldx >= K, ldy >= N, ldx % 8 == 0, "
                                       "ldy % 8 == 0");
  if (experts < 1 || experts > FP8_MAX_EXPERTS) return fail(SVDQ_ERR_SHAPE, name + ": need 1 <= experts <= 512");
  if (gelu_col_begin < 0 || gelu_col_begin > N) return fail(SVDQ_ERR_SHAPE, name + ": gelu_col_begin outside [0, N]");
  // units of work are counted in int, with room for the tiles that ragged experts add
  if ((static_cast<long long>(M) / 16 + 2ll * experts) * n_tiles(N) > 0x3FFFFFFFll)
    return fail(SVDQ_ERR_SHAPE, name + ": M x N is too large");
  if (!aligned16(X) || !aligned16(packed) || !aligned16(Y) || !aligned16(workspace))
    return fail(SVDQ_ERR_ALIGNMENT, name + ": pointers must be 16-byte aligned");
  DeviceState *st = current_device_state();
  if (!st) return SVDQ_ERR_NOT_INITIALIZED;
  int rc = launch_quantize_act(fn, X, M, K, ldx, workspace, st->sm_count, stream);
  if (rc != SVDQ_OK) return rc;

  Params p{};
  p.x = static_cast<const uint8_t *>(workspace);
  p.sx = reinterpret_cast<const uint32_t *>(p.x + act_code_bytes(M, K));
  p.w = static_cast<const uint8_t *>(packed);
  p.sw = p.w + weight_code_bytes(K, N, experts);
  p.bias = static_cast<const uint16_t *>(bias);
  p.Y = static_cast<uint16_t *>(Y);
  p.ldy = static_cast<size_t>(ldy);
  p.offsets = offsets;
  p.experts = experts;
  p.M = M;
  p.Mp = padded_rows(M);
  p.N = N;
  p.ntn = n_tiles(N);
  p.KS = k_stages(K);
  p.KW = k_words(K);
  p.gelu_col_begin = gelu_col_begin;
  p.status = st->status_word;
  p.limit_ns = kWaitLimitNs;
  // rows per token tile: the smallest that holds an expert's average share
  const long long share = (static_cast<long long>(M) + experts - 1) / experts;
  if (share > 128) {
    rc = launch_gemm_pair(fn, p, epilogue, st->sm_count, stream);
    return rc == SVDQ_OK ? ok() : rc;
  }
  const int tok = share <= 16 ? 16 : share <= 32 ? 32 : share <= 64 ? 64 : 128;
  const long long units = (static_cast<long long>(M) / tok + (experts > 1 ? 2ll * experts : 1)) * p.ntn;
  rc = tok == 16   ? launch<16>(fn, p, epilogue, units, st->sm_count, stream)
       : tok == 32 ? launch<32>(fn, p, epilogue, units, st->sm_count, stream)
       : tok == 64 ? launch<64>(fn, p, epilogue, units, st->sm_count, stream)
                   : launch<128>(fn, p, epilogue, units, st->sm_count, stream);
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
