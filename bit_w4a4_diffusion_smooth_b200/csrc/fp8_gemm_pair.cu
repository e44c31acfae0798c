// Block-scaled FP8 GEMM for many rows: 256 x 240 output tiles on SM pairs.
//
// Clusters of two CTAs, one per SM of a TPC; every MMA is a cta_group::2 MMA
// of 256 x 240 x 32: CTA h holds rows 128h..128h+127 of the token tile and
// weight rows (output columns) 120h..120h+119, and its TMEM receives its own
// 128 rows of the accumulator, so each SM reads 248 operand rows per k-stage
// for 256 x 120 outputs.  (One CTA alone would read 256 for 128 x 128, and the
// operand traffic from L2 bounds it.)  240 columns instead of 256 leave TMEM
// room for two accumulators and the block scales: draining one (2,300 cycles a
// tile, 12% at K = 4096) runs under the next tile's MMAs.
//
// Roles (one CTA per SM, persistent over units of work, 12 warps):
//   warp 0      producer in both CTAs: per k-stage its halves of the two
//               operands, completing on the even CTA's `full` barrier
//   warp 1      owns TMEM (pair allocation); in the even CTA one thread issues
//               the MMAs and commits each stage to both CTAs
//   warp 2      scale words of the next four stages, in both CTAs: the words
//               of its own 128 token rows and of all 240 weight rows (which
//               both TMEMs need)
//   warp 3      even CTA: copies them into both TMEMs (tcgen05.cp)
//   warps 4-11  epilogue in both CTAs: 16 columns at a time from TMEM, bias,
//               GELU, bf16; a thread holds 32 contiguous bytes of its row and
//               stores them itself, whole sectors, so ragged ends are a
//               condition on its row
// Every wait is bounded; one that runs out records SVDQ_ERR_TIMEOUT and raises
// the abort flag of both CTAs; in-flight work is drained, the pair meets at a
// cluster barrier and frees TMEM.
#include <cuda_runtime.h>

#include <string>

#include "fp8_gemm.cuh"

namespace svdq {
namespace fp8 {
namespace {

constexpr int TOK = 256;                       // rows per pair tile
constexpr int TILE_N = 240;                    // output columns per pair tile
constexpr int STAGES = 6;
constexpr int X_BYTES = 128 * kBlock;          // this CTA's token rows of a stage
constexpr int W_BYTES = TILE_N / 2 * kBlock;   // this CTA's weight rows
constexpr int STAGE = X_BYTES + W_BYTES;
constexpr int SF_BUFS = 4;                     // scale words of 4 x 4 k-stages in shared memory
constexpr int SF_TMEM = 2;                     // ... of 2 x 4 in TMEM
constexpr int SF_BYTES = 3 * kScaleAtom;       // own token atom, the two weight atoms
constexpr int EPI_WARPS = 8;
constexpr int THREADS = (4 + EPI_WARPS) * 32;
constexpr int SF_OFF = STAGES * STAGE;
constexpr int TAB_OFF = SF_OFF + SF_BUFS * SF_BYTES;
constexpr int BAR_OFF = (TAB_OFF + static_cast<int>(sizeof(ExpertTable)) + 15) & ~15;
constexpr int SMEM_BYTES = 1024 + BAR_OFF + 256;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SF_COL = 2 * TILE_N;        // buffer b: token scales at +12b, weight scales at +12b + 4
constexpr int MAP_ROW = 1024;                  // the operands as rows of 8 x 128 bytes
static_assert(STAGE % 1024 == 0 && X_BYTES % 1024 == 0, "operand tiles start on 1024-byte boundaries");
static_assert(SMEM_BYTES <= 232448, "fits in shared memory");
static_assert(SF_COL + 12 * SF_TMEM <= TMEM_COLS, "accumulators and scales fit in TMEM");

struct Maps {
  CUtensorMap x, w;
};

__device__ __forceinline__ void umma_mxf8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}

// Row of the weights' tensor map where this CTA's rows of a unit's stage start.
__device__ __forceinline__ int weight_row(const Params &p, const Item &u, int ks, uint32_t h) {
  return (u.expert * p.KS + ks) * (p.N / 8) + (u.nt * TILE_N + static_cast<int>(h) * (TILE_N / 2)) / 8;
}

__device__ __forceinline__ void abort_pair(volatile int *abort_flag, uint32_t peer_abort, unsigned int *status) {
  *abort_flag = 1;
  dev::st_cluster_u32(peer_abort, 1u);
  dev::report(status, SVDQ_ERR_TIMEOUT);
}

// 32 bytes to a 32-byte aligned address.
__device__ __forceinline__ void store32(void *ptr, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(ptr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Bias, activation and rounding of 16 columns from `col` on, stored to row `y` if `row_ok`; `wide`: rows of Y
// are 32-byte aligned.
template <int EPI>
__device__ __forceinline__ void finish16(const Params &p, const uint16_t *bias, const uint32_t (&v)[16], int col,
                                         uint16_t *y, bool row_ok, bool wide) {
  uint32_t out[8];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint4 bb = make_uint4(0, 0, 0, 0);
    if (bias && col + 8 * g < p.N) bb = __ldg(reinterpret_cast<const uint4 *>(bias + col + 8 * g));   // N % 8 == 0
    const uint32_t bw[4] = {bb.x, bb.y, bb.z, bb.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = 8 * g + 2 * j;
      const float2 t = make_float2(__uint_as_float(v[i]) + __uint_as_float(bw[j] << 16),
                                   __uint_as_float(v[i + 1]) + __uint_as_float(bw[j] & 0xFFFF0000u));
      float2 a = activate2<EPI>(t);
      if constexpr (EPI != SVDQ_EPILOGUE_NONE) {
        a.x = col + i >= p.gelu_col_begin ? a.x : t.x;
        a.y = col + i + 1 >= p.gelu_col_begin ? a.y : t.y;
      }
      const __nv_bfloat162 hv = __floats2bfloat162_rn(a.x, a.y);
      out[4 * g + j] = *reinterpret_cast<const uint32_t *>(&hv);
    }
  }
  if (!row_ok) return;
  if (wide && col + 16 <= p.N) {
    store32(y + col, out);
  } else {
    if (col < p.N) *reinterpret_cast<uint4 *>(y + col) = make_uint4(out[0], out[1], out[2], out[3]);
    if (col + 8 < p.N) *reinterpret_cast<uint4 *>(y + col + 8) = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    fp8_gemm_pair_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + BAR_OFF);   // even CTA: both CTAs' bytes
  uint64_t *empty = full + STAGES;                                  // both CTAs: stage free again
  uint64_t *sf_full = empty + STAGES;                               // even CTA: both CTAs' scale words
  uint64_t *sf_empty = sf_full + SF_BUFS;                           // both CTAs: their copy into TMEM is done
  uint64_t *sft_full = sf_empty + SF_BUFS;                          // even CTA: scale words in both TMEMs
  uint64_t *sft_empty = sft_full + SF_TMEM;                         // even CTA: their MMAs are done
  uint64_t *tmem_full = sft_empty + SF_TMEM;                       // both CTAs: accumulator ready
  uint64_t *tmem_empty = tmem_full + 2;                             // even CTA: both CTAs drained it
  uint64_t *drain = tmem_empty + 2;
  uint64_t *drain_cp = drain + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain_cp + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  ExpertTable *tab = reinterpret_cast<ExpertTable *>(smem + TAB_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t h = dev::cluster_ctarank();         // 0: even CTA (issues the MMAs), 1: odd
  const int pair = static_cast<int>(dev::cluster_id_x());
  const int pairs = static_cast<int>(dev::num_clusters_x());
  const int ntn = (p.N + TILE_N - 1) / TILE_N;
  const uint32_t peer_abort = dev::mapa(dev::smem_u32(const_cast<int *>(abort_flag)), h ^ 1u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      dev::mbar_init(&full[s], 1);
      dev::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < SF_BUFS; ++b) {
      dev::mbar_init(&sf_full[b], 2);
      dev::mbar_init(&sf_empty[b], 1);
    }
    for (int b = 0; b < SF_TMEM; ++b) {
      dev::mbar_init(&sft_full[b], 1);
      dev::mbar_init(&sft_empty[b], 1);
    }
    for (int a = 0; a < 2; ++a) {
      dev::mbar_init(&tmem_full[a], 1);
      dev::mbar_init(&tmem_empty[a], 2 * EPI_WARPS);
    }
    dev::mbar_init(drain, 1);
    dev::mbar_init(drain_cp, 1);
    *abort_flag = 0;
    dev::fence_mbar_init();
  }
  if (warp == 1) {
    dev::tmem_alloc_pair(tmem_slot, TMEM_COLS);
    dev::tmem_relinquish_pair();
  }
  if (warp == 2) fill_expert_table(p, TOK, 8, tab);
  dev::tc_fence_before();
  __syncwarp();
  dev::cluster_sync();                               // both CTAs' barriers exist before anyone arrives remotely
  dev::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int items = tab->tiles[p.experts] * ntn;
  dev::grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (elect_one()) {
      dev::prefetch_tmap(&maps.x);
      dev::prefetch_tmap(&maps.w);
      // the weights of the first unit's first stages, before the activations are there to wait for
      int ahead = 0;
      if (pair < items) {
        const Item u = find_item(p, tab, TOK, 8, ntn, pair);
        for (; ahead < min(STAGES, p.KS); ++ahead) {
          if (h == 0) dev::mbar_arrive_expect_tx(&full[ahead], 2u * STAGE);
          dev::tma_load_2d_pair(smem + ahead * STAGE + X_BYTES, &maps.w, dev::mapa(dev::smem_u32(&full[ahead]), 0), 0,
                                weight_row(p, u, ahead, h));
        }
      }
      dev::grid_dependency_wait();
      int it = 0;
      bool ok = true;
      for (int item = pair; item < items && ok; item += pairs) {
        const Item u = find_item(p, tab, TOK, 8, ntn, item);
        const int xrow = u.row0 / 8 + 16 * static_cast<int>(h);
        for (int ks = 0; ks < p.KS; ++ks, ++it) {
          const int s = it % STAGES;
          const uint32_t bar = dev::mapa(dev::smem_u32(&full[s]), 0);
          uint8_t *dst = smem + s * STAGE;
          // rows past the end of a stage's rows hold the next stage's, past the buffer zeros: neither reaches
          // an output
          if (it >= ahead) {
            if (!dev::mbar_wait_cluster(&empty[s], ((it / STAGES) & 1) ^ 1, p.limit_ns, abort_flag)) {
              ok = false;
              break;
            }
            if (h == 0) dev::mbar_arrive_expect_tx(&full[s], 2u * STAGE);
            dev::tma_load_2d_pair(dst + X_BYTES, &maps.w, bar, 0, weight_row(p, u, ks, h));
          }
          dev::tma_load_2d_pair(dst, &maps.x, bar, 0, xrow + ks * (p.Mp / 8));
        }
      }
      if (!ok) abort_pair(abort_flag, peer_abort, p.status);
      // before the pair may leave, every stage the even CTA armed completes (the odd CTA's copies with it)
      if (h == 0)
        for (int j = max(0, it - STAGES); j < it; ++j)
          dev::mbar_wait_cluster(&full[j % STAGES], (j / STAGES) & 1, p.limit_ns, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ scales into TMEM, MMAs (even CTA)
    if (h == 0 && elect_one()) {
      constexpr uint32_t idesc = idesc_mxf8(TOK, TILE_N);
      int it = 0, quad = 0, n = 0;
      bool ok = true, issued = false;
      for (int item = pair; item < items && ok; item += pairs, ++n) {
        const int a = n & 1;
        if (!dev::mbar_wait_cluster(&tmem_empty[a], ((n >> 1) & 1) ^ 1, p.limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        dev::tc_fence_after();
        const uint32_t acc = tmem + a * TILE_N;
        uint32_t sfx = 0, sfw = 0;
        for (int ks = 0; ks < p.KS; ++ks, ++it) {
          const int s = it % STAGES, b = quad % SF_TMEM;
          if ((ks & 3) == 0) {
            if (!dev::mbar_wait(&sft_full[b], (quad / SF_TMEM) & 1, p.limit_ns, abort_flag)) {
              ok = false;
              break;
            }
            sfx = tmem + SF_COL + 12 * b;
            sfw = sfx + 4;
          }
          if (!dev::mbar_wait_cluster(&full[s], (it / STAGES) & 1, p.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          dev::tc_fence_after();
          const uint32_t sx = dev::smem_u32(smem + s * STAGE), sw = sx + X_BYTES;
          const uint32_t id = with_scale_bytes(idesc, ks & 3, ks & 3);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            umma_mxf8_pair(acc, dev::desc_sw128(sx + 32 * j), dev::desc_sw128(sw + 32 * j), id, sfx, sfw,
                           ks > 0 || j > 0 ? 1u : 0u);
          issued = true;
          dev::tc_commit_pair_mc(&empty[s], 0x3);
          if ((ks & 3) == 3 || ks == p.KS - 1) {
            dev::tc_commit_pair(&sft_empty[b]);
            ++quad;
          }
        }
        if (!ok) break;
        dev::tc_commit_pair_mc(&tmem_full[a], 0x3);
      }
      if (!ok) abort_pair(abort_flag, peer_abort, p.status);
      if (issued) {                                  // the tensor cores are idle before TMEM is freed
        dev::tc_commit_pair(drain);
        dev::mbar_wait(drain, 0, p.limit_ns, nullptr);
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ scale words (both CTAs)
    dev::grid_dependency_wait();
    int quad = 0;
    bool ok = true;
    for (int item = pair; item < items && ok; item += pairs) {
      const Item u = find_item(p, tab, TOK, 8, ntn, item);
      for (int kw = 0; kw < p.KW; ++kw, ++quad) {
        const int b = quad % SF_BUFS;
        const uint32_t *xs = p.sx + static_cast<size_t>(kw) * p.Mp;
        uint32_t xw[4], ww[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = u.row0 + 128 * static_cast<int>(h) + 32 * i + lane;
          xw[i] = row < p.Mp ? xs[row] : 0u;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 32 * i + lane, col = u.nt * TILE_N + r;
          ww[i] = r < TILE_N && col < p.N
                      ? __ldg(weight_atom(p, u.expert, col >> 7, kw) + (col & 31) * 4 + ((col >> 5) & 3))
                      : 0u;
        }
        const bool got = dev::mbar_wait_cluster(&sf_empty[b], ((quad / SF_BUFS) & 1) ^ 1, p.limit_ns, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        uint4 *dst = reinterpret_cast<uint4 *>(smem + SF_OFF + b * SF_BYTES);
        dst[lane] = make_uint4(xw[0], xw[1], xw[2], xw[3]);
        dst[32 + lane] = make_uint4(ww[0], ww[1], ww[2], ww[3]);
        dst[64 + lane] = make_uint4(ww[4], ww[5], ww[6], ww[7]);
        dev::fence_proxy_async();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive_cluster(dev::mapa(dev::smem_u32(&sf_full[b]), 0));
      }
    }
    if (!ok && lane == 0) abort_pair(abort_flag, peer_abort, p.status);
  } else if (warp == 3) {
    // ------------------------------------------------------------ scale words into TMEM (even CTA)
    // from a warp of its own: in the MMA thread's order the copies would stand between the MMAs
    if (h == 0 && elect_one()) {
      int quad = 0;
      bool ok = true;
      for (int item = pair; item < items && ok; item += pairs) {
        for (int kw = 0; kw < p.KW; ++kw, ++quad) {
          const int b = quad % SF_BUFS, t = quad % SF_TMEM;
          if (!dev::mbar_wait_cluster(&sf_full[b], (quad / SF_BUFS) & 1, p.limit_ns, abort_flag) ||
              !dev::mbar_wait(&sft_empty[t], ((quad / SF_TMEM) & 1) ^ 1, p.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          dev::tc_fence_after();
          const uint32_t src = dev::smem_u32(smem + SF_OFF + b * SF_BYTES);
          const uint32_t dst = tmem + SF_COL + 12 * t;
          dev::tmem_cp_32x128b_x4_pair(dst, dev::desc_sf(src));
          dev::tmem_cp_32x128b_x4_pair(dst + 4, dev::desc_sf(src + kScaleAtom));
          dev::tmem_cp_32x128b_x4_pair(dst + 8, dev::desc_sf(src + 2 * kScaleAtom));
          dev::tc_commit_pair(&sft_full[t]);
          dev::tc_commit_pair_mc(&sf_empty[b], 0x3);
        }
      }
      if (!ok) abort_pair(abort_flag, peer_abort, p.status);
      if (quad > 0) {
        dev::tc_commit_pair(drain_cp);
        dev::mbar_wait(drain_cp, 0, p.limit_ns, nullptr);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int e = warp - 4, q = warp & 3, half = e >> 2;   // TMEM lane quarter; columns 0..127 or 128..239
    const uint32_t tmem_empty_even = dev::mapa(dev::smem_u32(tmem_empty), 0);
    const bool wide = ((reinterpret_cast<uintptr_t>(p.Y) | (p.ldy * 2)) & 31) == 0;
    dev::grid_dependency_wait();
    int n = 0;
    for (int item = pair; item < items; item += pairs, ++n) {
      const Item u = find_item(p, tab, TOK, 8, ntn, item);
      const int a = n & 1;
      const bool got = dev::mbar_wait_cluster(&tmem_full[a], (n >> 1) & 1, p.limit_ns, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        if (lane == 0) abort_pair(abort_flag, peer_abort, p.status);
        break;
      }
      dev::tc_fence_after();
      const int row = u.row0 + 128 * static_cast<int>(h) + 32 * q + lane;
      const bool row_ok = row >= u.begin && row < u.end;
      uint16_t *y = p.Y + static_cast<size_t>(row) * p.ldy;
      const uint16_t *bias = p.bias ? p.bias + static_cast<size_t>(u.expert) * p.N : nullptr;
      const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(a * TILE_N);
      if (row - lane < u.end) {                            // some row of this warp's 32 is the expert's
#pragma unroll 1
        for (int c = 128 * half; c < (half ? TILE_N : 128); c += 32) {
          const int col = u.nt * TILE_N + c;
          if (col >= p.N) break;                           // the whole warp
          const bool two = c + 16 < TILE_N;
          uint32_t v0[16], v1[16];
          tmem_ld_32x32b_x16(taddr + c, v0);
          if (two) tmem_ld_32x32b_x16(taddr + c + 16, v1);
          dev::tmem_wait_ld();
          finish16<EPI>(p, bias, v0, col, y, row_ok, wide);
          if (two && col + 16 < p.N) finish16<EPI>(p, bias, v1, col + 16, y, row_ok, wide);
        }
      }
      dev::tc_fence_before();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive_cluster(tmem_empty_even + 8 * a);
    }
  }

  dev::tc_fence_before();
  __syncwarp();
  dev::cluster_sync();                               // no MMA or copy of the pair is still running
  if (warp == 1) {
    dev::tc_fence_after();
    dev::tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

template <int EPI>
int launch(const char *fn, const Params &p, const Maps &maps, int pairs, cudaStream_t stream) {
  int rc = smem_optin_once<fp8_gemm_pair_kernel<EPI>>(SMEM_BYTES, fn);
  if (rc != SVDQ_OK) return rc;
  DependentLaunch dl(dim3(2 * pairs), dim3(THREADS), SMEM_BYTES, stream);
  cudaError_t e = cudaLaunchKernelEx(&dl.cfg, fp8_gemm_pair_kernel<EPI>, p, maps);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string(fn) + " launch: " + cudaGetErrorString(e));
  return SVDQ_OK;
}

}  // namespace

int launch_gemm_pair(const char *fn, const Params &p, int epilogue, int sm_count, cudaStream_t stream) {
  const auto u64 = CU_TENSOR_MAP_DATA_TYPE_UINT64;
  const auto none = CU_TENSOR_MAP_SWIZZLE_NONE;
  Maps maps;
  int rc = encode_tmap_2d(&maps.x, u64, p.x, MAP_ROW / 8, static_cast<uint64_t>(p.KS) * (p.Mp / 8), MAP_ROW, MAP_ROW / 8,
                          X_BYTES / MAP_ROW, none);
  if (rc == SVDQ_OK)
    rc = encode_tmap_2d(&maps.w, u64, p.w, MAP_ROW / 8, static_cast<uint64_t>(p.experts) * p.KS * (p.N / 8), MAP_ROW,
                        MAP_ROW / 8, W_BYTES / MAP_ROW, none);
  if (rc != SVDQ_OK) return rc;
  const long long units = (p.M / TOK + (p.offsets ? 2ll * p.experts : 1ll)) * ((p.N + TILE_N - 1) / TILE_N);
  const int pairs = static_cast<int>(units < sm_count / 2 ? units : sm_count / 2);
  return epilogue == SVDQ_EPILOGUE_GELU_ERF    ? launch<SVDQ_EPILOGUE_GELU_ERF>(fn, p, maps, pairs, stream)
         : epilogue == SVDQ_EPILOGUE_GELU_TANH ? launch<SVDQ_EPILOGUE_GELU_TANH>(fn, p, maps, pairs, stream)
                                               : launch<SVDQ_EPILOGUE_NONE>(fn, p, maps, pairs, stream);
}

}  // namespace fp8
}  // namespace svdq
