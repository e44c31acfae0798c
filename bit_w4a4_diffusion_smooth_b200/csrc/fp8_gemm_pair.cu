// Block-scaled FP8 GEMM for many rows: 256 x 256 output tiles on SM pairs.
//
// Clusters of two CTAs, one per SM of a TPC; every MMA is a cta_group::2 MMA
// of 256 x 256 x 32: CTA h holds rows 128h..128h+127 of the token tile and
// weight rows (output columns) 128h..128h+127, and its TMEM receives its own
// 128 rows of the accumulator, so each SM reads 256 operand rows per k-stage
// for 256 x 128 outputs.  (One CTA alone would read 256 for 128 x 128, and the
// operand traffic from L2 bounds it.)
//
// Roles (one CTA per SM, persistent over units of work, 12 warps):
//   warp 0      producer in both CTAs: per k-stage its 16 KB halves of the two
//               operands, completing on the even CTA's `full` barrier
//   warp 1      owns TMEM (pair allocation); in the even CTA one thread issues
//               the MMAs and commits each stage to both CTAs
//   warp 2      scale words of the next four stages, in both CTAs: the words
//               of its own 128 token rows and of all 256 weight rows (which
//               both TMEMs need)
//   warp 3      even CTA: copies them into both TMEMs (tcgen05.cp)
//   warps 4-11  epilogue in both CTAs: drain the accumulator into registers,
//               hand TMEM back, then bias, GELU, bf16, and 32 x 32 tiles
//               through shared memory, written by TMA where the tile lies
//               inside the expert's rows and row by row at its ragged ends
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
constexpr int STAGES = 6;
constexpr int STAGE = 2 * kTileBytes;          // this CTA's 128 token rows, then its 128 weight rows
constexpr int SF_BUFS = 4;
constexpr int SF_BYTES = 3 * kScaleAtom;       // own token atom, the two weight atoms
constexpr int EPI_WARPS = 8;
constexpr int EPI_TILE = 32 * 64;              // 32 rows x 32 bf16, 64-byte swizzle
constexpr int THREADS = (4 + EPI_WARPS) * 32;
constexpr int SF_OFF = STAGES * STAGE;
constexpr int EPI_OFF = SF_OFF + SF_BUFS * SF_BYTES;
constexpr int TAB_OFF = EPI_OFF + EPI_WARPS * EPI_TILE;
constexpr int BAR_OFF = (TAB_OFF + static_cast<int>(sizeof(ExpertTable)) + 15) & ~15;
constexpr int SMEM_BYTES = 1024 + BAR_OFF + 256;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SF_COL = 256;               // buffer b: token scales at +12b, weight scales at +12b + 4
constexpr int WROW = 2048, XROW = 1024;        // row bytes of the operands' tensor maps
static_assert(SMEM_BYTES <= 232448, "fits in shared memory");
static_assert(EPI_OFF % 512 == 0, "staging tiles start on swizzle atoms");

struct Maps {
  CUtensorMap x, w, y;
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

__device__ __forceinline__ void abort_pair(volatile int *abort_flag, uint32_t peer_abort, unsigned int *status) {
  *abort_flag = 1;
  dev::st_cluster_u32(peer_abort, 1u);
  dev::report(status, SVDQ_ERR_TIMEOUT);
}

template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    fp8_gemm_pair_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + BAR_OFF);   // even CTA: both CTAs' bytes
  uint64_t *empty = full + STAGES;                                  // both CTAs: stage free again
  uint64_t *sf_full = empty + STAGES;                               // even CTA: both CTAs' scale words
  uint64_t *sf_empty = sf_full + SF_BUFS;                           // both CTAs
  uint64_t *sf_tmem = sf_empty + SF_BUFS;                           // even CTA: scale words in both TMEMs
  uint64_t *tmem_full = sf_tmem + SF_BUFS;                         // both CTAs: accumulator ready
  uint64_t *tmem_empty = tmem_full + 1;                             // even CTA: both CTAs drained it
  uint64_t *drain = tmem_empty + 1;
  uint64_t *drain_cp = drain + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain_cp + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  ExpertTable *tab = reinterpret_cast<ExpertTable *>(smem + TAB_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t h = dev::cluster_ctarank();         // 0: even CTA (issues the MMAs), 1: odd
  const int pair = static_cast<int>(dev::cluster_id_x());
  const int pairs = static_cast<int>(dev::num_clusters_x());
  const int ntn2 = (p.ntn + 1) / 2;                  // 256-column tiles
  const uint32_t peer_abort = dev::mapa(dev::smem_u32(const_cast<int *>(abort_flag)), h ^ 1u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      dev::mbar_init(&full[s], 1);
      dev::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < SF_BUFS; ++b) {
      dev::mbar_init(&sf_full[b], 2);
      dev::mbar_init(&sf_empty[b], 1);
      dev::mbar_init(&sf_tmem[b], 1);
    }
    dev::mbar_init(tmem_full, 1);
    dev::mbar_init(tmem_empty, 2 * EPI_WARPS);
    dev::mbar_init(drain, 1);
    dev::mbar_init(drain_cp, 1);
    *abort_flag = 0;
    dev::fence_mbar_init();
  }
  if (warp == 1) {
    dev::tmem_alloc_pair(tmem_slot, TMEM_COLS);
    dev::tmem_relinquish_pair();
  }
  dev::grid_dependency_wait();
  dev::grid_launch_dependents();
  if (warp == 2) fill_expert_table(p, TOK, tab);
  dev::tc_fence_before();
  __syncwarp();
  dev::cluster_sync();                               // both CTAs' barriers exist before anyone arrives remotely
  dev::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int items = tab->tiles[p.experts] * ntn2;

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (elect_one()) {
      dev::prefetch_tmap(&maps.x);
      dev::prefetch_tmap(&maps.w);
      int it = 0;
      bool ok = true;
      for (int item = pair; item < items && ok; item += pairs) {
        const Item u = find_item(p, tab, TOK, ntn2, item);
        // the last 128-column tile of an odd count stands in for the one past it (its columns are not stored)
        const int nt = min(2 * u.nt + static_cast<int>(h), p.ntn - 1);
        const int wrow = (u.expert * p.ntn + nt) * p.KS * (kTileBytes / WROW);
        const int xrow = u.row0 / 8 + 16 * static_cast<int>(h);
        for (int ks = 0; ks < p.KS; ++ks, ++it) {
          const int s = it % STAGES;
          if (!dev::mbar_wait_cluster(&empty[s], ((it / STAGES) & 1) ^ 1, p.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t bar = dev::mapa(dev::smem_u32(&full[s]), 0);
          uint8_t *dst = smem + s * STAGE;
          if (h == 0) dev::mbar_arrive_expect_tx(&full[s], 2u * STAGE);
          // rows past the end of a stage's rows hold the next stage's, past the buffer zeros: neither reaches
          // an output
          dev::tma_load_2d_pair(dst, &maps.x, bar, 0, xrow + ks * (p.Mp / 8));
          dev::tma_load_2d_pair(dst + kTileBytes, &maps.w, bar, 0, wrow + ks * (kTileBytes / WROW));
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
      constexpr uint32_t idesc = idesc_mxf8(256, 256);
      int it = 0, quad = 0, n = 0;
      bool ok = true, issued = false;
      for (int item = pair; item < items && ok; item += pairs, ++n) {
        if (!dev::mbar_wait_cluster(tmem_empty, (n & 1) ^ 1, p.limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        dev::tc_fence_after();
        uint32_t sfx = 0, sfw = 0;
        for (int ks = 0; ks < p.KS; ++ks, ++it) {
          const int s = it % STAGES, b = quad % SF_BUFS;
          if ((ks & 3) == 0) {
            if (!dev::mbar_wait(&sf_tmem[b], (quad / SF_BUFS) & 1, p.limit_ns, abort_flag)) {
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
          const uint32_t sx = dev::smem_u32(smem + s * STAGE), sw = sx + kTileBytes;
          const uint32_t id = with_scale_byte(idesc, static_cast<uint32_t>(ks & 3));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            umma_mxf8_pair(tmem, dev::desc_sw128(sx + 32 * j), dev::desc_sw128(sw + 32 * j), id, sfx, sfw,
                           ks > 0 || j > 0 ? 1u : 0u);
          issued = true;
          dev::tc_commit_pair_mc(&empty[s], 0x3);
          if ((ks & 3) == 3 || ks == p.KS - 1) {
            dev::tc_commit_pair_mc(&sf_empty[b], 0x3);
            ++quad;
          }
        }
        if (!ok) break;
        dev::tc_commit_pair_mc(tmem_full, 0x3);
      }
      if (!ok) abort_pair(abort_flag, peer_abort, p.status);
      if (issued) {                                  // the tensor cores are idle before TMEM is freed
        dev::tc_commit_pair(drain);
        dev::mbar_wait(drain, 0, p.limit_ns, nullptr);
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ scale words (both CTAs)
    int quad = 0;
    bool ok = true;
    for (int item = pair; item < items && ok; item += pairs) {
      const Item u = find_item(p, tab, TOK, ntn2, item);
      const size_t tile = static_cast<size_t>(u.expert) * p.ntn;
      const uint8_t *w0 = p.sw + (tile + 2 * u.nt) * p.KW * kScaleAtom;
      const uint8_t *w1 = p.sw + (tile + min(2 * u.nt + 1, p.ntn - 1)) * p.KW * kScaleAtom;
      for (int kw = 0; kw < p.KW; ++kw, ++quad) {
        const int b = quad % SF_BUFS;
        const uint4 a0 = __ldg(reinterpret_cast<const uint4 *>(w0 + static_cast<size_t>(kw) * kScaleAtom) + lane);
        const uint4 a1 = __ldg(reinterpret_cast<const uint4 *>(w1 + static_cast<size_t>(kw) * kScaleAtom) + lane);
        const uint32_t *xs = p.sx + static_cast<size_t>(kw) * p.Mp;
        uint32_t xw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = u.row0 + 128 * static_cast<int>(h) + 32 * i + lane;
          xw[i] = row < p.Mp ? xs[row] : 0u;
        }
        const bool got = dev::mbar_wait_cluster(&sf_empty[b], ((quad / SF_BUFS) & 1) ^ 1, p.limit_ns, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        uint4 *dst = reinterpret_cast<uint4 *>(smem + SF_OFF + b * SF_BYTES);
        dst[lane] = make_uint4(xw[0], xw[1], xw[2], xw[3]);
        dst[32 + lane] = a0;
        dst[64 + lane] = a1;
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
          const int b = quad % SF_BUFS;
          if (!dev::mbar_wait_cluster(&sf_full[b], (quad / SF_BUFS) & 1, p.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          dev::tc_fence_after();
          const uint32_t src = dev::smem_u32(smem + SF_OFF + b * SF_BYTES);
          const uint32_t dst = tmem + SF_COL + 12 * b;
          dev::tmem_cp_32x128b_x4_pair(dst, dev::desc_sf(src));
          dev::tmem_cp_32x128b_x4_pair(dst + 4, dev::desc_sf(src + kScaleAtom));
          dev::tmem_cp_32x128b_x4_pair(dst + 8, dev::desc_sf(src + 2 * kScaleAtom));
          dev::tc_commit_pair(&sf_tmem[b]);
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
    const int e = warp - 4, q = warp & 3, half = e >> 2;   // TMEM lane quarter; which 128 of the 256 columns
    uint8_t *stage = smem + EPI_OFF + e * EPI_TILE;
    const uint32_t tmem_empty_even = dev::mapa(dev::smem_u32(tmem_empty), 0);
    int n = 0;
    for (int item = pair; item < items; item += pairs, ++n) {
      const Item u = find_item(p, tab, TOK, ntn2, item);
      const bool got = dev::mbar_wait_cluster(tmem_full, n & 1, p.limit_ns, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        if (lane == 0) abort_pair(abort_flag, peer_abort, p.status);
        break;
      }
      dev::tc_fence_after();
      uint32_t v[4][32];
      const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(128 * half);
#pragma unroll
      for (int c = 0; c < 4; ++c) dev::tmem_ld_32x32b_x32(taddr + 32 * c, v[c]);
      dev::tmem_wait_ld();
      dev::tc_fence_before();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive_cluster(tmem_empty_even);   // the next tile's MMAs may start

      const int row0 = u.row0 + 128 * static_cast<int>(h) + 32 * q;
      const int col0 = 256 * u.nt + 128 * half;
      if (row0 >= u.end) continue;                         // no row of this expert (the whole warp)
      const bool inside = row0 >= u.begin && row0 + 32 <= u.end;
      const uint16_t *bias = p.bias ? p.bias + static_cast<size_t>(u.expert) * p.N : nullptr;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = col0 + 32 * c;
        if (col >= p.N) break;                             // the whole warp
        uint32_t out[16];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t bw[4] = {0, 0, 0, 0};
          if (bias && col + 8 * g < p.N) {                 // N % 8 == 0: all eight or none
#pragma unroll
            for (int j = 0; j < 4; ++j)
              bw[j] = static_cast<uint32_t>(__ldg(bias + col + 8 * g + 2 * j)) |
                      (static_cast<uint32_t>(__ldg(bias + col + 8 * g + 2 * j + 1)) << 16);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 8 * g + 2 * j;
            const float2 y = make_float2(__uint_as_float(v[c][i]) + __uint_as_float(bw[j] << 16),
                                         __uint_as_float(v[c][i + 1]) + __uint_as_float(bw[j] & 0xFFFF0000u));
            float2 a = activate2<EPI>(y);
            if constexpr (EPI != SVDQ_EPILOGUE_NONE) {
              a.x = col + i >= p.gelu_col_begin ? a.x : y.x;
              a.y = col + i + 1 >= p.gelu_col_begin ? a.y : y.y;
            }
            const __nv_bfloat162 hv = __floats2bfloat162_rn(a.x, a.y);
            out[4 * g + j] = *reinterpret_cast<const uint32_t *>(&hv);
          }
        }
        if (lane == 0) dev::bulk_wait_group_read<0>();     // the staging tile is free again
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 4; ++g)                        // row `lane`, 16-byte chunk g, 64-byte swizzle
          *reinterpret_cast<uint4 *>(stage + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(out[4 * g], out[4 * g + 1], out[4 * g + 2], out[4 * g + 3]);
        if (inside) {
          dev::fence_proxy_async();
          __syncwarp();
          if (lane == 0) {                                 // the TMA clips columns past N
            dev::tma_store_2d(&maps.y, stage, col, row0);
            dev::bulk_commit_group();
          }
        } else {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = 8 * i + (lane >> 2), seg = lane & 3, row = row0 + t;
            if (row >= u.begin && row < u.end && col + 8 * seg < p.N)
              *reinterpret_cast<uint4 *>(p.Y + static_cast<size_t>(row) * p.ldy + col + 8 * seg) =
                  *reinterpret_cast<const uint4 *>(stage + t * 64 + ((seg ^ ((t >> 1) & 3)) << 4));
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) dev::bulk_wait_group<0>();
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
  int rc = encode_tmap_2d(&maps.x, u64, p.x, XROW / 8, static_cast<uint64_t>(p.KS) * (p.Mp / 8), XROW, XROW / 8, 16, none);
  if (rc == SVDQ_OK)
    rc = encode_tmap_2d(&maps.w, u64, p.w, WROW / 8,
                        static_cast<uint64_t>(p.experts) * p.ntn * p.KS * (kTileBytes / WROW), WROW, WROW / 8,
                        kTileBytes / WROW, none);
  if (rc == SVDQ_OK)
    rc = encode_tmap_2d(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.Y, static_cast<uint64_t>(p.N),
                        static_cast<uint64_t>(p.M), p.ldy * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (rc != SVDQ_OK) return rc;
  const long long units = (p.M / TOK + (p.offsets ? 2ll * p.experts : 1ll)) * ((p.ntn + 1) / 2);
  const int pairs = static_cast<int>(units < sm_count / 2 ? units : sm_count / 2);
  return epilogue == SVDQ_EPILOGUE_GELU_ERF    ? launch<SVDQ_EPILOGUE_GELU_ERF>(fn, p, maps, pairs, stream)
         : epilogue == SVDQ_EPILOGUE_GELU_TANH ? launch<SVDQ_EPILOGUE_GELU_TANH>(fn, p, maps, pairs, stream)
                                               : launch<SVDQ_EPILOGUE_NONE>(fn, p, maps, pairs, stream);
}

}  // namespace fp8
}  // namespace svdq
