// Block-scaled FP8 GEMM for many rows: 256 x 240 output tiles on SM pairs.
//
// Clusters of two CTAs, one per SM of a TPC; every MMA is a cta_group::2 MMA
// of 256 x 240 x 32: CTA h holds rows 128h..128h+127 of the token tile and
// weight rows (output columns) 120h..120h+119, and its TMEM receives its own
// 128 rows of the accumulator, so each SM reads 248 operand rows per k-stage
// for 256 x 120 outputs.  (One CTA alone would read 256 for 128 x 128.)  240
// columns instead of 256 leave TMEM room for two accumulators and the block
// scales, so that a tile's epilogue runs under the next tile's MMAs.
//
// What bounds it: shared memory.  A stage is written once and read once by the
// MMAs, 2 x 248 rows x 128 bytes in the 480 cycles of its MMAs: 132 bytes a
// cycle of the 128 an SM has, 140 with the epilogue's.  Under load the power
// cap lowers the clock besides.  (That and whole rounds explain 82 of the 106 us
// that 4608 x 2560 -> 10240 takes behind its quantizer; the rest is lost per
// tile, in waits that have not been recorded.)
//
// Roles (one CTA per SM, persistent over units of work, 20 warps):
//   warp 0      producer in both CTAs: per k-stage its halves of the two
//               operands, completing on the even CTA's `full` barrier
//   warp 1      owns TMEM (pair allocation); in the even CTA one thread issues
//               the MMAs and commits each stage to both CTAs.  It has 480
//               cycles a stage: it asks for the next stage's barrier before it
//               issues this one's MMAs, and keeps its place in the ring by
//               increments
//   warp 2      scale words of the next four stages, in both CTAs: the words
//               of its own 128 token rows and of all 240 weight rows (which
//               both TMEMs need).  Their loads run two sets ahead
//   warp 3      even CTA: copies them into both TMEMs (tcgen05.cp); from the
//               MMA thread they would stand between its MMAs
//   warps 4-19  epilogue in both CTAs: 16 columns at a time from TMEM, bias,
//               GELU, bf16, and 32 rows x 32 columns through shared memory to
//               global memory, a row's 64 bytes by 4 lanes.  Sixteen warps,
//               since GELU's chains leave a scheduler idle under two of them
//               (10,000 cycles a tile of 9,000 of MMAs at K = 2560), and a
//               rolled loop: unrolled over the tile the code outgrew the
//               instruction cache
// What crosses the pair is read by the asynchronous proxy (operands, scale
// words) or lies in TMEM, so its barriers need no cluster-scope fence: with
// one, an arrival waited for every load the warp had in flight, and the scale
// words alone took 2,400 cycles a set against 1,800 of MMAs.
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
constexpr int SF_BUFS = 2;                     // scale words of 2 x 4 k-stages in shared memory
constexpr int SF_TMEM = 2;                     // ... and in TMEM
constexpr int SF_BYTES = 3 * kScaleAtom;       // own token atom, two weight atoms
constexpr int SF_COLS = 12;                    // token scales 4 columns, weight scales 8
constexpr int EPI_WARPS = 16;
constexpr int EPI_TILE = 32 * 64;              // a warp's 32 rows x 32 bf16
constexpr int THREADS = (4 + EPI_WARPS) * 32;
constexpr int SF_OFF = STAGES * STAGE;
constexpr int EPI_OFF = SF_OFF + SF_BUFS * SF_BYTES;
constexpr int TAB_OFF = EPI_OFF + EPI_WARPS * EPI_TILE;
constexpr int BAR_OFF = (TAB_OFF + static_cast<int>(sizeof(ExpertTable)) + 15) & ~15;
constexpr int SMEM_BYTES = 1024 + BAR_OFF + 256;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SF_COL = 2 * TILE_N;
constexpr int MAP_ROW = 1024;                  // the operands as rows of 8 x 128 bytes
static_assert(STAGE % 1024 == 0 && X_BYTES % 1024 == 0, "operand tiles start on 1024-byte boundaries");
static_assert(SMEM_BYTES <= 232448, "fits in shared memory");
static_assert(SF_COL + SF_COLS * SF_TMEM <= TMEM_COLS, "accumulators and scales fit in TMEM");

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

// Bias (16 bf16, if there is one), activation and rounding of 16 columns, the GELU from column `act` of the 16 on.
template <int EPI>
__device__ __forceinline__ void finish16(const uint32_t (&v)[16], bool biased, const uint4 (&bb)[2], int act,
                                         uint32_t (&out)[8]) {
  float2 t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
  if (biased) {
    const uint32_t bw[8] = {bb[0].x, bb[0].y, bb[0].z, bb[0].w, bb[1].x, bb[1].y, bb[1].z, bb[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      t[j] = add2_rn(t[j], make_float2(__uint_as_float(bw[j] << 16), __uint_as_float(bw[j] & 0xFFFF0000u)));
  }
  if constexpr (EPI != SVDQ_EPILOGUE_NONE) {
    if (act <= 0) {                                // the usual case, the same for all lanes
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = activate2<EPI>(t[j]);
    } else if (act < 16) {
#pragma unroll 1
      for (int j = 0; j < 8; ++j) {
        float2 x = t[0];                           // through the first place, so that the loop stays rolled
        const float2 g = activate2<EPI>(x);
        x = make_float2(2 * j >= act ? g.x : x.x, 2 * j + 1 >= act ? g.y : x.y);
#pragma unroll
        for (int i = 0; i < 7; ++i) t[i] = t[i + 1];
        t[7] = x;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(t[j].x, t[j].y);
    out[j] = *reinterpret_cast<const uint32_t *>(&h);
  }
}

// Whether the phase of `bar` with parity `parity` has completed, without waiting.
__device__ __forceinline__ uint32_t mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(dev::smem_u32(bar)), "r"(parity)
      : "memory");
  return done;
}

template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    fp8_gemm_pair_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + BAR_OFF);  // even CTA: both CTAs' bytes
  uint64_t *empty = full + STAGES;                                  // both CTAs: stage free again
  uint64_t *sf_full = empty + STAGES;                               // even CTA: both CTAs' scale words
  uint64_t *sf_empty = sf_full + SF_BUFS;                           // both CTAs: their copy into TMEM is done
  uint64_t *sft_full = sf_empty + SF_BUFS;                          // even CTA: scale words in both TMEMs
  uint64_t *sft_empty = sft_full + SF_TMEM;                         // even CTA: their MMAs are done
  uint64_t *tmem_full = sft_empty + SF_TMEM;                        // both CTAs: accumulator ready
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
  // The kernel in front is the quantizer, which lets this one start only after its own wait: everything older
  // (offsets and weights among it) has completed by now, and only X's codes and scales have to be waited for,
  // where they are first read.
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
      // rows past the end of a stage's rows hold the next stage's, past the buffer zeros: neither reaches an output
      const auto load_weights = [&](const Item &u, int ks, int s) {
        if (h == 0) dev::mbar_arrive_expect_tx(&full[s], 2u * STAGE);
        dev::tma_load_2d_pair(smem + s * STAGE + X_BYTES, &maps.w, dev::mapa(dev::smem_u32(&full[s]), 0), 0,
                              weight_row(p, u, ks, h));
      };
      int ahead = 0;                                 // stages whose weights are under way before X is there
      if (pair < items) {
        const Item u = find_item(p, tab, TOK, 8, ntn, pair);
        for (; ahead < min(STAGES, p.KS); ++ahead) load_weights(u, ahead, ahead);
      }
      dev::grid_dependency_wait();
      int it = 0;
      bool ok = true;
      for (int item = pair; item < items && ok; item += pairs) {
        const Item u = find_item(p, tab, TOK, 8, ntn, item);
        const int xrow = u.row0 / 8 + 16 * static_cast<int>(h);
        for (int ks = 0; ks < p.KS; ++ks, ++it) {
          const int s = it % STAGES;
          if (it >= ahead) {
            if (!dev::mbar_wait(&empty[s], ((it / STAGES) & 1) ^ 1, p.limit_ns, abort_flag)) {
              ok = false;
              break;
            }
            load_weights(u, ks, s);
          }
          dev::tma_load_2d_pair(smem + s * STAGE, &maps.x, dev::mapa(dev::smem_u32(&full[s]), 0), 0,
                                xrow + ks * (p.Mp / 8));
        }
      }
      if (!ok) abort_pair(abort_flag, peer_abort, p.status);
      // before the pair may leave, every stage the even CTA armed completes (the odd CTA's copies with it)
      if (h == 0)
        for (int j = max(0, it - STAGES); j < it; ++j)
          dev::mbar_wait(&full[j % STAGES], (j / STAGES) & 1, p.limit_ns, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ scales into TMEM, MMAs (even CTA)
    if (h == 0 && elect_one()) {
      constexpr uint32_t idesc = idesc_mxf8(TOK, TILE_N);
      const uint64_t desc0 = dev::desc_sw128(dev::smem_u32(smem));
      uint64_t dx = desc0;                           // the ring place's operands, its number and its phase
      int s = 0;
      uint32_t phase = 0, ready = 0;
      int b = 0, n = 0;
      uint32_t b_phase = 0;
      bool ok = true, issued = false;
      for (int item = pair; item < items && ok; item += pairs, ++n) {
        const int a = n & 1;
        if (!dev::mbar_wait(&tmem_empty[a], ((n >> 1) & 1) ^ 1, p.limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        dev::tc_fence_after();
        const uint32_t acc = tmem + a * TILE_N;
        uint32_t accumulate = 0;
        for (int ks0 = 0; ks0 < p.KS && ok; ks0 += 4) {    // four stages under one set of scale words
          if (!dev::mbar_wait(&sft_full[b], b_phase, p.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t sf = tmem + SF_COL + SF_COLS * b;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (ks0 + i >= p.KS) break;
            if (!ready && !dev::mbar_wait(&full[s], phase, p.limit_ns, abort_flag)) {
              ok = false;
              break;
            }
            dev::tc_fence_after();
            const bool wrap = s == STAGES - 1;
            const int next = wrap ? 0 : s + 1;
            phase ^= wrap ? 1u : 0u;
            ready = mbar_test(&full[next], phase);
            const uint32_t id = with_scale_bytes(idesc, i, i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              umma_mxf8_pair(acc, dx + desc_step(32 * j), dx + desc_step(X_BYTES + 32 * j), id, sf, sf + 4, accumulate);
              accumulate = 1;
            }
            issued = true;
            dev::tc_commit_pair_mc(&empty[s], 0x3);
            dx = wrap ? desc0 : dx + desc_step(STAGE);
            s = next;
          }
          if (!ok) break;
          dev::tc_commit_pair(&sft_empty[b]);
          b_phase ^= b == SF_TMEM - 1 ? 1u : 0u;
          b = b == SF_TMEM - 1 ? 0 : b + 1;
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
    uint32_t xw[SF_BUFS][4], ww[SF_BUFS][8];
    int item[SF_BUFS], kw[SF_BUFS];
    Item u[SF_BUFS];
    // `sets` sets on in the CTA's sequence, and the words of the set there
    const auto advance = [&](int d, int sets) {
      const int was = item[d];
      for (kw[d] += sets; kw[d] >= p.KW; kw[d] -= p.KW) item[d] += pairs;
      if (item[d] != was && item[d] < items) u[d] = find_item(p, tab, TOK, 8, ntn, item[d]);
    };
    const auto load = [&](int d) {
      if (item[d] >= items) return;
      const uint32_t *xs = p.sx + static_cast<size_t>(kw[d]) * p.Mp;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = u[d].row0 + 128 * static_cast<int>(h) + 32 * i + lane;
        xw[d][i] = row < p.Mp ? xs[row] : 0u;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int col = u[d].nt * TILE_N + 32 * i + lane;
        ww[d][i] = 32 * i + lane < TILE_N && col < p.N ? __ldg(weight_atom(p, u[d].expert, col >> 7, kw[d]) + (col & 31) * 4 + ((col >> 5) & 3)) : 0u;
      }
    };
    if (pair < items) {
      const Item first = find_item(p, tab, TOK, 8, ntn, pair);
#pragma unroll
      for (int d = 0; d < SF_BUFS; ++d) {
        item[d] = pair;
        kw[d] = 0;
        u[d] = first;
        advance(d, d);
        load(d);
      }
      bool ok = true;
      uint32_t phase = 1;
      while (ok && item[0] < items) {
#pragma unroll
        for (int d = 0; d < SF_BUFS; ++d) {
          if (!ok || item[d] >= items) break;
          const bool got = dev::mbar_wait(&sf_empty[d], phase, p.limit_ns, abort_flag);
          if (!__all_sync(0xFFFFFFFFu, got)) {
            ok = false;
            break;
          }
          uint4 *dst = reinterpret_cast<uint4 *>(smem + SF_OFF + d * SF_BYTES);
          dst[lane] = make_uint4(xw[d][0], xw[d][1], xw[d][2], xw[d][3]);
          dst[32 + lane] = make_uint4(ww[d][0], ww[d][1], ww[d][2], ww[d][3]);
          dst[64 + lane] = make_uint4(ww[d][4], ww[d][5], ww[d][6], ww[d][7]);
          dev::fence_proxy_async();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive_remote(dev::mapa(dev::smem_u32(&sf_full[d]), 0));
          advance(d, SF_BUFS);
          load(d);
        }
        phase ^= 1;
      }
      if (!ok && lane == 0) abort_pair(abort_flag, peer_abort, p.status);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ scale words into TMEM (even CTA)
    // from a warp of its own: in the MMA thread's order the copies would stand between the MMAs
    if (h == 0 && elect_one()) {
      int quad = 0;
      bool ok = true;
      for (int item = pair; item < items && ok; item += pairs) {
        for (int kw = 0; kw < p.KW; ++kw, ++quad) {
          const int b = quad % SF_BUFS, t = quad % SF_TMEM;
          if (!dev::mbar_wait(&sf_full[b], (quad / SF_BUFS) & 1, p.limit_ns, abort_flag) ||
              !dev::mbar_wait(&sft_empty[t], ((quad / SF_TMEM) & 1) ^ 1, p.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          dev::tc_fence_after();
          const uint32_t src = dev::smem_u32(smem + SF_OFF + b * SF_BYTES);
          const uint32_t dst = tmem + SF_COL + SF_COLS * t;
#pragma unroll
          for (int i = 0; i < 3; ++i) dev::tmem_cp_32x128b_x4_pair(dst + 4 * i, dev::desc_sf(src + i * kScaleAtom));
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
    const int e = warp - 4, q = warp & 3, part = e >> 2;   // TMEM lane quarter; 64 columns, or the last 48
    const int begin = 64 * part, cols = min(64, TILE_N - begin);
    uint8_t *stage = smem + EPI_OFF + e * EPI_TILE;
    const uint32_t tmem_empty_even = dev::mapa(dev::smem_u32(tmem_empty), 0);
    dev::grid_dependency_wait();
    int n = 0;
    for (int item = pair; item < items; item += pairs, ++n) {
      const Item u = find_item(p, tab, TOK, 8, ntn, item);
      const int row0 = u.row0 + 128 * static_cast<int>(h) + 32 * q, a = n & 1;
      const int col0 = u.nt * TILE_N + begin;
      const uint16_t *bias = p.bias ? p.bias + static_cast<size_t>(u.expert) * p.N + col0 : nullptr;
      // the warp's columns that exist, none if none of its 32 rows is the expert's
      const int live = row0 >= u.end ? 0 : min(cols, p.N - col0);
      const int t0 = lane >> 2, seg = lane & 3;
      uint16_t *yrow = p.Y + static_cast<size_t>(row0 + t0) * p.ldy + col0 + 8 * seg;
      const bool got = dev::mbar_wait(&tmem_full[a], (n >> 1) & 1, p.limit_ns, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        if (lane == 0) abort_pair(abort_flag, peer_abort, p.status);
        break;
      }
      dev::tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(a * TILE_N + begin);
#pragma unroll 1
      for (int c = 0; c < live; c += 16) {
        uint32_t v[16], out[8];
        tmem_ld_32x32b_x16(taddr + c, v);
        uint4 bb[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (bias) {
          bb[0] = __ldg(reinterpret_cast<const uint4 *>(bias + c));
          if (c + 8 < live) bb[1] = __ldg(reinterpret_cast<const uint4 *>(bias + c + 8));   // N % 8 == 0
        }
        dev::tmem_wait_ld();
        finish16<EPI>(v, bias != nullptr, bb, p.gelu_col_begin - col0 - c, out);
        // row `lane`, 16-byte chunk k of the 32 columns at chunk k ^ (row / 2 % 4): few bank conflicts either way
        const int k = (c & 16) >> 3, x = (lane >> 1) & 3;
        *reinterpret_cast<uint4 *>(stage + lane * 64 + ((k ^ x) << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
        *reinterpret_cast<uint4 *>(stage + lane * 64 + (((k + 1) ^ x) << 4)) = make_uint4(out[4], out[5], out[6], out[7]);
        if ((c & 16) != 0 || c + 16 >= live) {             // 32 columns, or the last: 8 rows at a time
          const int c32 = c & ~31;
          const bool there = c32 + 8 * seg < live;
          __syncwarp();
          uint16_t *y = yrow + c32;
#pragma unroll
          for (int i = 0; i < 4; ++i, y += 8 * p.ldy) {
            const int t = 8 * i + t0, row = row0 + t;
            if (there && row >= u.begin && row < u.end)
              *reinterpret_cast<uint4 *>(y) = *reinterpret_cast<const uint4 *>(stage + t * 64 + ((seg ^ ((t >> 1) & 3)) << 4));
          }
          __syncwarp();
        }
      }
      dev::tc_fence_before();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive_remote(tmem_empty_even + 8 * a);
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
  // token tiles: one per 256 rows, and two that each expert may leave unfilled
  const long long tiles = p.offsets ? p.M / TOK + 2ll * p.experts : (p.M + TOK - 1) / TOK;
  const long long units = tiles * ((p.N + TILE_N - 1) / TILE_N);
  const int pairs = static_cast<int>(units < sm_count / 2 ? units : sm_count / 2);
  return epilogue == SVDQ_EPILOGUE_GELU_ERF    ? launch<SVDQ_EPILOGUE_GELU_ERF>(fn, p, maps, pairs, stream)
         : epilogue == SVDQ_EPILOGUE_GELU_TANH ? launch<SVDQ_EPILOGUE_GELU_TANH>(fn, p, maps, pairs, stream)
                                               : launch<SVDQ_EPILOGUE_NONE>(fn, p, maps, pairs, stream);
}

}  // namespace fp8
}  // namespace svdq
