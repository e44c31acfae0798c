// Block-scaled FP8 GEMM for few rows: 128 output columns by 16..128 rows of X.
//
// The weight is on the M side of the MMA (lanes of tensor memory), the rows of
// X on the N side (columns), so a call of a few rows multiplies few rows and is
// bound by one pass over the weight.
//
// Up to 16 rows a tile (FUSED) each CTA quantizes the rows it needs itself,
// stage by stage: X is small and sits in L2, and a quantizer kernel in front
// would cost a launch and its latency (2 rows, 2560 -> 15360: 8.9 us, and 10.9
// with the quantizer in front).  With more rows the CTAs' repeated
// quantizing takes longer than the weights (77 rows, 4096 -> 2560: 22 us
// against 14), and the quantizer runs once in front.
//
// Roles (one CTA per SM, persistent over units of work):
//   warp 0     producer: per stage of two blocks of 128 along K, 128 weight
//              rows of each, their scale atom and (quantized before) the rows
//              of X, by bulk copies: all are stored as their shared-memory
//              images.  The atom covers four blocks and comes with every two
//              (1.5% more from L2)
//   warp 1     owns TMEM; one thread copies scale words into TMEM (tcgen05.cp)
//              and issues the MMAs
//   warp 2     quantized before: brings the activations' scale words of the
//              next four blocks into shared memory in the copy's layout
//   warps 4-7  epilogue: drain the accumulator (two of them in TMEM, so the
//              next unit's MMAs run meanwhile), bias, GELU, bf16, and turn
//              the tile through shared memory into 16-byte row segments
//   warps 8-15 FUSED: quantize X, the warps taking the stages in turn; each
//              loads its next stage before it waits for this one's place, so
//              that the loads' latency (longer than a stage's 0.4 us of
//              weights) overlaps
// Few units of work leave SMs idle; then clusters of 2, 4 or 8 CTAs split K,
// and add their accumulators in a fixed order through distributed shared
// memory (no workspace, no atomics, the same bits every time).
// Two blocks a stage halve what the MMA thread spends between MMAs (a wait, a
// commit, the loop: 350 cycles), which had set the pace: a weight stream of
// 16 KB per 540 cycles and SM.
// Every wait is bounded; one that runs out records SVDQ_ERR_TIMEOUT, raises
// the abort flag, and the CTA drains its copies and MMAs, frees TMEM and ends.
#include <cuda_runtime.h>

#include <atomic>
#include <string>

#include "fp8_gemm.cuh"
#include "fp8_quant.cuh"

namespace svdq {
namespace fp8 {
namespace {

constexpr int TILE_N = 128;                    // output columns per unit
constexpr int W_BLOCK = TILE_N * kBlock;
constexpr int W_BYTES = 2 * W_BLOCK;           // a stage: two blocks of 128 along K
constexpr int EPI_WARPS = 4;
constexpr int SF_BUFS = 4;                     // not FUSED: the activations' scale words of 4 x 4 blocks
constexpr int EPI_STAGE = 32 * 64;             // a warp's 32 rows x 32 columns of bf16

template <int TOK>
struct Shape {
  static constexpr bool FUSED = few_fused(TOK);
  static constexpr int ALIGN = FUSED ? 1 : 8;             // first rows of token tiles
  static constexpr int XW = FUSED ? 8 : 0;                // quantizing warps
  static constexpr int XG = 2;                            // ... that share a stage, a block each
  static constexpr int TURNS = XW / XG;                   // stages in work at once
  static constexpr int X_BLOCK = TOK * kBlock;
  static constexpr int THREADS = (8 + XW) * 32;
  static constexpr int STAGE = W_BYTES + 2 * X_BLOCK;
  // as many stages as 196 KB holds: each has 32 KB of weights in flight
  static constexpr int STAGES = (196 * 1024) / STAGE;
  static constexpr int SFX_BUFS = FUSED ? STAGES : SF_BUFS;   // the activations' scale atoms: per stage if FUSED
  static constexpr int SFX_OFF = STAGES * STAGE;
  static constexpr int SFW_OFF = SFX_OFF + SFX_BUFS * kScaleAtom;   // the weights' scale atoms, per stage
  static constexpr int EPI_OFF = SFW_OFF + STAGES * kScaleAtom;
  static constexpr int TAB_OFF = EPI_OFF + EPI_WARPS * EPI_STAGE;
  static constexpr int BAR_OFF = (TAB_OFF + static_cast<int>(sizeof(ExpertTable)) + 15) & ~15;
  static constexpr int BYTES = 1024 + BAR_OFF + 512;
  static constexpr uint32_t SFX_COL = 2 * TOK;            // behind the two accumulators
  static constexpr uint32_t SFW_COL = SFX_COL + 4 * SFX_BUFS;
  static constexpr uint32_t TMEM_COLS = SFW_COL + 4 * STAGES <= 128 ? 128 : TOK <= 64 ? 256 : 512;
  static_assert(!FUSED || TOK == 16, "a quantizing warp takes 16 rows of a block");
  static_assert(STAGE % 1024 == 0, "operand tiles start on 1024-byte boundaries");
  static_assert(SFW_COL + 4 * STAGES <= TMEM_COLS, "accumulators and scales fit in TMEM");
  static_assert(TOK * TILE_N * 4 + 4 * EPI_STAGE <= SFX_OFF, "a split's sums and staging fit over the stages");
  static_assert(BYTES <= 232448, "fits in shared memory");
};

__device__ __forceinline__ void st_cluster_v2(uint32_t cluster_addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(cluster_addr), "r"(a), "r"(b) : "memory");
}

// A place in a CTA's sequence of stages: its unit of work and the stage in it.
struct Cursor {
  int item, kp;
  Item u;
};

// Asks for the weights of this CTA's first stages in L2 while the kernel in front still runs: a hint without
// effect on what later loads return, so it may run ahead of the wait.  For a dense call, whose first unit's
// column tile does not depend on the table.
__device__ __forceinline__ void prefetch_weights(const Params &p, int split, int stages) {
  const int rank = static_cast<int>(blockIdx.x) % split, nt = static_cast<int>(blockIdx.x) / split;
  const int cols = min(TILE_N, p.N - nt * TILE_N);
  const int pairs = (p.KS + 1) / 2;
  const int ks0 = 2 * (pairs * rank / split), ks1 = min(min(2 * (pairs * (rank + 1) / split), ks0 + 2 * stages), p.KS);
  const int ks = ks0 + static_cast<int>(threadIdx.x);
  if (cols > 0 && ks < ks1)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.w + (static_cast<size_t>(ks) * p.N +
                                                                           static_cast<size_t>(nt) * TILE_N) *
                                                                              kBlock),
                 "r"(cols * kBlock)
                 : "memory");
}

template <int TOK, int EPI>
__global__ void __launch_bounds__(Shape<TOK>::THREADS, 1)
    fp8_gemm_few_kernel(const __grid_constant__ Params p, int split) {
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
      dev::mbar_init(&full[s], S::FUSED ? 1 + S::XG : 1);
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
  // FUSED: nothing is read before the kernel in front has completed.  Otherwise that kernel is the quantizer,
  // which lets this one start only after its own wait: everything older (offsets and weights among it) has
  // completed by now, and only X's codes and scales have to be waited for, where they are first read.
  if constexpr (S::FUSED) {
    if (p.offsets == nullptr && warp == 0) prefetch_weights(p, split, S::STAGES);
    dev::grid_dependency_wait();
  }
  dev::grid_launch_dependents();
  if (warp == 2) fill_expert_table(p, TOK, S::ALIGN, tab);
  dev::tc_fence_before();
  __syncwarp();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int ntn = (p.N + TILE_N - 1) / TILE_N;
  const int items = tab->tiles[p.experts] * ntn;
  // this CTA's share of K: its rank in the cluster of `split` CTAs that share a unit
  const int rank = static_cast<int>(blockIdx.x) % split;
  const int first_item = static_cast<int>(blockIdx.x) / split, stride = static_cast<int>(gridDim.x) / split;
  const int pairs = (p.KS + 1) / 2;                       // stages of the whole K
  const int kp0 = pairs * rank / split, kp1 = pairs * (rank + 1) / split;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      // a stage's weights and their scales; its rows of X come with them or behind them.  Rows past the end of a
      // buffer are not copied: what the stage holds there reaches no output.
      const auto load_weights = [&](const Item &u, int kp, int s) {
        const uint32_t wbytes = static_cast<uint32_t>(min(TILE_N, p.N - u.nt * TILE_N)) * kBlock;
        const uint32_t xbytes = S::FUSED ? 0u : static_cast<uint32_t>(min(TOK, p.Mp - u.row0)) * kBlock;
        const int blocks = min(2, p.KS - 2 * kp);
        dev::mbar_arrive_expect_tx(&full[s], blocks * (wbytes + xbytes) + kScaleAtom);
        for (int b = 0; b < blocks; ++b)
          dev::bulk_load(smem + s * S::STAGE + b * W_BLOCK,
                         p.w + ((static_cast<size_t>(u.expert) * p.KS + 2 * kp + b) * p.N +
                                static_cast<size_t>(u.nt) * TILE_N) *
                                   kBlock,
                         wbytes, &full[s]);
        dev::bulk_load(smem + S::SFW_OFF + s * kScaleAtom, weight_atom(p, u.expert, u.nt, kp >> 1), kScaleAtom, &full[s]);
      };
      int ahead = 0;                                      // stages whose weights are under way before X is there
      if constexpr (!S::FUSED) {
        if (first_item < items) {
          const Item u = find_item(p, tab, TOK, S::ALIGN, ntn, first_item);
          for (; ahead < min(S::STAGES, kp1 - kp0); ++ahead) load_weights(u, kp0 + ahead, ahead);
        }
        dev::grid_dependency_wait();
      }
      int it = 0;
      bool ok = true;
      for (int item = first_item; item < items && ok; item += stride) {
        const Item u = find_item(p, tab, TOK, S::ALIGN, ntn, item);
        for (int kp = kp0; kp < kp1; ++kp, ++it) {
          const int s = it % S::STAGES;
          if (it >= ahead) {
            if (!dev::mbar_wait(&empty[s], ((it / S::STAGES) & 1) ^ 1, p.limit_ns, abort_flag)) {
              ok = false;
              break;
            }
            load_weights(u, kp, s);
          }
          if constexpr (!S::FUSED) {
            for (int b = 0; b < min(2, p.KS - 2 * kp); ++b)
              dev::bulk_load(smem + s * S::STAGE + W_BYTES + b * S::X_BLOCK,
                             p.x + (static_cast<size_t>(2 * kp + b) * p.Mp + u.row0) * kBlock,
                             static_cast<uint32_t>(min(TOK, p.Mp - u.row0)) * kBlock, &full[s]);
          }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        dev::report(p.status, SVDQ_ERR_TIMEOUT);
      }
      // every copy in flight lands before the CTA ends (if the quantizing warps gave up, `full` never completes:
      // then the copies had the whole limit to land)
      for (int j = max(0, it - S::STAGES); j < it; ++j)
        dev::mbar_wait(&full[j % S::STAGES], (j / S::STAGES) & 1, p.limit_ns, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ scales into TMEM, MMAs
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_mxf8(TILE_N, TOK);
      const uint32_t base = dev::smem_u32(smem);
      const uint64_t desc0 = dev::desc_sw128(base), sfw0 = dev::desc_sf(base + S::SFW_OFF), sfx0 = dev::desc_sf(base + S::SFX_OFF);
      int it = 0, quad = 0, n = 0;
      bool ok = true, issued = false;
      for (int item = first_item; item < items && ok; item += stride, ++n) {
        const int a = n & 1;
        if (!dev::mbar_wait(&tmem_empty[a], ((n >> 1) & 1) ^ 1, p.limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        dev::tc_fence_after();
        const uint32_t acc = tmem + a * TOK;
        uint32_t accumulate = 0;
        for (int kp = kp0; kp < kp1; ++kp, ++it) {
          const int s = it % S::STAGES, b = quad % SF_BUFS;
          const uint32_t sfw = tmem + S::SFW_COL + 4 * s, sfx = tmem + S::SFX_COL + 4 * (S::FUSED ? s : b);
          if constexpr (!S::FUSED) {
            if ((kp & 1) == 0 || kp == kp0) {
              if (!dev::mbar_wait(&sf_full[b], (quad / SF_BUFS) & 1, p.limit_ns, abort_flag)) {
                ok = false;
                break;
              }
              dev::tc_fence_after();
              dev::tmem_cp_32x128b_x4(sfx, sfx0 + desc_step(kScaleAtom) * b);
              issued = true;
            }
          }
          if (!dev::mbar_wait(&full[s], (it / S::STAGES) & 1, p.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          dev::tc_fence_after();
          issued = true;
          dev::tmem_cp_32x128b_x4(sfw, sfw0 + desc_step(kScaleAtom) * s);
          if constexpr (S::FUSED) dev::tmem_cp_32x128b_x4(sfx, sfx0 + desc_step(kScaleAtom) * s);
          const uint64_t dw = desc0 + desc_step(S::STAGE) * s;
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {
            if (2 * kp + blk >= p.KS) break;
            const uint32_t w_byte = 2 * (kp & 1) + blk;   // of a word of four blocks
            const uint32_t id = with_scale_bytes(idesc, w_byte, S::FUSED ? blk : w_byte);
#pragma unroll
            for (int j = 0; j < 4; ++j) {                 // K = 32 codes = 32 bytes per MMA
              umma_mxf8(acc, dw + desc_step(blk * W_BLOCK + 32 * j), dw + desc_step(W_BYTES + blk * S::X_BLOCK + 32 * j),
                        id, sfw, sfx, accumulate);
              accumulate = 1;
            }
          }
          dev::tc_commit(&empty[s]);
          if (!S::FUSED && ((kp & 1) == 1 || kp == kp1 - 1)) {
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
  } else if (!S::FUSED && warp == 2) {
    // ------------------------------------------------------------ the activations' scale words
    dev::grid_dependency_wait();
    int quad = 0;
    bool ok = true;
    for (int item = first_item; item < items && ok; item += stride) {
      const Item u = find_item(p, tab, TOK, S::ALIGN, ntn, item);
      for (int kw = kp0 >> 1; 2 * kw < kp1; ++kw, ++quad) {
        const int b = quad % SF_BUFS;
        uint32_t xw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = u.row0 + 32 * i + lane;
          xw[i] = 32 * i + lane < TOK && row < p.Mp ? p.sx[static_cast<size_t>(kw) * p.Mp + row] : 0u;
        }
        if (!dev::mbar_wait_warp(&sf_empty[b], ((quad / SF_BUFS) & 1) ^ 1, p.limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        reinterpret_cast<uint4 *>(smem + S::SFX_OFF + b * kScaleAtom)[lane] = make_uint4(xw[0], xw[1], xw[2], xw[3]);
        dev::fence_proxy_async();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&sf_full[b]);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      dev::report(p.status, SVDQ_ERR_TIMEOUT);
    }
  }
  if constexpr (S::FUSED) {
    if (warp >= 8) {
      // ---------------------------------------------------------- quantize X
      const int blk = (warp - 8) % S::XG, turn = (warp - 8) / S::XG, sub = lane >> 3, chunk = lane & 7;
      uint32_t raw[4][8];                                 // 16 rows of a block, 4 at a time
      const auto load = [&](const Cursor &c) {
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          const int row = c.u.row0 + 4 * st + sub, k = (2 * c.kp + blk) * kBlock + chunk * 16;
          const uint4 *src = reinterpret_cast<const uint4 *>(p.X + static_cast<size_t>(row) * p.ldx + k);
          const bool live = row < c.u.end;
          const uint4 v0 = live && k < p.K ? __ldcg(src) : make_uint4(0, 0, 0, 0);
          const uint4 v1 = live && k + 8 < p.K ? __ldcg(src + 1) : make_uint4(0, 0, 0, 0);
          raw[st][0] = v0.x, raw[st][1] = v0.y, raw[st][2] = v0.z, raw[st][3] = v0.w;
          raw[st][4] = v1.x, raw[st][5] = v1.y, raw[st][6] = v1.z, raw[st][7] = v1.w;
        }
      };
      // `stages` stages on in the CTA's sequence
      const auto advance = [&](Cursor &c, int stages) {
        const int item = c.item;
        for (c.kp += stages; c.kp >= kp1; c.kp -= kp1 - kp0) c.item += stride;
        if (c.item != item && c.item < items) c.u = find_item(p, tab, TOK, S::ALIGN, ntn, c.item);
      };
      bool ok = true;
      Cursor c{first_item, kp0, {}};
      if (first_item < items) {
        c.u = find_item(p, tab, TOK, S::ALIGN, ntn, first_item);
        advance(c, turn);
        if (c.item < items) load(c);
      }
      for (int it = turn; c.item < items; it += S::TURNS) {
        const int s = it % S::STAGES;
        uint8_t *dst = smem + s * S::STAGE + W_BYTES + blk * S::X_BLOCK, *sfx = smem + S::SFX_OFF + s * kScaleAtom + blk;
        uint32_t code[4][4], byte[4];
        const int rows = 2 * c.kp + blk < p.KS ? c.u.end - c.u.row0 : 0;   // step st has rows if 4 st is below this
#pragma unroll
        for (int st = 0; st < 4; ++st)
          if (4 * st < rows) byte[st] = quantize16(raw[st], code[st]);
        advance(c, S::TURNS);
        if (c.item < items) load(c);
        if (!dev::mbar_wait_warp(&empty[s], ((it / S::STAGES) & 1) ^ 1, p.limit_ns, abort_flag)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          if (4 * st >= rows) break;
          const int r = 4 * st + sub;                     // rows past the expert's: zeros, which reach no output
          *reinterpret_cast<uint4 *>(dst + r * kBlock + ((chunk ^ (r & 7)) << 4)) =
              make_uint4(code[st][0], code[st][1], code[st][2], code[st][3]);
          if (chunk == 0) sfx[r * 16] = static_cast<uint8_t>(byte[st]);
        }
        dev::fence_proxy_async();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&full[s]);
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        dev::report(p.status, SVDQ_ERR_TIMEOUT);
      }
    }
  }

  // ------------------------------------------------------------ epilogue
  const int q = warp & 3;                                 // TMEM lane quarter this warp may access
  uint8_t *stage = smem + S::EPI_OFF + q * EPI_STAGE;
  // bias, activation and rounding of two rows of a column into a staged chunk
  const auto finish2 = [&](float y0, float y1, float bias, bool act, int t) {
    const float2 y = make_float2(y0 + bias, y1 + bias);
    float2 g = activate2<EPI>(y);
    if constexpr (EPI != SVDQ_EPILOGUE_NONE) {
      g.x = act ? g.x : y.x;
      g.y = act ? g.y : y.y;
    }
    reinterpret_cast<__nv_bfloat16 *>(stage + t * 64)[lane] = __float2bfloat16_rn(g.x);
    reinterpret_cast<__nv_bfloat16 *>(stage + (t + 1) * 64)[lane] = __float2bfloat16_rn(g.y);
  };
  // `rows` (at most 32) staged rows of 32 columns to Y, 8 rows x 4 segments of 16 bytes at a time
  const auto store = [&](const Item &u, int row0, int rows) {
    const int col0 = u.nt * TILE_N + 32 * q;
    __syncwarp();
    for (int i = 0; i < rows; i += 8) {
      const int t = i + (lane >> 2), seg = lane & 3, row = row0 + t;
      if (t < rows && row >= u.begin && row < u.end && col0 + 8 * seg < p.N)
        *reinterpret_cast<uint4 *>(p.Y + static_cast<size_t>(row) * p.ldy + col0 + 8 * seg) =
            *reinterpret_cast<const uint4 *>(stage + t * 64 + seg * 16);
    }
    __syncwarp();
  };
  const auto bias_of = [&](const Item &u, int col) {
    return p.bias && col < p.N
               ? __uint_as_float(static_cast<uint32_t>(__ldg(p.bias + static_cast<size_t>(u.expert) * p.N + col)) << 16)
               : 0.0f;
  };
  constexpr int CH = TOK < 32 ? TOK : 32;                 // rows per chunk
  const auto read_chunk = [&](int a, int c, uint32_t (&v)[CH]) {
    const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(a * TOK + c);
    if constexpr (CH == 32) dev::tmem_ld_32x32b_x32(taddr, v);
    else tmem_ld_32x32b_x16(taddr, v);
    dev::tmem_wait_ld();
  };
  if constexpr (!S::FUSED)
    if (warp >= 4 || split > 1) dev::grid_dependency_wait();   // nothing is written before it
  if (split == 1) {
    if (warp >= 4 && warp < 8) {
      int n = 0;
      for (int item = first_item; item < items; item += stride, ++n) {
        const Item u = find_item(p, tab, TOK, S::ALIGN, ntn, item);
        const int a = n & 1, col = u.nt * TILE_N + 32 * q + lane;
        const float bias = bias_of(u, col);
        if (!dev::mbar_wait_warp(&tmem_full[a], (n >> 1) & 1, p.limit_ns, abort_flag)) {
          if (lane == 0) {
            *abort_flag = 1;
            dev::report(p.status, SVDQ_ERR_TIMEOUT);
          }
          break;
        }
        dev::tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < TOK && u.row0 + c < u.end; c += CH) {
          uint32_t v[CH];
          read_chunk(a, c, v);
#pragma unroll
          for (int t = 0; t < CH; t += 2)
            finish2(__uint_as_float(v[t]), __uint_as_float(v[t + 1]), bias, col >= p.gelu_col_begin, t);
          store(u, u.row0 + c, CH);
        }
        dev::tc_fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&tmem_empty[a]);
      }
    }
  } else {
    // One unit per cluster.  CTA j of the cluster finishes rows [j TC, (j + 1) TC) of the tile; the others send
    // it their sums of those rows, over its (idle) stages: [rank][two rows][column][2] floats, 8 bytes a lane, so
    // a warp's store or load is 256 contiguous bytes.  The first eight warps share the rows, their roles being
    // over.
    const int TC = TOK / split, half = warp >> 2;
    const bool mine = first_item < items;
    const Item u = mine ? find_item(p, tab, TOK, S::ALIGN, ntn, first_item) : Item{};
    const int col = u.nt * TILE_N + 32 * q + lane;
    bool ok = mine && warp < 8;
    const float bias = ok ? bias_of(u, col) : 0.0f;       // read under the exchange
    if (warp < 4) stage = smem + TOK * TILE_N * 4 + q * EPI_STAGE;   // behind the sums
    __syncwarp();
    if (ok && !dev::mbar_wait_warp(&tmem_full[0], 0, p.limit_ns, abort_flag)) {
      if (lane == 0) {
        *abort_flag = 1;
        dev::report(p.status, SVDQ_ERR_TIMEOUT);
      }
      ok = false;
    }
    __syncwarp();
    dev::cluster_sync();                                  // every CTA of the cluster is done with its stages
    if (ok) {
      dev::tc_fence_after();
      const uint32_t base = dev::smem_u32(smem) + static_cast<uint32_t>(rank * TC * TILE_N + 64 * q + 2 * lane) * 4u;
#pragma unroll 1
      for (int c = half * 16; c < TOK && u.row0 + c < u.end; c += 32) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(c), v);
        dev::tmem_wait_ld();
#pragma unroll
        for (int t = 0; t < 16; t += 2) {
          const int j = (c + t) / TC;
          st_cluster_v2(dev::mapa(base + static_cast<uint32_t>((c + t - j * TC) * TILE_N) * 4u, j), v[t], v[t + 1]);
        }
      }
    }
    __syncwarp();
    dev::cluster_sync();                                  // all sums have arrived
    if (ok) {
      const int row0 = u.row0 + rank * TC;
      const float2 *part = reinterpret_cast<const float2 *>(smem) + 32 * q + lane;
#pragma unroll 1
      for (int c = half * 16; c < TC && row0 + c < u.end; c += 32) {
        const int rows = min(16, TC - c);
        float2 y[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) y[t] = make_float2(0.0f, 0.0f);
        for (int j = 0; j < split; ++j) {                 // in the order of K
#pragma unroll
          for (int t = 0; t < 8; ++t)
            if (2 * t < rows) {
              const float2 f = part[(j * TC + c + 2 * t) / 2 * TILE_N];
              y[t].x += f.x;
              y[t].y += f.y;
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t)
          if (2 * t < rows) finish2(y[t].x, y[t].y, bias, col >= p.gelu_col_begin, 2 * t);
        store(u, row0 + c, rows);
      }
    }
  }

  // The elected threads' warps meet first: the 31 lanes that skipped a role would otherwise arrive at the barrier
  // without the 32nd, count as a whole warp, and let TMEM go while other warps still read it.
  dev::tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    dev::tc_fence_after();
    dev::tmem_dealloc(tmem, S::TMEM_COLS);
  }
}

// How many clusters of 2^log2 CTAs the current device runs at a time.  A cluster needs its SMs in one GPC, so clusters of
// 4 and 8 leave some SMs out (33 and 15 on a B200 with 148).  Asked once per device and size.
template <auto Kernel>
int resident_clusters(const cudaLaunchConfig_t &cfg, int log2) {
  static std::atomic<int> known[64][4];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if ((n = known[dev][log2].load(std::memory_order_relaxed)) != 0) return n - 1;
  if (cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  known[dev][log2].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int TOK, int EPI>
int launch(const char *fn, const Params &p, long long units, int sm_count, cudaStream_t stream) {
  using S = Shape<TOK>;
  int rc = smem_optin_once<fp8_gemm_few_kernel<TOK, EPI>>(S::BYTES, fn);
  if (rc != SVDQ_OK) return rc;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(S::THREADS);
  cfg.dynamicSmemBytes = S::BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  // Split K where that leaves every CTA four blocks of 128 along K and all clusters still run at once: a second wave
  // of them costs more than a split saves (16 rows, 4096 -> 2048, 16 units: 14.2 us as clusters of 8, of which 15 fit;
  // 7.6 us as clusters of 4).
  int split = 1;
  for (int log2 = 1; log2 <= 3 && p.KS >= 4 << log2 && units << log2 <= sm_count; ++log2) {
    attr[1].val.clusterDim.x = 1 << log2;
    cfg.gridDim = dim3(1 << log2);
    cfg.numAttrs = 2;
    if (units > resident_clusters<fp8_gemm_few_kernel<TOK, EPI>>(cfg, log2)) break;
    split = 1 << log2;
  }
  attr[1].val.clusterDim.x = split;
  cfg.gridDim = dim3(split > 1 ? static_cast<int>(units) * split : static_cast<int>(units < sm_count ? units : sm_count));
  cfg.numAttrs = split > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_gemm_few_kernel<TOK, EPI>, p, split);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string(fn) + " launch: " + cudaGetErrorString(e));
  return SVDQ_OK;
}
template <int TOK>
int launch(const char *fn, const Params &p, int epilogue, int sm_count, cudaStream_t stream) {
  // token tiles: one per TOK rows, and one that each expert with rows may leave unfilled
  // (two with rows rounded down to a multiple of 8)
  const long long live = p.experts < p.M ? p.experts : p.M;
  const long long tiles = p.offsets ? p.M / TOK + live + (Shape<TOK>::FUSED ? 0 : live) : (p.M + TOK - 1) / TOK;
  const long long units = tiles * ((p.N + TILE_N - 1) / TILE_N);
  return epilogue == SVDQ_EPILOGUE_GELU_ERF    ? launch<TOK, SVDQ_EPILOGUE_GELU_ERF>(fn, p, units, sm_count, stream)
         : epilogue == SVDQ_EPILOGUE_GELU_TANH ? launch<TOK, SVDQ_EPILOGUE_GELU_TANH>(fn, p, units, sm_count, stream)
                                               : launch<TOK, SVDQ_EPILOGUE_NONE>(fn, p, units, sm_count, stream);
}

}  // namespace

int launch_gemm_few(const char *fn, const Params &p, int tile, int epilogue, int sm_count, cudaStream_t stream) {
  return tile == 16   ? launch<16>(fn, p, epilogue, sm_count, stream)
         : tile == 32 ? launch<32>(fn, p, epilogue, sm_count, stream)
         : tile == 64 ? launch<64>(fn, p, epilogue, sm_count, stream)
                      : launch<128>(fn, p, epilogue, sm_count, stream);
}

}  // namespace fp8
}  // namespace svdq
