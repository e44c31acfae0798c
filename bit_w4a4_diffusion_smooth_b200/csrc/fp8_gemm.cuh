// Block-scaled FP8 GEMM, device side: what its kernels share.
//
//   Y[m][n] = bf16( act( sum_k (sx qx)[m][k] (sw qw)[n][k] + bias[n] ) )
//
// The products run as tcgen05.mma kind::mxf8f6f4 with block scales: the tensor
// core takes a ue8m0 byte per row and 32 elements from tensor memory and adds
// sx sw qx qw into an fp32 accumulator.  A block of 128 elements is four MMAs
// of K = 32 that all name the same byte: a scale word in tensor memory holds
// the bytes of four consecutive blocks, and the instruction's scale-factor ids
// pick one, so one 512-byte copy per 128 rows serves 512 elements along K.
#pragma once

#include <cuda_runtime.h>

#include "device_common.cuh"
#include "fp8_layout.h"
#include "svdq_internal.h"

namespace svdq {
namespace fp8 {

struct Params {
  const uint16_t *X;            // activations [M][ldx] bf16
  size_t ldx;
  const uint8_t *x;             // their codes [KS][Mp][128] and
  const uint32_t *sx;           // scale words [KW][Mp] (many rows only)
  const uint8_t *w;             // weight codes [experts][KS][N][128]
  const uint32_t *sw;           // weight scale atoms [experts][ceil(N / 128)][KW][128 words]
  const uint16_t *bias;         // [experts][N] bf16 or null
  uint16_t *Y;
  size_t ldy;
  const int *offsets;           // [experts + 1] or null: one expert with all rows
  int experts, M, Mp, N, K, KS, KW, gelu_col_begin;
  unsigned int *status;
  unsigned long long limit_ns;
};

// D(tmem) (+)= sum over K of (A . 2^sfa) (B . 2^sfb)^T, e4m3 inputs, one ue8m0 scale per 32 elements.
__device__ __forceinline__ void umma_mxf8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}

// True in one lane of a full, converged warp.  Code under `if (elect_one())` is known to run in a single thread, so
// the operands of tcgen05 and bulk-copy instructions go straight to uniform registers; under `if (lane == 0)` the
// compiler has to allow for several and issues each through a loop: 200 cycles an MMA against 110, measured on
// the 256 x 256 x 32 MMAs, which take 128.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(pred));
  return pred != 0;
}

// Operand descriptors as a 64-bit value to add to: `bytes` further on in shared memory, inside its 256 KB.
__host__ __device__ constexpr uint64_t desc_step(int bytes) { return static_cast<uint64_t>(bytes >> 4); }

// Instruction descriptor: A and B e4m3 (0), ue8m0 scales (bit 23), N >> 3 at 17, M >> 4 at 24, K-major.
__host__ __device__ constexpr uint32_t idesc_mxf8(int m, int n) {
  return (1u << 23) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
// ... with byte `a` of A's scale words (bit 29) and byte `b` of B's (bit 4).
__device__ __forceinline__ uint32_t with_scale_bytes(uint32_t idesc, uint32_t a, uint32_t b) {
  return idesc | (b << 4) | (a << 29);
}

// The weights' scale atom kw of the 128 columns of tile `tile128`.
__device__ __forceinline__ const uint32_t *weight_atom(const Params &p, int expert, int tile128, int kw) {
  return p.sw + ((static_cast<size_t>(expert) * ((p.N + 127) / 128) + tile128) * p.KW + kw) * (kScaleAtom / 4);
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Two float32 sums (one packed instruction).
__device__ __forceinline__ float2 add2_rn(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t *>(&a)), "l"(*reinterpret_cast<const uint64_t *>(&b)));
  return *reinterpret_cast<const float2 *>(&r);
}

// GELU, tanh form, of two values: 0.5 y (1 + tanh z) = y / (1 + exp(-2 z)), z = sqrt(2/pi) (y + 0.044715 y^3):
// no cancellation for negative y, and exp and the reciprocal come from the hardware approximations (a few
// 1e-7 relative), far below the bf16 rounding of the result.  exp(-2 z) overflows to infinity only where the
// result is below 1e-37, and 1 / infinity is the 0 it rounds to.
__device__ __forceinline__ float2 gelu_tanh2(float2 y) {
  const float2 y2 = dev::mul2_rn(y, y);
  // -2 z log2(e) = y (c0 + c1 y^2), c0 = -2 sqrt(2/pi) log2(e), c1 = 0.044715 c0
  const float2 p = dev::fma2_rn(make_float2(-0.10294324f, -0.10294324f), y2, make_float2(-2.3022082f, -2.3022082f));
  const float2 z = dev::mul2_rn(y, p);
  const float2 e = add2_rn(make_float2(dev::ex2_approx_ftz(z.x), dev::ex2_approx_ftz(z.y)), make_float2(1.0f, 1.0f));
  return dev::mul2_rn(y, make_float2(dev::rcp_approx_ftz(e.x), dev::rcp_approx_ftz(e.y)));
}
// GELU, erf form, of two values: y Phi(y) = max(y, 0) - |y| Phi(-|y|), Phi the normal distribution function.
// Phi(-a) = 2^P(-a): P is a polynomial of degree 10 fitted to log2 Phi(-a) for a in [0, 13.1] (least largest error, the
// error allowed to grow as (a / 1.4)^2.3 beyond 1.4), so the result is right in relative terms however small it gets:
// evaluated in float32, off by at most 6.1e-6 of itself down to y = -2, 4.8e-5 down to -5, 4.1e-4 (a tenth of bf16's half
// step) down to -13, and by 4.4e-7 anywhere.  A form whose error is bounded absolutely, as the handbooks' formulas for erf
// are, loses bf16's last bits from -3.5 on.  One special-function instruction a value and 17 instructions a pair
// (4608 x 2560 -> 10240: 126.3 us, 120.7 with the tanh form, 117.5 without a GELU).  a is capped at 13.1, where 2^P is no normal
// float32 any more and becomes 0 (results below 2^-121); the maximum passes NaN on.
__device__ __forceinline__ float max0_nan(float y) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(y));
  return r;
}
__device__ __forceinline__ float2 gelu_erf2_exp(float2 y) {
  const float2 na = make_float2(fmaxf(-fabsf(y.x), -13.1f), fmaxf(-fabsf(y.y), -13.1f));
  float2 d = dev::fma2_rn(make_float2(-2.680573818e-10f, -2.680573818e-10f), na, make_float2(-1.322072053e-08f, -1.322072053e-08f));
  d = dev::fma2_rn(d, na, make_float2(-2.133037498e-07f, -2.133037498e-07f));
  d = dev::fma2_rn(d, na, make_float2(1.023924412e-07f, 1.023924412e-07f));
  d = dev::fma2_rn(d, na, make_float2(5.282396887e-05f, 5.282396887e-05f));
  d = dev::fma2_rn(d, na, make_float2(8.985690656e-04f, 8.985690656e-04f));
  d = dev::fma2_rn(d, na, make_float2(8.424942382e-03f, 8.424942382e-03f));
  d = dev::fma2_rn(d, na, make_float2(5.383007973e-02f, 5.383007973e-02f));
  d = dev::fma2_rn(d, na, make_float2(-0.4585629106f, -0.4585629106f));
  d = dev::fma2_rn(d, na, make_float2(1.151224375f, 1.151224375f));
  d = dev::fma2_rn(d, na, make_float2(-0.9999963641f, -0.9999963641f));
  const float2 q = make_float2(dev::ex2_approx_ftz(d.x), dev::ex2_approx_ftz(d.y));
  return dev::fma2_rn(na, q, make_float2(max0_nan(y.x), max0_nan(y.y)));
}
template <int EPI>
__device__ __forceinline__ float2 activate2(float2 y) {
  if constexpr (EPI == SVDQ_EPILOGUE_GELU_ERF) return gelu_erf2_exp(y);
  if constexpr (EPI == SVDQ_EPILOGUE_GELU_TANH) return gelu_tanh2(y);
  return y;
}

// Rows and token tiles of the experts, in shared memory: expert e owns rows
// [start[e], start[e + 1]) and token tiles [tiles[e], tiles[e + 1]).  Offsets
// are taken as they come and clamped: into [0, M], and never below an earlier
// one, so whatever they hold, the experts' rows are disjoint and inside Y.
// Token tiles start at the expert's first row rounded down to a multiple of
// `align` (8 where operand rows come from the quantized layout).
struct ExpertTable {
  int start[FP8_MAX_EXPERTS + 1];
  int tiles[FP8_MAX_EXPERTS + 1];
};

// Fills the table; called by one full warp.
__device__ __forceinline__ void fill_expert_table(const Params &p, int tile_rows, int align, ExpertTable *t) {
  const int lane = threadIdx.x & 31;
  if (p.offsets == nullptr) {
    if (lane == 0) {
      t->start[0] = 0;
      t->start[1] = p.M;
      t->tiles[0] = 0;
      t->tiles[1] = (p.M + tile_rows - 1) / tile_rows;
    }
    return;
  }
  int first = min(max(__ldcg(p.offsets), 0), p.M);   // start of the expert `base`, the same in every lane
  int tiles = 0;
  for (int base = 0; base < p.experts; base += 32) {
    const int e = base + lane;
    int end = e < p.experts ? min(max(__ldcg(p.offsets + e + 1), 0), p.M) : 0;
    end = max(end, first);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {               // running maximum of the ends
      const int v = __shfl_up_sync(0xFFFFFFFFu, end, o);
      if (lane >= o) end = max(end, v);
    }
    int start = __shfl_up_sync(0xFFFFFFFFu, end, 1);
    if (lane == 0) start = first;
    const int mine = e < p.experts && end > start ? (end - (start & -align) + tile_rows - 1) / tile_rows : 0;
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    if (e < p.experts) {
      t->start[e] = start;
      t->tiles[e] = tiles + sum - mine;
      if (e == p.experts - 1) {
        t->start[p.experts] = end;
        t->tiles[p.experts] = tiles + sum;
      }
    }
    first = __shfl_sync(0xFFFFFFFFu, end, 31);
    tiles += __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
}

// A unit of work: the token tile [row0, row0 + tile_rows) of an expert against tile nt of the output columns.
// Rows below `begin` or from `end` on belong to others.  An expert's units are consecutive, in panels of kPanel
// column tiles, the panel's columns fastest: the units that run at the same time form a block of about as many
// token tiles as column tiles, and read few distinct operand rows.
constexpr int kPanel = 8;
struct Item {
  int expert, nt, row0, begin, end;
};
__device__ __forceinline__ Item find_item(const Params &p, const ExpertTable *t, int tile_rows, int align,
                                          int nt_count, int item) {
  int lo = 0, hi = p.experts;                         // the last expert whose first unit is <= item
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t->tiles[mid] * nt_count <= item) lo = mid;
    else hi = mid;
  }
  const int mts = t->tiles[lo + 1] - t->tiles[lo];
  int r = item - t->tiles[lo] * nt_count;
  const int panel = r / (kPanel * mts), width = min(kPanel, nt_count - panel * kPanel);
  r -= panel * kPanel * mts;
  Item it;
  it.expert = lo;
  it.nt = panel * kPanel + r % width;
  it.begin = t->start[lo];
  it.end = t->start[lo + 1];
  it.row0 = (it.begin & -align) + (r / width) * tile_rows;
  return it;
}

}  // namespace fp8
}  // namespace svdq
