// Rotary positions over several axes (time, height, width) for the query and
// key heads of a fused projection, after an optional RMS norm of each head.
//
// Head dimension D splits into D/2 pairs; pair i belongs to axis a(i) with
// frequency f(i), and a token at position pos[a] turns it by pos[a(i)] f(i):
//   (x, y) -> (x cos - y sin, x sin + y cos)
// (sin negated for the inverse, which is also the turn's transpose).  With a
// norm weight, x is first x * rsqrt(mean x^2 + eps) * w over its head.
//
// Angles are taken in float64: a float32 product pos * f is off by up to
// pos 2^-24 radians, which at positions in the ten thousands is already bf16's
// own step.  They are counted in turns, with what the two products' roundings
// left out carried along, so that the whole turns come off right at any
// position; what is left, within half a turn, goes to float32, whose cosine and
// sine take the rest (up to 2^-26 turns) as a first-order term.  Both are then
// off by 3 * 2^-24 of their own value at most (a unit in the last place of
// sincospif and the term's rounding), next to a quarter turn too, where a
// rounded angle would lose a small cosine whole; everything else is float32,
// rounded once to bf16.  (Without the two terms: 0.1 us of 18.8 less for 4608
// normed rows x 40 heads x 128, 4.5 us against 4.7 for 9000 rows x 4 heads x
// 64.)  A block computes each of its tokens'
// D/2 angles once, into shared memory, and every head of those tokens uses
// them, so the call needs no table in memory and no launch to fill one.
//
// Bound by memory: each element is read and written once (4 bytes).  A lane
// holds 4 pairs of a head (8 elements): 16 contiguous bytes in the interleaved
// pairing (2i, 2i + 1), two runs of 8 bytes in the half-split one (i, i + D/2).
// A group of lanes keeps one token's cos and sin, times the norm weights of one
// tensor, in registers and walks over that tensor's heads, four heads' loads in
// flight at a time, each place loaded again as soon as its head is turned; the
// first four are under way while the block computes its angles.  64 registers
// let 8 blocks share an SM (4608 normed rows x 40 heads x 128: 18.8 us; 1.6
// more with 7, 4.2 with 9, which spill).  The arithmetic runs on f32x2 instructions, two pairs at once: with
// scalar ones, and the tensor chosen head by head, the normed call was bound by
// issue (30 us for those rows).
#include <cuda_runtime.h>

#include <cstdlib>
#include <string>
#include <utility>

#include "device_common.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace rope {
namespace {

constexpr int THREADS = 128;
constexpr int BLOCKS = 8;         // on an SM
constexpr int MAX_D = 256;
// 1 / 2 pi as the sum of two float64
constexpr double PER_RADIAN = 0.15915494309189535, PER_RADIAN_LOW = -9.839338337591243e-18;
static_assert(4 * (MAX_D / 8) <= THREADS, "a token's heads go to four groups of lanes at least");

struct Tensor {
  const uint16_t *x;
  uint16_t *y;
  const uint16_t *norm;         // [D] bf16 or null
  long long x_row, x_head, y_row, y_head;   // strides in elements
  int heads;
};
struct Params {
  Tensor t[2];                  // query, key (heads 0 when absent)
  const void *pos;              // [M][pos_row]: int32 or float32
  long long pos_row;
  int M, D;
  int lanes_log2, groups_log2;  // log2 of the lanes per head and of the groups per token
  int q_groups;                 // of which the first so many take the query's heads
  int pos_float, inverse;
  float eps, inv_d;
  double freq[MAX_D / 2];       // radians per position
  unsigned char axis[MAX_D / 2];
};

template <bool HALF>
__device__ __forceinline__ void load8(const uint16_t *p, int c, int D, uint32_t (&w)[4]) {
  if constexpr (HALF) {
    const uint2 a = *reinterpret_cast<const uint2 *>(p + 4 * c), b = *reinterpret_cast<const uint2 *>(p + D / 2 + 4 * c);
    w[0] = a.x;
    w[1] = a.y;
    w[2] = b.x;
    w[3] = b.y;
  } else {
    const uint4 a = *reinterpret_cast<const uint4 *>(p + 8 * c);
    w[0] = a.x;
    w[1] = a.y;
    w[2] = a.z;
    w[3] = a.w;
  }
}
template <bool HALF>
__device__ __forceinline__ void store8(uint16_t *p, int c, int D, const uint32_t (&w)[4]) {
  if constexpr (HALF) {
    *reinterpret_cast<uint2 *>(p + 4 * c) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2 *>(p + D / 2 + 4 * c) = make_uint2(w[2], w[3]);
  } else {
    *reinterpret_cast<uint4 *>(p + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

constexpr int UNROLL = 4;

// The 4 pairs of a lane as two sets of two: first and second elements.
template <bool HALF>
__device__ __forceinline__ void split(const uint32_t (&w)[4], float2 (&x0)[2], float2 (&x1)[2]) {
  const auto lo = [](uint32_t v) { return __uint_as_float(v << 16); };
  const auto hi = [](uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (HALF) {                     // words 0, 1: first elements; 2, 3: second elements
      x0[i] = make_float2(lo(w[i]), hi(w[i]));
      x1[i] = make_float2(lo(w[2 + i]), hi(w[2 + i]));
    } else {                                  // a word is a pair
      x0[i] = make_float2(lo(w[2 * i]), lo(w[2 * i + 1]));
      x1[i] = make_float2(hi(w[2 * i]), hi(w[2 * i + 1]));
    }
  }
}

template <bool HALF, bool NORM>
__global__ void __launch_bounds__(THREADS, BLOCKS) rope_nd_kernel(const __grid_constant__ Params p) {
  __shared__ float2 turn[THREADS];            // [tokens][D/2] (cos, sin)
  const int half_d = p.D / 2, lanes = 1 << p.lanes_log2;
  const int tokens = THREADS >> (p.lanes_log2 + p.groups_log2);
  const int m0 = static_cast<int>(blockIdx.x) * tokens;
  // A thread has at most one angle: with four groups a token or more, tokens D / 2 <= THREADS.  Its pair's axis and
  // frequency are loaded through generic addresses: as constants, which the compiler would read them as, a warp's 32
  // pairs took 32 accesses one after the other (9000 rows x 4 heads x 64: 3.3 us more).
  const int a_tok = static_cast<int>(threadIdx.x) / half_d, pair = static_cast<int>(threadIdx.x) % half_d;
  const double *freq = p.freq;
  const unsigned char *axis = p.axis;
  asm volatile("" : "+l"(freq), "+l"(axis));
  const double pair_freq = freq[pair];
  const int pair_axis = axis[pair];
  dev::grid_dependency_wait();
  dev::grid_launch_dependents();
  int raw = 0;
  if (a_tok < tokens && m0 + a_tok < p.M)
    raw = __ldcg(static_cast<const int *>(p.pos) + (m0 + a_tok) * p.pos_row + pair_axis);
  const int c = threadIdx.x & (lanes - 1);                              // 8 elements of a head; past D / 8 idle
  const int group = (threadIdx.x >> p.lanes_log2) & ((1 << p.groups_log2) - 1);
  const int tok = threadIdx.x >> (p.lanes_log2 + p.groups_log2);
  const bool on = c < p.D / 8 && m0 + tok < p.M;
  const long long m = m0 + tok;
  // this group's tensor, its first head and the step to the next
  const bool is_q = group < p.q_groups;
  const Tensor &t = p.t[is_q ? 0 : 1];
  const int first = is_q ? group : group - p.q_groups;
  const int step = is_q ? p.q_groups : (1 << p.groups_log2) - p.q_groups, heads = on ? t.heads : 0;
  // the same number of rounds for every lane: the norm's shuffles need full warps
  const int k_groups = (1 << p.groups_log2) - p.q_groups;
  const int rounds = max((p.t[0].heads + p.q_groups - 1) / p.q_groups, k_groups ? (p.t[1].heads + k_groups - 1) / k_groups : 0);
  const uint16_t *x = t.x + m * t.x_row;
  uint16_t *y = t.y + m * t.y_row;

  uint32_t w[UNROLL][4];
  const auto load = [&](int i, int round) {
    const int h = first + (round + i) * step;
    if (h < heads) {
      load8<HALF>(x + h * t.x_head, c, p.D, w[i]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[i][k] = 0u;
    }
  };
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) load(i, 0);
  const bool normed = NORM && t.norm != nullptr;
  uint32_t nw[4] = {0u, 0u, 0u, 0u};
  if constexpr (NORM)
    if (on && normed) load8<HALF>(t.norm, c, p.D, nw);

  // The frequency in turns and the position's product with it, each with what its rounding left out; then whole turns off.
  // (Where even a unit in the last place is whole turns, the second remainder keeps the angle within half a turn.)
  const double per = pair_freq * PER_RADIAN, per_low = fma(pair_freq, PER_RADIAN, -per) + pair_freq * PER_RADIAN_LOW;
  const double at = p.pos_float ? static_cast<double>(__int_as_float(raw)) : static_cast<double>(raw);
  const double turns = at * per, turns_low = fma(at, per_low, fma(at, per, -turns));
  double rest = (turns - rint(turns)) + turns_low;
  rest -= rint(rest);
  const float near = static_cast<float>(rest), off = static_cast<float>(rest - static_cast<double>(near)) * 6.2831853f;
  float sine, cosine;
  sincospif(2.0f * near, &sine, &cosine);
  const float sine_near = sine;
  sine = fmaf(cosine, off, sine);
  cosine = fmaf(-sine_near, off, cosine);
  turn[threadIdx.x] = make_float2(cosine, p.inverse ? -sine : sine);
  __syncthreads();
  // y0 = x0 c0 - x1 s1, y1 = x0 s0 + x1 c1: cos and sin, with the norm weight of the element they multiply
  float2 c0[2], s0[2], c1[2], s1[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = on ? turn[tok * half_d + 4 * c + 2 * i] : make_float2(0.0f, 0.0f);
    const float2 b = on ? turn[tok * half_d + 4 * c + 2 * i + 1] : make_float2(0.0f, 0.0f);
    c0[i] = c1[i] = make_float2(a.x, b.x);
    s0[i] = s1[i] = make_float2(a.y, b.y);
  }
  if constexpr (NORM) {
    if (on && normed) {
      float2 g0[2], g1[2];
      split<HALF>(nw, g0, g1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        c0[i] = dev::mul2_rn(c0[i], g0[i]);
        s0[i] = dev::mul2_rn(s0[i], g0[i]);
        c1[i] = dev::mul2_rn(c1[i], g1[i]);
        s1[i] = dev::mul2_rn(s1[i], g1[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) s1[i] = make_float2(-s1[i].x, -s1[i].y);

  for (int round = 0; round < rounds; round += UNROLL) {
    float scale[UNROLL];
    if constexpr (NORM) {                     // four heads' sums side by side: their shuffles overlap
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        float2 x0[2], x1[2];
        split<HALF>(w[i], x0, x1);
        float2 sum = dev::mul2_rn(x0[0], x0[0]);
        sum = dev::fma2_rn(x1[0], x1[0], sum);
        sum = dev::fma2_rn(x0[1], x0[1], sum);
        sum = dev::fma2_rn(x1[1], x1[1], sum);
        scale[i] = sum.x + sum.y;
      }
      if (round + UNROLL / 2 < rounds) {
        for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < UNROLL; ++i) scale[i] += __shfl_xor_sync(0xFFFFFFFFu, scale[i], o);
      } else {                                // two heads are left
        for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < UNROLL / 2; ++i) scale[i] += __shfl_xor_sync(0xFFFFFFFFu, scale[i], o);
      }
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) scale[i] = normed ? rsqrtf(fmaf(scale[i], p.inv_d, p.eps)) : 1.0f;
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      if (round + i >= rounds) break;
      float2 x0[2], x1[2], y0[2], y1[2];
      uint32_t out[4];
      split<HALF>(w[i], x0, x1);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        y0[k] = dev::fma2_rn(x1[k], s1[k], dev::mul2_rn(x0[k], c0[k]));
        y1[k] = dev::fma2_rn(x1[k], c1[k], dev::mul2_rn(x0[k], s0[k]));
        if constexpr (NORM) {
          y0[k] = dev::mul2_rn(y0[k], make_float2(scale[i], scale[i]));
          y1[k] = dev::mul2_rn(y1[k], make_float2(scale[i], scale[i]));
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if constexpr (HALF) {
          out[k] = pack2(y0[k].x, y0[k].y);
          out[2 + k] = pack2(y1[k].x, y1[k].y);
        } else {
          out[2 * k] = pack2(y0[k].x, y1[k].x);
          out[2 * k + 1] = pack2(y0[k].y, y1[k].y);
        }
      }
      // this place's next head before the store: no lane stores what another loads
      if (round + UNROLL < rounds) load(i, round + UNROLL);
      const int h = first + (round + i) * step;
      if (h < heads) store8<HALF>(y + h * t.y_head, c, p.D, out);
    }
  }
}

// Whether the M x heads vectors of D elements lie apart.
bool apart(int64_t row, int64_t head, int M, int heads, int D) {
  if (M == 1) return heads == 1 || head >= D;
  if (heads == 1) return row >= D;
  return row <= head ? row >= D && head / M >= row : head >= D && row / heads >= head;
}
// Whether a vector of `b` (a Y's) shares an element with one of `a`.  Exact where both have the same strides and neither
// overlaps itself; otherwise ranges that meet count as shared, unless the two lie beside one another in rows (or head
// planes) of one stride, as the heads of a fused projection do.
struct Heads {
  const void *at;
  int64_t row, head;
  int heads;
};
bool overlap(const Heads &a, const Heads &b, int M, int D) {
  const int64_t delta = (static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.at)) -
                         static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.at))) / 2;
  // the elements of each, from its first address on: strides may be negative or 0 (an X's), and nothing bounds them
  struct Range {
    __int128 lo, hi;
  };
  const auto range = [&](const Heads &t) {
    const __int128 rows = static_cast<__int128>(t.row) * (M - 1), heads = static_cast<__int128>(t.head) * (t.heads - 1);
    return Range{(rows < 0 ? rows : 0) + (heads < 0 ? heads : 0), (rows > 0 ? rows : 0) + (heads > 0 ? heads : 0) + D};
  };
  const Range ra = range(a), rb = range(b);
  if (rb.lo + delta >= ra.hi || ra.lo >= rb.hi + delta) return false;
  const bool one_row = M == 1 || a.row == b.row, one_head = a.heads == 1 || b.heads == 1 || a.head == b.head;
  if (one_row && one_head && apart(a.row, a.head, M, a.heads, D)) {
    const int64_t head = a.heads > 1 ? a.head : b.head;
    // m row + h head + d = delta, with |d| < D, m and h a difference of two rows and of two heads: the wider stride's
    // factor is one of the two next to the quotient, then the other's
    struct Dim {
      int64_t step, lo, hi;
    } wide = {M > 1 ? b.row : 0, 1 - M, M - 1}, near = {a.heads > 1 || b.heads > 1 ? head : 0, 1 - b.heads, a.heads - 1};
    if (wide.step < near.step) std::swap(wide, near);
    const auto quotient = [](int64_t n, const Dim &dim) {
      return dim.step > 0 ? n / dim.step - (n % dim.step < 0) : 0;
    };
    const int64_t i0 = quotient(delta, wide);
    for (int64_t i = i0; i <= i0 + 1; ++i) {
      if (i < wide.lo || i > wide.hi) continue;
      const int64_t rest = delta - i * wide.step, j0 = quotient(rest, near);
      for (int64_t j = j0; j <= j0 + 1; ++j)
        if (j >= near.lo && j <= near.hi && std::abs(rest - j * near.step) < D) return true;
    }
    return false;
  }
  // each a run of `run` elements, and those `period` apart: beside one another if the second's place in the first's
  // period is behind the first's run and ends before the next
  const auto beside = [&](int64_t period, __int128 run_a, __int128 run_b) {
    if (period <= 0) return false;
    const int64_t place = (delta % period + period) % period;
    return place >= run_a && place + run_b <= period;
  };
  const auto run = [&](int64_t step, int n) { return static_cast<__int128>(step) * (n - 1) + D; };
  if (M > 1 && a.row == b.row && (a.heads == 1 || a.head >= 0) && (b.heads == 1 || b.head >= 0) &&
      beside(a.row, run(a.heads > 1 ? a.head : 0, a.heads), run(b.heads > 1 ? b.head : 0, b.heads)))
    return false;
  return !(a.heads > 1 && b.heads > 1 && a.head == b.head && (M == 1 || (a.row >= 0 && b.row >= 0)) &&
           beside(a.head, run(M > 1 ? a.row : 0, M), run(M > 1 ? b.row : 0, M)));
}
int check_tensor(const char *which, const rope_nd_tensor_t &t, int M, int D) {
  const std::string name = std::string("rope_nd: ") + which;
  if (!t.X || !t.Y) return fail(SVDQ_ERR_INVALID_ARG, name + ": null pointer");
  if (t.x_row % 8 || t.x_head % 8 || t.y_row % 8 || t.y_head % 8)
    return fail(SVDQ_ERR_ALIGNMENT, name + ": strides must be multiples of 8 elements");
  if (!aligned16(t.X) || !aligned16(t.Y) || (t.norm && !aligned16(t.norm)))
    return fail(SVDQ_ERR_ALIGNMENT, name + ": pointers must be 16-byte aligned");
  if (!apart(t.y_row, t.y_head, M, t.heads, D))
    return fail(SVDQ_ERR_SHAPE, name + ": the heads of Y overlap");
  if (t.X == t.Y && ((M > 1 && t.x_row != t.y_row) || (t.heads > 1 && t.x_head != t.y_head)))
    return fail(SVDQ_ERR_INVALID_ARG, name + ": Y may be X only with the same strides");
  return SVDQ_OK;
}

}  // namespace
}  // namespace rope
}  // namespace svdq

using namespace svdq;

extern "C" int rope_nd(const rope_nd_tensor_t *Q, const rope_nd_tensor_t *K, int M, const rope_nd_plan_t *plan,
                       const void *pos, int64_t pos_row, int pos_is_float, int inverse, float eps,
                       svdq_stream_t stream) {
  using namespace svdq::rope;
  if (!Q || !plan || !pos) return fail(SVDQ_ERR_INVALID_ARG, "rope_nd: null pointer");
  if (plan->pairing != ROPE_ND_INTERLEAVED && plan->pairing != ROPE_ND_HALF)
    return fail(SVDQ_ERR_INVALID_ARG, "rope_nd: unknown pairing");
  const int D = plan->D;
  if (M < 1 || M > ROPE_ND_MAX_ROWS || D < 8 || D > MAX_D || D % 8 || plan->axes < 1 || plan->axes > D / 2 || Q->heads < 1 ||
      (K && K->heads < 1) || pos_row < 0 ||
      Q->heads > 65535 || (K && K->heads > 65535))
    return fail(SVDQ_ERR_SHAPE, "rope_nd: need 1 <= M <= 2^30, D % 8 == 0, 8 <= D <= 256, 1 <= axes <= D / 2, 1 <= heads <= "
                                "65535, pos_row >= 0");
  Params p{};
  for (int i = 0; i < D / 2; ++i) {
    if (plan->axis[i] >= plan->axes) return fail(SVDQ_ERR_SHAPE, "rope_nd: a pair's axis is outside [0, axes)");
    p.axis[i] = plan->axis[i];
    p.freq[i] = plan->freq[i];
  }
  int rc = check_tensor("query", *Q, M, D);
  if (rc == SVDQ_OK && K) rc = check_tensor("key", *K, M, D);
  if (rc != SVDQ_OK) return rc;
  if (inverse && (Q->norm || (K && K->norm)))
    return fail(SVDQ_ERR_INVALID_ARG, "rope_nd: the inverse undoes the turn only and takes no norm");
  if (reinterpret_cast<uintptr_t>(pos) & 3u) return fail(SVDQ_ERR_ALIGNMENT, "rope_nd: pos must be 4-byte aligned");
  const auto shared = [&](const rope_nd_tensor_t &a, bool out, const rope_nd_tensor_t &b) {   // a's X or Y and b's Y
    return overlap(out ? Heads{a.Y, a.y_row, a.y_head, a.heads} : Heads{a.X, a.x_row, a.x_head, a.heads},
                   Heads{b.Y, b.y_row, b.y_head, b.heads}, M, D);
  };
  if ((Q->X != Q->Y && shared(*Q, false, *Q)) ||
      (K && ((K->X != K->Y && shared(*K, false, *K)) || shared(*Q, false, *K) || shared(*K, false, *Q) || shared(*Q, true, *K))))
    return fail(SVDQ_ERR_INVALID_ARG, "rope_nd: a Y overlaps another Y, another tensor's X, or part of its own");
  DeviceState *st = current_device_state();
  if (!st) return SVDQ_ERR_NOT_INITIALIZED;
  for (int i = 0; i < 2; ++i) {
    const rope_nd_tensor_t *s = i == 0 ? Q : K;
    if (!s) continue;
    p.t[i] = Tensor{static_cast<const uint16_t *>(s->X), static_cast<uint16_t *>(s->Y),
                    static_cast<const uint16_t *>(s->norm), s->x_row, s->x_head, s->y_row, s->y_head, s->heads};
  }
  p.pos = pos;
  p.pos_row = pos_row;
  p.M = M;
  p.D = D;
  p.pos_float = pos_is_float;
  p.inverse = inverse;
  p.eps = eps;
  p.inv_d = 1.0f / static_cast<float>(D);
  while ((1 << p.lanes_log2) < D / 8) ++p.lanes_log2;
  // Groups per token: four, which with a block's tokens makes one angle a thread (eight: 21.4 us for 4608 normed rows x
  // 40 heads x 128, and 7.6 us for 9000 rows x 4 heads x 64); more while that leaves SMs without a block or two.  Each tensor's heads take a share of the groups by
  // their number.
  const int hq = Q->heads, hk = K ? K->heads : 0, most = 7 - p.lanes_log2;   // log2 of a block's groups
  const auto blocks_at = [&](int g) {
    const int tokens = 1 << (most - g);
    return (M + tokens - 1) / tokens;
  };
  p.groups_log2 = most < 2 ? most : 2;
  while (p.groups_log2 < most && (2 << p.groups_log2) <= hq + hk && blocks_at(p.groups_log2) < 2 * st->sm_count)
    ++p.groups_log2;
  const int groups = 1 << p.groups_log2;
  p.q_groups = groups;
  if (hk) {
    p.q_groups = (groups * hq + (hq + hk) / 2) / (hq + hk);
    p.q_groups = p.q_groups < 1 ? 1 : p.q_groups > groups - 1 ? groups - 1 : p.q_groups;
  }
  DependentLaunch dl(dim3(blocks_at(p.groups_log2)), dim3(THREADS), 0, stream);
  const bool norm = Q->norm || (K && K->norm);
  cudaError_t e = plan->pairing == ROPE_ND_HALF
                      ? (norm ? cudaLaunchKernelEx(&dl.cfg, rope_nd_kernel<true, true>, p)
                              : cudaLaunchKernelEx(&dl.cfg, rope_nd_kernel<true, false>, p))
                      : (norm ? cudaLaunchKernelEx(&dl.cfg, rope_nd_kernel<false, true>, p)
                              : cudaLaunchKernelEx(&dl.cfg, rope_nd_kernel<false, false>, p));
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string("rope_nd launch: ") + cudaGetErrorString(e));
  return ok();
}
