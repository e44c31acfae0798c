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
// own step.  They cost little: a block computes each of its tokens' D/2 angles
// once, into shared memory, and every head of those tokens uses them, so the
// call needs no table in memory and no launch to fill one.  Everything else is
// float32, rounded once to bf16.
//
// Bound by memory: each element is read and written once (4 bytes).  A lane
// holds 4 pairs of a head (8 elements): 16 contiguous bytes in the interleaved
// pairing (2i, 2i + 1), two runs of 8 bytes in the half-split one (i, i + D/2).
#include <cuda_runtime.h>

#include <string>

#include "device_common.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace rope {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_D = 256;

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
  int M, D, tokens, group_log2; // tokens per block; log2 of the lanes per head
  int pos_float, inverse;
  float eps;
  double freq[MAX_D / 2];
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
__device__ __forceinline__ void widen(const uint32_t (&w)[4], float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

template <bool HALF>
__global__ void __launch_bounds__(THREADS) rope_nd_kernel(const __grid_constant__ Params p) {
  extern __shared__ float2 turn[];            // [tokens][D/2] (cos, sin)
  dev::grid_dependency_wait();
  dev::grid_launch_dependents();
  const int half_d = p.D / 2;
  const int m0 = static_cast<int>(blockIdx.x) * p.tokens;
  const int live = min(p.tokens, p.M - m0);
  for (int i = threadIdx.x; i < live * half_d; i += THREADS) {
    const int tok = i / half_d, pair = i % half_d;
    const long long at = static_cast<long long>(m0 + tok) * p.pos_row + p.axis[pair];
    const double pos = p.pos_float ? static_cast<double>(__ldg(static_cast<const float *>(p.pos) + at))
                                   : static_cast<double>(__ldg(static_cast<const int *>(p.pos) + at));
    double s, c;
    sincos(pos * p.freq[pair], &s, &c);
    turn[i] = make_float2(static_cast<float>(c), static_cast<float>(p.inverse ? -s : s));
  }
  __syncthreads();

  // a group of 2^group_log2 lanes per head vector, the lanes past D/8 idle
  const int lanes = 1 << p.group_log2, c = threadIdx.x & (lanes - 1);
  const int groups = THREADS >> p.group_log2;
  const bool on = c < p.D / 8;
  const int heads = p.t[0].heads + p.t[1].heads;
  const int total = live * heads;
  const int rounds = (total + groups - 1) / groups;   // the same for all lanes: the norm's shuffles need full warps
  for (int r = 0; r < rounds; ++r) {
    const int v = r * groups + static_cast<int>(threadIdx.x >> p.group_log2);
    const bool act = on && v < total;
    const int tok = act ? v / heads : 0, h = act ? v % heads : 0;
    const Tensor &t = p.t[h < p.t[0].heads ? 0 : 1];
    const int th = h < p.t[0].heads ? h : h - p.t[0].heads;
    uint32_t w[4] = {0, 0, 0, 0};
    if (act) load8<HALF>(t.x + (m0 + tok) * t.x_row + th * t.x_head, c, p.D, w);
    float f[8];
    widen(w, f);
    float scale = 1.0f;
    if (p.t[0].norm || p.t[1].norm) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
      for (int o = lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      scale = rsqrtf(sum / static_cast<float>(p.D) + p.eps);
    }
    if (!act) continue;
    if (t.norm) {
      uint32_t nw[4];
      load8<HALF>(t.norm, c, p.D, nw);
      float g[8];
      widen(nw, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * scale * g[i];
    }
    const float2 *cs = turn + tok * half_d + 4 * c;
    uint32_t out[4];
    if constexpr (HALF) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = f[i] * cs[i].x - f[4 + i] * cs[i].y;
        b[i] = f[i] * cs[i].y + f[4 + i] * cs[i].x;
      }
      out[0] = pack2(a[0], a[1]);
      out[1] = pack2(a[2], a[3]);
      out[2] = pack2(b[0], b[1]);
      out[3] = pack2(b[2], b[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        out[i] = pack2(f[2 * i] * cs[i].x - f[2 * i + 1] * cs[i].y, f[2 * i] * cs[i].y + f[2 * i + 1] * cs[i].x);
    }
    store8<HALF>(t.y + (m0 + tok) * t.y_row + th * t.y_head, c, p.D, out);
  }
}

// Whether the M x heads vectors of D elements lie apart.
bool apart(int64_t row, int64_t head, int M, int heads, int D) {
  if (M == 1) return heads == 1 || head >= D;
  if (heads == 1) return row >= D;
  return row <= head ? row >= D && head / M >= row : head >= D && row / heads >= head;
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
  if (M < 1 || D < 8 || D > MAX_D || D % 8 || plan->axes < 1 || plan->axes > D / 2 || Q->heads < 1 ||
      (K && K->heads < 1) || pos_row < 0 ||
      Q->heads > 65535 || (K && K->heads > 65535))
    return fail(SVDQ_ERR_SHAPE, "rope_nd: need M >= 1, D % 8 == 0, 8 <= D <= 256, 1 <= axes <= D / 2, 1 <= heads <= "
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
  while ((1 << p.group_log2) < D / 8) ++p.group_log2;
  // one angle per thread: as many tokens a block as have THREADS pairs together, unless that leaves SMs idle
  p.tokens = M >= 4 * st->sm_count ? (2 * THREADS + D - 1) / D : 1;
  const int blocks = (M + p.tokens - 1) / p.tokens;
  const size_t smem = static_cast<size_t>(p.tokens) * (D / 2) * sizeof(float2);
  DependentLaunch dl(dim3(blocks), dim3(THREADS), smem, stream);
  cudaError_t e = plan->pairing == ROPE_ND_HALF ? cudaLaunchKernelEx(&dl.cfg, rope_nd_kernel<true>, p)
                                                : cudaLaunchKernelEx(&dl.cfg, rope_nd_kernel<false>, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string("rope_nd launch: ") + cudaGetErrorString(e));
  return ok();
}
