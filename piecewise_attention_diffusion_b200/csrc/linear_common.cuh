// Shared by the two kernels of bsa_linear (linear.cu: many rows, linear_few.cu: few rows): the
// epilogue's operands and activations, how the work is split over the sums, the tensor maps.
#pragma once
#include <algorithm>

#include "common.cuh"
#include "forward_tiles.cuh"
#include "internal.h"
#include "sm100.cuh"
#include "types.cuh"

namespace bsa {
namespace linear {

using namespace sm100;

constexpr int kBK = 64;  // columns of X and W per step: one 128-byte swizzled row

// What the epilogue needs of a [Bt, H, L, d] operand with H * d = N columns.
struct View {
  int64_t batch, head, row;
  int cols;  // d
};

template <typename T>
struct Params {
  int Bt, L, N;
  int gate_rows;        // rows of an entry that share one gate vector
  int x_steps;          // 64-column steps per head of X
  int xb, xh;           // 0 where X's batch or head stride is 0 (one copy for all)
  int k_steps, row_tiles, m_tiles, n_tiles;
  int split;            // the groups share (tile, step) units instead of whole tiles
  const T* bias;
  const T* gate;
  const T* res;
  T* y;
  View rv, yv;
  int tma_out;          // Y's base and strides allow TMA stores
  int tma_res;          // R's base and strides allow TMA loads
  int rb, rh;           // 0 where R's batch or head stride is 0
  float* part;          // split sums: [2 groups][rows of a tile][columns of a tile]
  int part_rows;
  int32_t* status;
  uint64_t wait_ns;
};

// One run of steps [k0, k1) of a tile. A group g of G takes whole tiles g, g + G, ... or, where
// the work is split, an equal run of the units (tile, step): at most one tile whose sum an
// earlier group began and one that a later group ends. Such partial sums go to slot 2 g or
// 2 g + 1, and k_finish adds a tile's slots in the order of its steps.
struct Work {
  int tile, k0, k1;
};

// Group g's first unit of `units`: the first units % groups groups have one more.
__host__ __device__ __forceinline__ int first_unit(int units, int groups, int g) {
  const int q = units / groups, r = units - q * groups;
  return g * q + (g < r ? g : r);
}

struct WorkIter {
  int u, end, step;  // in units where the work is split, else in tiles
  template <typename P>
  __device__ __forceinline__ WorkIter(const P& p, int g, int groups) {
    const int tiles = p.m_tiles * p.n_tiles;
    if (p.split) {
      u = first_unit(tiles * p.k_steps, groups, g);
      end = first_unit(tiles * p.k_steps, groups, g + 1);
    } else {
      u = g;
      end = tiles;
    }
    step = groups;
  }
  template <typename P>
  __device__ __forceinline__ bool next(const P& p, Work& w) {
    if (u >= end) return false;
    if (p.split) {
      w.tile = u / p.k_steps;
      w.k0 = u - w.tile * p.k_steps;
      w.k1 = min(p.k_steps, w.k0 + (end - u));
      u += w.k1 - w.k0;
    } else {
      w.tile = u;
      w.k0 = 0;
      w.k1 = p.k_steps;
      u = end - u > step ? u + step : end;
    }
    return true;
  }
};

template <typename P>
__device__ __forceinline__ bool partial(const P& p, const Work& w) {
  return w.k1 - w.k0 != p.k_steps;
}

// Where group g leaves the partial sum of w (part_rows x cols floats).
template <typename P>
__device__ __forceinline__ float* slot_of(const P& p, const Work& w, int g, int cols) {
  return p.part + (2 * (int64_t)g + (w.k0 == 0 ? 1 : 0)) * p.part_rows * cols;
}

// z / (1 + 2^-w) for a pair
__device__ __forceinline__ float2 sigmoid_times(float2 z, float2 w) {
  return make_float2(__fdividef(z.x, 1.0f + ex2(-w.x)), __fdividef(z.y, 1.0f + ex2(-w.y)));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  return fma2(a, b, make_float2(-0.f, -0.f));
}

// 1 - Phi(a) = e^(-a^2 / 2) t Q(t), t = 1 / (1 + kTailP a), for a >= 0: t Q(t) is half the scaled
// complementary error function, Q of degree 6 with the least relative error, 6.3e-7 (a linear
// program over t). With fp32's rounding the product z Phi(z) is off by 5.3e-7 |z|.
constexpr float kTailP = 0.26516503f;
__device__ __forceinline__ float2 normal_tail(float2 a) {
  constexpr float kTail[7] = {0.105669923f, 0.107841954f, 0.0833459124f, 0.141495913f,
                              -0.0647517219f, 0.193937004f, -0.0675393045f};
  const float2 t = make_float2(__fdividef(1.0f, fmaf(a.x, kTailP, 1.0f)),
                               __fdividef(1.0f, fmaf(a.y, kTailP, 1.0f)));
  float2 q = make_float2(kTail[6], kTail[6]);
#pragma unroll
  for (int i = 5; i >= 0; --i) q = fma2(q, t, make_float2(kTail[i], kTail[i]));
  const float2 x = mul2(mul2(a, a), make_float2(-0.72134752f, -0.72134752f));  // -log2(e) / 2
  return mul2(mul2(q, t), make_float2(ex2(x.x), ex2(x.y)));
}

// The activation is a template argument: with a branch per element nothing overlapped, and
// the epilogue of a 128 x 256 tile took 40000 cycles where its products take 8300 (K = 1024).
template <int kAct>
__device__ __forceinline__ float2 activate(float2 z) {
  constexpr float kLog2e = 1.4426950408889634f;
  if (kAct == BSA_ACT_GELU_TANH) {  // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
    constexpr float c = 1.5957691216057308f * kLog2e, d = c * 0.044715f;
    const float2 t = fma2(mul2(z, z), make_float2(d, d), make_float2(c, c));
    return sigmoid_times(z, mul2(z, t));
  }
  if (kAct == BSA_ACT_GELU_ERF) {  // z Phi(z) by the normal tail, which keeps negative z's digits
    const float2 h = normal_tail(make_float2(fabsf(z.x), fabsf(z.y)));
    return make_float2(z.x * (z.x < 0.f ? h.x : 1.0f - h.x), z.y * (z.y < 0.f ? h.y : 1.0f - h.y));
  }
  if (kAct == BSA_ACT_SILU) return sigmoid_times(z, mul2(z, make_float2(kLog2e, kLog2e)));
  return z;
}

// ------------------------------------------------------------------ host side
// A [Bt][H][L][d] operand as a 4-D map with boxes of box_cols x box_rows.
template <typename T>
inline bool map_4d(CUtensorMap* m, const void* ptr, int d, int L, int H, int Bt, const bsa_strides& s,
            int box_cols, int box_rows) {
  fwdtiles::EncodeTiledFn enc = fwdtiles::encode_fn();
  if (!enc) return false;
  // a dimension that is never stepped over still needs a legal stride
  auto bytes = [](int64_t v) { return (cuuint64_t)(v > 0 ? v * 2 : 16); };
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)L, (cuuint64_t)(s.head ? H : 1),
                        (cuuint64_t)(s.batch ? Bt : 1)};
  cuuint64_t strides[3] = {bytes(s.row), bytes(s.head), bytes(s.batch)};
  cuuint32_t box[4] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, is_bf16<T>() ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols == kBK ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
inline bool map_w(CUtensorMap* m, const void* ptr, int K, int N, int64_t row, int box_rows) {
  fwdtiles::EncodeTiledFn enc = fwdtiles::encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)N};
  cuuint64_t strides[1] = {(cuuint64_t)(N > 1 ? row * 2 : 16)};
  cuuint32_t box[2] = {kBK, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, is_bf16<T>() ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
             const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool whole16(const void* ptr, const bsa_strides& s) {
  return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0 && s.batch % 8 == 0 && s.head % 8 == 0 &&
         s.row % 8 == 0;
}

// The plan of a call: which kernel, its tile, and whether its groups (CTA pairs or CTAs)
// share tiles.
struct Plan {
  bool few;     // the few-rows kernel (tiles of 128 columns, all rows) or CTA pairs
  int cols;     // columns per tile
  int rows;     // rows per tile (few: of X, a multiple of 16)
  int groups;
  bool split;
  size_t workspace(int L) const {
    return split ? (size_t)2 * groups * std::min(L, rows) * cols * sizeof(float) + kAlignSlack : 0;
  }
};
Plan plan_of(int Bt, int L, int k_steps, int N);

// What both kernels' parameters have in common.
template <typename T>
Params<T> params_of(const LinearArgs& a, const Plan& plan) {
  Params<T> p;
  p.Bt = a.Bt;
  p.L = a.L;
  p.N = a.N;
  p.gate_rows = a.gate_rows;
  const int dx = a.K / a.x_heads, dy = a.N / a.y_heads;
  p.x_steps = ceil_div(dx, kBK);
  p.xb = a.xs.batch != 0;
  p.xh = a.xs.head != 0;
  p.k_steps = p.x_steps * a.x_heads;
  p.row_tiles = ceil_div(a.L, plan.rows);
  p.m_tiles = a.Bt * p.row_tiles;
  p.n_tiles = ceil_div(a.N, plan.cols);
  p.split = plan.split;
  p.bias = static_cast<const T*>(a.bias);
  p.gate = static_cast<const T*>(a.gate);
  p.res = static_cast<const T*>(a.R);
  p.y = static_cast<T*>(a.Y);
  p.rv = View{a.rs.batch, a.rs.head, a.rs.row, dy};
  p.yv = View{a.ys.batch, a.ys.head, a.ys.row, dy};
  p.tma_out = whole16(a.Y, a.ys);
  p.tma_res = a.R != nullptr && whole16(a.R, a.rs) && (a.L == 1 || a.rs.row > 0);
  p.rb = a.rs.batch != 0;
  p.rh = a.rs.head != 0;
  p.part = align32(a.ws);
  p.part_rows = std::min(a.L, plan.rows);
  p.status = a.status;
  p.wait_ns = a.wait_ns > 0 ? a.wait_ns : kWaitTimeoutNs;
  return p;
}

// linear_few.cu; act as in LinearArgs.
template <typename T>
cudaError_t run_few(const LinearArgs& a, const Plan& plan, cudaStream_t st);

}  // namespace linear
}  // namespace bsa
