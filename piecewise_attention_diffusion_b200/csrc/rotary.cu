// bsa_rotary: rotary positions with up to four axes on a [Bt, H, L, d] tensor.
//
// Every pair (x_lo, x_hi) of components turns by phi = pos[axis] * base^(-2 i / axis_dim):
//     y_lo = x_lo cos phi - x_hi sin phi,   y_hi = x_lo sin phi + x_hi cos phi.
// phi depends on the token and the pair, not on the head, so a thread takes W pairs of one
// token, forms their sines and cosines once, and walks over a group of heads: per head it
// loads its components, turns them and stores them. The kernel reads x and writes y once
// and is bound by memory; what keeps enough bytes in flight is that kUnroll heads are
// loaded before the first is turned, the first of them before the sines are formed.
// Inputs out of L2: 40 heads x 16384 tokens x 128 bf16 components in 55.4 us, 6.07 TB/s of
// reads and writes (56.5 with the sines first); 2 x 12 heads x 4099 tokens x 120 fp32
// components in 18.3 to 19.3 us, 4.9 to 5.2 TB/s (20.0).
//
// The angle is formed in 64 bits as a number of turns, pos * base^(-2 i / axis_dim) / 2 pi,
// whose whole part is dropped before rounding to fp32: in 32 bits the angle of position
// 16384 would already be off by 1e-3. With u = ln(base) 2 i / axis_dim the rate is off by
// (u + 3.4) 2^-53 of itself (the exponent's rounding, pow to an ulp, pi, the quotient) and the
// product by 2^-53 more, so an angle by |pos| e^-u (u + 4.4) 2^-53 < |pos| 2^-50 radians.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "forward_tiles.cuh"
#include "internal.h"
#include "types.cuh"

namespace bsa {
namespace rotary {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;  // d <= 256
constexpr int kUnroll = 4;      // heads in flight per thread
constexpr int kCopy = 255;      // axis of the components that no axis turns

struct Params {
  const void* x;
  void* y;
  bsa_strides xs, ys;
  const float* pos;
  int Bt, H, L, n_axes, pos_per_batch, heads_per_cta;
  int groups;  // threads per token: pairs / W
  int64_t n;   // tokens in all: Bt * L
  float sign;
  // of every pair: turns per unit of position, axis, first and second component
  double rate[kMaxPairs];
  uint8_t axis[kMaxPairs], lo[kMaxPairs], hi[kMaxPairs];
};

// N bytes, as words where there are any.
template <int N>
struct alignas(N < 16 ? N : 16) Bytes {
  uint32_t w[N / 4];
};
template <>
struct alignas(2) Bytes<2> {
  uint16_t w[1];
};

// Element i of a run of T.
template <typename T, int N>
__device__ __forceinline__ float element(const Bytes<N>& b, int i) {
  if constexpr (N == 2) return to_f32(*reinterpret_cast<const T*>(&b.w[0]));
  else if constexpr (sizeof(T) == 4) return __uint_as_float(b.w[i]);
  else return i % 2 == 0 ? unpack2<T>(b.w[i / 2]).x : unpack2<T>(b.w[i / 2]).y;
}

// A run of T from fp32 values.
template <typename T, int N>
__device__ __forceinline__ Bytes<N> run_of(const float (&f)[N / sizeof(T)]) {
  Bytes<N> b;
  if constexpr (N == 2) {
    const T t = from_f32<T>(f[0]);
    b.w[0] = *reinterpret_cast<const uint16_t*>(&t);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      if constexpr (sizeof(T) == 4) b.w[i] = __float_as_uint(f[i]);
      else b.w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
    }
  }
  return b;
}

// W pairs per thread. kAdjacent: 2W consecutive components; else W consecutive first
// components and W consecutive second ones (the host chose W so that neither run crosses
// a section). kAgain: CTAs that fill the SMs go on to further tokens, instead of CTAs for all.
template <typename T, int W, bool kAdjacent, bool kAgain>
__global__ void __launch_bounds__(kThreads)
k_rotary(const __grid_constant__ Params p) {
  // the pair tables, from the parameters (whose reads are serial where lanes differ)
  __shared__ double rate_s[kMaxPairs];
  __shared__ uint8_t axis_s[kMaxPairs];
  const int pairs = p.groups * W;
  for (int i = threadIdx.x; i < pairs; i += kThreads) {
    rate_s[i] = p.rate[i];
    axis_s[i] = p.axis[i];
  }
  __syncthreads();
  int g;
  int64_t token;
  if constexpr (kAgain) {
    const int per_cta = kThreads / p.groups;
    if (threadIdx.x >= per_cta * p.groups) return;
    g = threadIdx.x % p.groups;
    token = (int64_t)blockIdx.x * per_cta + threadIdx.x / p.groups;
  } else {
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    g = (int)(id % p.groups);
    token = id / p.groups;
  }
  do {
    if (token >= p.n) return;
    int t, b;
    if constexpr (kAgain) {
      b = (uint32_t)token / (uint32_t)p.L;
      t = (uint32_t)token - b * (uint32_t)p.L;
    } else {
      t = (int)(token % p.L);
      b = (int)(token / p.L);
    }
    const float* pos = p.pos + ((p.pos_per_batch ? (int64_t)b * p.L : 0) + t) * p.n_axes;

    const int lo = p.lo[g * W], hi = p.hi[g * W];
    const int h0 = blockIdx.y * p.heads_per_cta;
    const int h1 = min(h0 + p.heads_per_cta, p.H);
    const T* x = static_cast<const T*>(p.x) + b * p.xs.batch + t * p.xs.row + h0 * p.xs.head;
    T* y = static_cast<T*>(p.y) + b * p.ys.batch + t * p.ys.row + h0 * p.ys.head;
    constexpr int kRun = (int)sizeof(T) * W * (kAdjacent ? 2 : 1);

    // the first heads' components are asked for before the sines are formed
    Bytes<kRun> first[kUnroll], second[kUnroll];
    auto fetch = [&](int h) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (h + u < h1) {
          const T* row = x + u * p.xs.head;
          first[u] = *reinterpret_cast<const Bytes<kRun>*>(row + lo);
          if (!kAdjacent) second[u] = *reinterpret_cast<const Bytes<kRun>*>(row + hi);
        }
      x += kUnroll * p.xs.head;
    };
    fetch(h0);

    float c[W], s[W];
    bool copy[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const int axis = axis_s[g * W + j];
      copy[j] = axis == kCopy;
      c[j] = 1.f;
      s[j] = 0.f;
      if (!copy[j]) {
        double turns = (double)__ldg(pos + axis) * rate_s[g * W + j];
        turns -= rint(turns);
        sincospif((float)(2.0 * turns), &s[j], &c[j]);
        s[j] *= p.sign;
      }
    }
    for (int h = h0; h < h1; h += kUnroll) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (h + u < h1) {
          T* row = y + u * p.ys.head;
          if constexpr (kAdjacent) {
            float f[2 * W];
#pragma unroll
            for (int j = 0; j < W; ++j) {
              const float xa = element<T>(first[u], 2 * j), xb = element<T>(first[u], 2 * j + 1);
              f[2 * j] = xa * c[j] - xb * s[j];
              f[2 * j + 1] = xa * s[j] + xb * c[j];
            }
            Bytes<kRun> out = run_of<T, kRun>(f);
            // copied components are taken bit for bit: an infinity, a NaN stays as it is
            constexpr int kPairWords = (int)sizeof(T) / 2;
#pragma unroll
            for (int i = 0; i < kRun / 4; ++i)
              if (copy[i / kPairWords]) out.w[i] = first[u].w[i];
            *reinterpret_cast<Bytes<kRun>*>(row + lo) = out;
          } else {
            // the run lies in one section: turned or copied as a whole
            if (!copy[0]) {
              float f[W], d[W];
#pragma unroll
              for (int j = 0; j < W; ++j) {
                const float xa = element<T>(first[u], j), xb = element<T>(second[u], j);
                f[j] = xa * c[j] - xb * s[j];
                d[j] = xa * s[j] + xb * c[j];
              }
              first[u] = run_of<T, kRun>(f);
              second[u] = run_of<T, kRun>(d);
            }
            *reinterpret_cast<Bytes<kRun>*>(row + lo) = first[u];
            *reinterpret_cast<Bytes<kRun>*>(row + hi) = second[u];
          }
        }
      y += kUnroll * p.ys.head;
      fetch(h + kUnroll);
    }
    if constexpr (kAgain) token += (int64_t)gridDim.x * (kThreads / p.groups);
  } while (kAgain);
}

template <typename T, int W, bool kAdjacent>
cudaError_t run(Params& p, cudaStream_t st) {
  int pairs = 0;
  while (pairs < kMaxPairs && p.axis[pairs] != 254) ++pairs;
  p.groups = pairs / W;
  p.n = (int64_t)p.Bt * p.L;
  const int64_t ctas = (p.n * p.groups + kThreads - 1) / kThreads;
  // all heads in one thread share its sines; fewer per thread where that leaves the card
  // short of CTAs
  const int sms = fwdtiles::sm_count();
  const int64_t want = sms * 8;
  int split = (int)std::min<int64_t>(ceil_div(p.H, kUnroll), (want + ctas - 1) / ctas);
  p.heads_per_cta = ceil_div(ceil_div(p.H, split), kUnroll) * kUnroll;
  const unsigned heads = (unsigned)ceil_div(p.H, p.heads_per_cta);
  // A thread with one pair of few heads ends before its CTA's tables have paid. bf16, halves paired,
  // odd sections of 128, 4 entries: 3 heads x 30323 tokens 89 us, 172 with CTAs for all; 16 x 12000
  // 99, 105.
  if (W == 1 && p.heads_per_cta <= 4 * kUnroll && ctas > 16 * sms)
    k_rotary<T, W, kAdjacent, W == 1><<<dim3(16 * sms, heads), kThreads, 0, st>>>(p);
  else
    k_rotary<T, W, kAdjacent, false><<<dim3((unsigned)ctas, heads), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch(Params& p, int pairing, int width, cudaStream_t st) {
  if (pairing == BSA_PAIR_ADJACENT) return run<T, 4, true>(p, st);
  if (width == 8) return run<T, 8, false>(p, st);
  if (width == 4) return run<T, 4, false>(p, st);
  if (width == 2) return run<T, 2, false>(p, st);
  return run<T, 1, false>(p, st);
}

}  // namespace rotary

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t st) {
  rotary::Params p;
  p.x = a.X;
  p.y = a.Y;
  p.xs = a.xs;
  p.ys = a.ys;
  p.pos = a.pos;
  p.Bt = a.Bt;
  p.H = a.H;
  p.L = a.L;
  p.n_axes = a.n_axes;
  p.pos_per_batch = a.pos_per_batch != 0;
  p.sign = a.inverse ? -1.f : 1.f;
  // the sections of d: one per axis, then the components that are copied
  int n = 0, begin = 0, rest = 0, width = 8;
  for (int i = 0; i < a.n_axes; ++i) rest += a.axis_dim[i];
  rest = a.d - rest;
  for (int i = 0; i <= a.n_axes; ++i) {
    const int dim = i < a.n_axes ? a.axis_dim[i] : rest;
    const int half = dim / 2;
    while (half % width != 0) width /= 2;
    for (int j = 0; j < half; ++j, ++n) {
      p.axis[n] = (uint8_t)(i < a.n_axes ? i : rotary::kCopy);
      p.rate[n] = i < a.n_axes ? pow(a.base, -2.0 * j / dim) / (2.0 * M_PI) : 0.0;
      const bool adj = a.pairing == BSA_PAIR_ADJACENT;
      p.lo[n] = (uint8_t)(begin + (adj ? 2 * j : j));
      p.hi[n] = (uint8_t)(begin + (adj ? 2 * j + 1 : j + half));
    }
    begin += dim;
  }
  if (n < rotary::kMaxPairs) p.axis[n] = 254;  // end of the table
  if (a.type == BSA_TYPE_BF16) return rotary::dispatch<__nv_bfloat16>(p, a.pairing, width, st);
  if (a.type == BSA_TYPE_FP16) return rotary::dispatch<__half>(p, a.pairing, width, st);
  return rotary::dispatch<float>(p, a.pairing, width, st);
}

}  // namespace bsa
