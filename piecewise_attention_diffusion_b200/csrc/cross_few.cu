// bsa_cross_forward for few query rows (a key head's query heads times Lq at most kMostRows):
// the keys and values are what is read, once, and there is too little work per key for the
// tensor cores' 128-row tiles. Plain fp32 arithmetic, bound by memory.
//
// A row of K is read by D / 8 lanes, 16 bytes each, so a warp holds 32 / (D / 8) keys at a time;
// a round is kAhead such groups, and the next round's are asked for before this one's are used.
// Each lane has its 8 components
// of every query row (scaled by s log2 e) and of every row's O; a score is a butterfly sum over
// the D / 8 lanes of a key, and every group of lanes keeps a running maximum and sum of its own
// for the keys it sees, so that nothing is exchanged between keys until the end: then the groups
// of a warp, and the warps through shared memory, are joined in a fixed order. A key that is not
// real is not read.
// The keys of a head are shared by CTAs whose parts k_join (cross.cu) adds in order. Each head
// gets CTAs in proportion to the real keys of its batch entry (cross_share.cuh; every CTA finds
// the same shares from the key counts), so that short entries leave no SM idle while a long one
// is read: 8 x 16 heads with 50 to 8192 keys of 8192 x 128 take 56 us, with as many CTAs for each head 99.
// 2 x 16 heads x 32768 keys x 64: 54 us with the join for 268 MB, 5.0 TB/s (the tensor-core kernel's
// split tiles: 92 us); one entry with half of them, 201 MB: 43.6 us; a fifth masked: 53 us (113).
#include "common.cuh"
#include "cross_share.cuh"
#include "internal.h"
#include "sm100.cuh"
#include "types.cuh"

namespace bsa {
namespace cross {

using sm100::ex2;

constexpr int kFewThreads = 32 * kFewWarps;

struct FewParams {
  const void *q, *k, *v;
  bsa_strides qs, ks, vs;
  int H, share, Lq;
  Shares sh;
  const uint8_t* key_mask;
  float scale_log2;
  float* part_o;
  float2* part_ml;
  int32_t* status;
  int64_t rows_all;  // Bt * H * Lq
};

// Maximum and weights of two parts: (m, wa, wb) with o = wa oa + wb ob. Parts that saw no key
// have m = -inf and weigh nothing.
__device__ __forceinline__ void join_two(float ma, float mb, float& m, float& wa, float& wb) {
  m = fmaxf(ma, mb);
  const float ref = m == -INFINITY ? 0.f : m;
  wa = ex2(ma - ref);
  wb = ex2(mb - ref);
}

template <typename T, int D, int G, int kAhead>
__global__ void __launch_bounds__(kFewThreads, kFewPerSm)
k_cross_few(const __grid_constant__ FewParams p) {
  constexpr int kLanes = D / 8, kKeys = 32 / kLanes;  // lanes per key, keys per warp at a time
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int c = lane % kLanes * 8, group = lane / kLanes;
  const int rows = p.share * p.Lq;  // <= G
  constexpr int kRound = kFewWarps * kKeys * kAhead;
  static_assert(kRound == few_round(D, G), "the host counts in the same rounds");
  __shared__ float o_sh[kFewWarps][G][D];
  __shared__ float2 ml_sh[kFewWarps][G];

  if (p.sh.key_len != nullptr && blockIdx.x == 0 && warp == 0)
    for (int i = lane; i < p.sh.Bt; i += 32)
      if (__ldg(p.sh.key_len + i) != p.sh.len(i)) report(p.status, BSA_ERR_BAD_PADDING);
  // this CTA's head, and its run of the head's keys, whole rounds of the CTA but at the end
  int b, hk, split, runs = p.sh.runs;
  if (p.sh.ctas == 0) {
    split = blockIdx.x % runs;
    hk = blockIdx.x / runs % p.sh.Hkv;
    b = blockIdx.x / runs / p.sh.Hkv;
  } else {
    const int per = rounds_per_cta(p.sh);
    int before = 0;  // CTAs of the entries before b
    for (b = 0;; b += 32) {
      runs = b + lane < p.sh.Bt ? ceil_div(p.sh.rounds(b + lane), per) : 0;
      int to = p.sh.Hkv * runs;
#pragma unroll
      for (int w = 1; w < 32; w *= 2) {
        const int left = __shfl_up_sync(0xffffffffu, to, w);
        if (lane >= w) to += left;
      }
      const uint32_t in = __ballot_sync(0xffffffffu, before + to > (int)blockIdx.x);
      if (in != 0) {
        const int at = __ffs(in) - 1;
        b += at;
        runs = __shfl_sync(0xffffffffu, runs, at);
        before += __shfl_sync(0xffffffffu, to, at) - p.sh.Hkv * runs;
        break;
      }
      before += __shfl_sync(0xffffffffu, to, 31);
      if (b + 32 >= p.sh.Bt) return;  // more CTAs than shares
    }
    hk = ((int)blockIdx.x - before) / runs;
    split = ((int)blockIdx.x - before) % runs;
  }
  const int len = p.sh.len(b);
  const int rounds = ceil_div(len, kRound);
  const int k0 = (rounds / runs * split + min(rounds % runs, split)) * kRound;
  const int k1 = min(len, k0 + (rounds / runs + (split < rounds % runs ? 1 : 0)) * kRound);

  float q[G][8], o[G][8], m[G], l[G];
#pragma unroll
  for (int r = 0; r < G; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) q[r][e] = o[r][e] = 0.f;
    if (r < rows) {
      const int h = hk * p.share + r / p.Lq, t = r % p.Lq;
      const uint4 u = *reinterpret_cast<const uint4*>(
          static_cast<const T*>(p.q) + b * p.qs.batch + h * p.qs.head + t * p.qs.row + c);
      unpack8<T>(u, q[r]);
#pragma unroll
      for (int e = 0; e < 8; ++e) q[r][e] *= p.scale_log2;
    }
  }
  const T* kp = static_cast<const T*>(p.k) + b * p.ks.batch + hk * p.ks.head + c;
  const T* vp = static_cast<const T*>(p.v) + b * p.vs.batch + hk * p.vs.head + c;
  const uint8_t* mask = p.key_mask + (int64_t)b * p.sh.Lk;

  uint4 ku[kAhead], vu[kAhead], kn[kAhead], vn[kAhead];
  bool real[kAhead], next[kAhead];
  auto fetch = [&](int key0) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int64_t key = (int64_t)key0 + a * kKeys + group;
      next[a] = key < k1 && (p.key_mask == nullptr || __ldg(mask + key) != 0);
      kn[a] = vn[a] = make_uint4(0u, 0u, 0u, 0u);
      if (next[a]) {
        kn[a] = __ldg(reinterpret_cast<const uint4*>(kp + key * p.ks.row));
        vn[a] = __ldg(reinterpret_cast<const uint4*>(vp + key * p.vs.row));
      }
    }
  };
  int key0 = k0 + warp * kAhead * kKeys;
  fetch(key0);
  for (; key0 < k1; key0 += kRound) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      ku[a] = kn[a];
      vu[a] = vn[a];
      real[a] = next[a];
    }
    fetch(key0 + kRound < k1 ? key0 + kRound : k1);
    float s[kAhead][G];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      float kf[8];
      unpack8<T>(ku[a], kf);
#pragma unroll
      for (int r = 0; r < G; ++r) {
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) d = fmaf(q[r][e], kf[e], d);
#pragma unroll
        for (int w = 1; w < kLanes; w *= 2) d += __shfl_xor_sync(0xffffffffu, d, w);
        s[a][r] = real[a] ? d : -INFINITY;
      }
    }
#pragma unroll
    for (int r = 0; r < G; ++r) {
      float mx = m[r];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) mx = fmaxf(mx, s[a][r]);
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float f = ex2(m[r] - ref);
      m[r] = mx;
      l[r] *= f;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[r][e] *= f;
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        s[a][r] = ex2(s[a][r] - ref);
        l[r] += s[a][r];
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      float vf[8];
      unpack8<T>(vu[a], vf);
#pragma unroll
      for (int r = 0; r < G; ++r)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[r][e] = fmaf(s[a][r], vf[e], o[r][e]);
    }
  }

  // the groups of the warp
#pragma unroll
  for (int w = kLanes; w < 32; w *= 2)
#pragma unroll
    for (int r = 0; r < G; ++r) {
      float mj, wa, wb;
      join_two(m[r], __shfl_xor_sync(0xffffffffu, m[r], w), mj, wa, wb);
      m[r] = mj;
      l[r] = wa * l[r] + wb * __shfl_xor_sync(0xffffffffu, l[r], w);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[r][e] = wa * o[r][e] + wb * __shfl_xor_sync(0xffffffffu, o[r][e], w);
    }
  // the warps
  if (lane < kLanes)
#pragma unroll
    for (int r = 0; r < G; ++r) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o_sh[warp][r][c + e] = o[r][e];
      if (lane == 0) ml_sh[warp][r] = make_float2(m[r], l[r]);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * D; i += kFewThreads) {
    const int r = i / D, d = i % D;
    float mx = -INFINITY, sum = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) mx = fmaxf(mx, ml_sh[w][r].x);
    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float f = ex2(ml_sh[w][r].x - ref);
      sum += f * o_sh[w][r][d];
      den += f * ml_sh[w][r].y;
    }
    const int h = hk * p.share + r / p.Lq, t = r % p.Lq;
    const int64_t at = (int64_t)split * p.rows_all + ((int64_t)b * p.H + h) * p.Lq + t;
    p.part_o[at * D + d] = sum;
    if (d == 0) p.part_ml[at] = make_float2(mx, den);
  }
}

template <typename T, int D, int G>
cudaError_t launch_few(int ctas, const FewParams& p, cudaStream_t st) {
  k_cross_few<T, D, G, G <= 2 ? 4 : 2><<<ctas, kFewThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t by_rows(int ctas, const FewParams& p, cudaStream_t st) {
  const int rows = p.share * p.Lq;
  if (rows <= 1) return launch_few<T, D, 1>(ctas, p, st);
  if (rows <= 2) return launch_few<T, D, 2>(ctas, p, st);
  return launch_few<T, D, 4>(ctas, p, st);
}

cudaError_t run_few(const CrossArgs& a, const Shares& shares, float* part_o, float2* part_ml,
                    cudaStream_t st) {
  FewParams p;
  p.q = a.Q;
  p.k = a.K;
  p.v = a.V;
  p.qs = a.qs;
  p.ks = a.ks;
  p.vs = a.vs;
  p.H = a.H;
  p.share = a.H / a.Hkv;
  p.Lq = a.Lq;
  p.sh = shares;
  p.key_mask = a.key_mask;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.part_o = part_o;
  p.part_ml = part_ml;
  p.status = a.status;
  p.rows_all = (int64_t)a.Bt * a.H * a.Lq;
  const int ctas = shares.ctas > 0 ? shares.ctas : a.Bt * a.Hkv * shares.runs;
  if (a.type == BSA_TYPE_BF16)
    return a.d == 64 ? by_rows<__nv_bfloat16, 64>(ctas, p, st) : by_rows<__nv_bfloat16, 128>(ctas, p, st);
  return a.d == 64 ? by_rows<__half, 64>(ctas, p, st) : by_rows<__half, 128>(ctas, p, st);
}

}  // namespace cross
}  // namespace bsa
