// bsa_cross_forward: attention of Lq queries over Lk keys of another sequence (an encoder's
// states) on the 5th-generation tensor cores (tcgen05 + TMEM + TMA), sm_100a.
//
//     o_t = sum_n p_tn v_n / l_t,  p_tn = e^{s q_t.k_n - m_t},  l_t = sum_n p_tn
// over the real keys n of the batch entry (the first key_len of them, and those whose
// key_mask byte is not 0), in one pass over the keys with a running maximum m and sum l per
// row, both fp32.
//
// k_cross: one persistent CTA per SM, 384 threads. A work item is 256 query rows of one head
// (and one run of key tiles, where the keys are split); its two tiles of 128 rows
// ("streams") share every K and V tile, and the softmax of one overlaps the tensor-core work
// of the other:
//   warps 0-3, 4-7  one softmax warpgroup per stream: thread r owns query row r (TMEM lane
//           r): scores to registers, row maximum, P = 2^(x - m) back to TMEM in 16 bits, O
//           rescaled only when the maximum grows by more than 2^8; then the epilogue, through a
//           staging buffer of each warp's own to TMA stores (3% faster at 16384 x 512 keys than
//           32-byte stores from registers, which touch 32 lines at a time);
//   warp 8  TMA producer of a ring of K and V tiles of 128 keys;
//   warp 9  MMA issuer: S(t) = Q K(t)^T, O += P(t) V(t) with P as the TMEM operand;
//   warp 11  clears the rows of V that key counts and masks exclude, so that what lies there
//           (infinities, NaN) meets no product;
//   warp 10 clears those rows of K where there is a key mask, so that their scores are 0, and
//           leaves the softmax a term per key, 0 or -inf, which is added to the scores: two keys
//           an instruction, where a select per score took three instructions a key (2 x 16 heads x
//           4101 queries x 4352 keys, a fifth masked: 287 us after idle time, 321 call after call,
//           whatever the scores; 325 after idle time with the select). To let the zeros through
//           and take their exponentials off the sum again took 278 us where the scores allowed
//           it, but what rounding left of them grew with the number of tiles: 2.7e-4 of a sum
//           after 256. Rows are cleared four at a time, a bit per row; row by row took 4% more.
// TMEM: S0 [0,128), S1 [128,256), O0 [256, 256 + D), O1 [256 + D, 256 + 2 D); P overlays S.
// Few rows: the keys are split into runs that separate items take; each leaves its O, m and l
// in the workspace, and k_join adds them in order. Query heads that share a key head are taken
// as one head of more rows where their strides allow it (always for one row; 8 x 40 heads of one
// query over 8 key heads x 8192 keys x 128: 54 us, a tile for each query head 285).
// Measured, bf16, K and V read once, out of L2: 40 heads x 16384 queries x 512 keys x 128 in
// 162 us after idle time, 1061 TFLOP/s, and in 191 us call after call, where the power limit holds
// the SMs at 1.54 GHz of 1.965; the tensor pipe is busy 53% of the cycles. What bounds it is the chain
// of one stream's step (scores, maximum, exponentials, P, products: about 2930 cycles for the two
// streams' 2048 cycles of products) and the turn from one item to the next: 2100 of the 13900
// cycles of an item of four steps, in which the first scores wait until the last P is taken and the
// softmax warps write O. (Cycles per item at 512, 1024 and 2048 keys: 13900, 26000, 49000.) It is
// not the exponentials' pipe (41%) nor memory.
// Every mbarrier wait is bounded; on a timeout the CTA drains, frees TMEM and reports
// BSA_ERR_TIMEOUT.
#include <algorithm>

#include "common.cuh"
#include "cross_share.cuh"
#include "forward_tiles.cuh"
#include "internal.h"
#include "sm100.cuh"
#include "types.cuh"

namespace bsa {
namespace cross {

using namespace sm100;

constexpr int kBQ = 128;  // query rows per stream
constexpr int kBK = 128;  // keys per tile
constexpr int kStreams = 2;
constexpr int kThreads = 384;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kClearKWarp = 10, kClearVWarp = 11;
static_assert(kClearKWarp == kMmaWarp + 1 && kClearVWarp == kThreads / 32 - 1, "the last two warps clear");
// register split as in the block attention: 128 x 88 + 256 x 208 = 384 x 168
constexpr int kRegsControl = 88, kRegsSoftmax = 208;
static_assert(128 * kRegsControl + 256 * kRegsSoftmax <= kThreads * 168, "register split");
constexpr float kRescaleLog2 = 8.0f;

struct Params {
  int Bt, H, share, Lq, Lk;  // share: query heads per key head
  int q_tiles;               // of 256 rows
  int splits, tiles_per_split;
  int n_items;
  int qb, qh, kb, kh, vb, vh;  // 0 where that stride is 0 (one copy for all)
  const int32_t* key_len;
  const uint8_t* key_mask;
  float scale_log2;
  float* lse;
  float* part_o;   // [splits, Bt H Lq, D]
  float2* part_ml; // [splits, Bt H Lq]: running maximum (base 2) and sum
  int32_t* status;
  uint64_t wait_ns;
};

template <int D>
struct Cfg {
  static constexpr int QBYTES = kBQ * D * 2;
  static constexpr int SLOT = kBK * D * 2;
  static constexpr int NK = D == 128 ? 2 : 4;  // slots of the K ring
  static constexpr int NV = D == 128 ? 2 : 4;  // and of the V ring
  static constexpr int OUT = 32 * 128;         // a warp's staging: 32 rows of 64 columns
  static constexpr int SMEM = kStreams * QBYTES + (NK + NV) * SLOT + 8 * OUT + 1024;
  __host__ __device__ static constexpr uint32_t S_COL(int x) { return 128u * x; }
  __host__ __device__ static constexpr uint32_t O_COL(int x) { return 256u + D * x; }
};

struct Item {
  int b, h, qt, split, len, t0, n;  // n key tiles from tile t0
  bool two;                         // the second stream has rows
};

__device__ __forceinline__ Item item_of(const Params& p, int i) {
  Item r;
  r.split = i % p.splits;
  i /= p.splits;
  r.qt = i % p.q_tiles;
  i /= p.q_tiles;
  r.h = i % p.H;
  r.b = i / p.H;
  r.len = p.key_len != nullptr ? min(max(__ldg(p.key_len + r.b), 0), p.Lk) : p.Lk;
  r.t0 = r.split * p.tiles_per_split;
  r.n = min(max(ceil_div(r.len, kBK) - r.t0, 0), p.tiles_per_split);
  r.two = r.qt * 2 * kBQ + kBQ < p.Lq;
  return r;
}

// Whether tile t of an item has keys that are not real.
__device__ __forceinline__ bool tile_masked(const Params& p, const Item& it, int t) {
  return p.key_mask != nullptr || (it.t0 + t + 1) * kBK > it.len;
}

// Of keys 4 lane .. 4 lane + 3 of tile t, those that are not real, a bit each.
__device__ __forceinline__ uint32_t excluded(const Params& p, const Item& it, int t, int lane) {
  uint32_t out = 0;
  if (t < it.n && tile_masked(p, it, t)) {
    const int key0 = (it.t0 + t) * kBK + 4 * lane;
    const uint8_t* mask = p.key_mask + (int64_t)it.b * p.Lk;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = key0 + j;
      const bool gone = key >= it.len || (p.key_mask != nullptr && __ldg(mask + key) == 0);
      out |= (gone ? 1u : 0u) << j;
    }
  }
  return out;
}

struct Barriers {
  uint64_t k_full[4], k_empty[4], k_clear[4], v_full[4], v_empty[4], v_clear[4];
  uint64_t q_full[kStreams];
  uint64_t s_full[kStreams], p_full[kStreams], p_half[kStreams];
  uint64_t o_final[kStreams], o_free[kStreams], q_empty[kStreams];
  uint64_t done;
};

// Row maximum that keeps NaN: three inputs at a time, four chains.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float row_max(const uint32_t (&r)[kBK]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < kBK; e += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m[j] = max3_nan(m[j], __uint_as_float(r[e + 2 * j]), __uint_as_float(r[e + 2 * j + 1]));
  return max3_nan(max3_nan(m[0], m[1], m[2]), m[3], m[3]);
}

// Coefficients of the degree-4 polynomial for 2^f on [-1/2, 1/2] of least maximum relative
// error (2.7e-6 with its coefficients rounded), from the Remez fit in exp2_poly_fit.py.
constexpr float kE0 = 0.9999993f, kE1 = 0.6931218f, kE2 = 0.24024744f, kE3 = 0.05591786f,
                kE4 = 0.009570102f;

// 2^x for a pair on the FMA pipe, x finite or -inf and <= 8: split as in ex2_poly2, whose
// degree 3 (7.5e-5) would show in the log-sum-exp. Below -126 the result is 2^-126.
__device__ __forceinline__ float2 ex2_poly4(float2 x) {
  constexpr float kShift = 12582912.0f;  // 1.5 * 2^23
  x.x = fmaxf(x.x, -126.0f);
  x.y = fmaxf(x.y, -126.0f);
  const float2 t = add2(x, make_float2(kShift, kShift));
  const float2 f = sub2(x, sub2(t, make_float2(kShift, kShift)));
  float2 q = fma2(f, make_float2(kE4, kE4), make_float2(kE3, kE3));
  q = fma2(q, f, make_float2(kE2, kE2));
  q = fma2(q, f, make_float2(kE1, kE1));
  q = fma2(q, f, make_float2(kE0, kE0));
  return make_float2(__uint_as_float(__float_as_uint(q.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(q.y) + (__float_as_uint(t.y) << 23)));
}

// Pairs of every 8 whose exponentials go to the FMA pipe, the rest to the special-function
// unit, which alone would need as long as the products (128 x 128 exponentials at 16 a cycle).
constexpr int kPolyOf8 = 2;

// P of one row: 2^(s * scale_log2 - m_ref), to TMEM in pairs of T at p_addr, arriving at `half`
// when the first 64 keys are there; returns the fp32 sum, of the weights before they are rounded.
// The rounding to T (2^-8 of a weight at most in bf16, 2^-11 in fp16, to nearest) is what the tensor
// core asks for, whose two operands have V's type. Against 64 bits an output is then off by 2.3e-3
// in bf16 (2.5e-4 in fp16), where 32-bit weights would give 1.7e-3 (2.1e-4), most of which is the
// output's own rounding; weights in two 16-bit parts would double the second product.
template <typename T, int kPoly>
__device__ __forceinline__ float row_exp(const uint32_t (&r)[kBK], float scale_log2, float m_ref,
                                         uint32_t p_addr, uint64_t* half) {
  const float2 sc = make_float2(scale_log2, scale_log2), nm = make_float2(-m_ref, -m_ref);
  float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                   make_float2(0.f, 0.f)};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
#pragma unroll
    for (int q = 0; q < 32; ++q) {
      const int e = h * 64 + 2 * q;
      const float2 x = fma2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), sc, nm);
      const float2 v = q % 8 < kPoly ? ex2_poly4(x) : make_float2(ex2(x.x), ex2(x.y));
      acc[q & 3] = add2(acc[q & 3], v);
      pk[q] = pack2<T>(v.x, v.y);
    }
    tmem_st32(p_addr + h * 32, pk);
    if (h == 0) {
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(half);
    }
  }
  const float2 a = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
  return a.x + a.y;
}

__device__ __forceinline__ void tma_store_5d(const CUtensorMap* map, const void* src, int x, int y,
                                             int z, int w, int v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5, %6}], [%1];"
      ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z), "r"(w),
      "r"(v)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar, int x,
                                            int y, int z, int w, int v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v),
      "r"(smem_u32(bar))
      : "memory");
}

// 32 bytes, aligned.
__device__ __forceinline__ void store8(void* dst, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// kKeyMask: key_mask is there, so that any tile may have keys that are not real; else only an
// item's last one has, behind the last real key.
template <typename T, int D, bool kKeyMask>
__global__ void __launch_bounds__(kThreads, 1)
k_cross(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
        const __grid_constant__ Params p) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sK = smem + kStreams * C::QBYTES;
  unsigned char* sV = sK + C::NK * C::SLOT;
  __shared__ Barriers bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  // With a key mask, of a tile of K: what is added to the scores (0, or -inf where a key is not
  // real), and how many keys are not real. The warp that clears K's rows writes them once the tile
  // is there: then the scores of the tile NK before it are computed, so that no softmax reads one
  // further back, and NK + 1 entries do.
  constexpr uint32_t kTermRing = kKeyMask ? C::NK + 1 : 1;
  __shared__ __align__(16) float term_sh[kTermRing][kBK];
  __shared__ uint32_t gone_sh[kTermRing];

  // k_join may take its place now; it waits for this grid before it reads a run
  if (p.splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    abort_sh = 0;
    for (int x = 0; x < kStreams; ++x) {
      mbar_init(&bars.q_full[x], 1);
      mbar_init(&bars.s_full[x], 1);
      mbar_init(&bars.p_full[x], 128);
      mbar_init(&bars.p_half[x], 128);
      mbar_init(&bars.o_final[x], 1);
      mbar_init(&bars.o_free[x], 128);
      mbar_init(&bars.q_empty[x], 1);
    }
    for (int i = 0; i < C::NK; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.k_clear[i], 32);
    }
    for (int i = 0; i < C::NV; ++i) {
      mbar_init(&bars.v_full[i], 1);
      mbar_init(&bars.v_empty[i], 1);
      mbar_init(&bars.v_clear[i], 32);
    }
    mbar_init(&bars.done, 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
    if (p.splits == 1) prefetch_tensormap(&tmO);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  volatile int* abort_flag = &abort_sh;
  const bool clearing = p.key_len != nullptr || p.key_mask != nullptr;

  if (warp >= kProducerWarp) {
    setmaxnreg_dec<kRegsControl>();
    if (warp == kProducerWarp) {
      // ------------------------------- TMA producer: K0, Q of both streams, V0, K1, V1, ...
      uint32_t nk = 0;  // tiles loaded so far, of K and of V
      uint32_t nq[kStreams] = {0, 0};
      bool ok = true;
      for (int i = blockIdx.x; i < p.n_items && ok; i += gridDim.x) {
        const Item it = item_of(p, i);
        const int hk = it.h / p.share;
        for (int t = 0; t < it.n && ok; ++t) {
          const int row = (it.t0 + t) * kBK;
          const int ks = nk % C::NK, vs = nk % C::NV;
          ok = mbar_wait_warp(&bars.k_empty[ks], ((nk / C::NK) & 1) ^ 1, abort_flag, p.wait_ns);
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&bars.k_full[ks], C::SLOT);
            tma_load_5d(sK + ks * C::SLOT, &tmK, &bars.k_full[ks], 0, row, 0, hk * p.kh, it.b * p.kb);
          }
          __syncwarp();
          // the item's queries, as soon as the last item's last scores are computed
#pragma unroll
          for (int x = 0; x < kStreams; ++x) {
            if (t > 0 || !ok || (x == 1 && !it.two)) break;
            ok = mbar_wait_warp(&bars.q_empty[x], (nq[x] & 1) ^ 1, abort_flag, p.wait_ns);
            if (!ok) break;
            if (elect_one()) {
              mbar_arrive_expect_tx(&bars.q_full[x], C::QBYTES);
              tma_load_5d(smem + x * C::QBYTES, &tmQ, &bars.q_full[x], 0,
                          it.qt * 2 * kBQ + x * kBQ, 0, it.h * p.qh, it.b * p.qb);
            }
            __syncwarp();
            ++nq[x];
          }
          ok = ok && mbar_wait_warp(&bars.v_empty[vs], ((nk / C::NV) & 1) ^ 1, abort_flag, p.wait_ns);
          ++nk;
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&bars.v_full[vs], C::SLOT);
            tma_load_5d(sV + vs * C::SLOT, &tmV, &bars.v_full[vs], 0, row, 0, hk * p.vh, it.b * p.vb);
          }
          __syncwarp();
        }
      }
      if (!ok) {
        // drain: wait (bounded, ignoring the abort flag) for copies still in flight
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t r = nk > (uint32_t)C::NK ? nk - C::NK : 0; r < nk; ++r)
          while (!mbar_try_wait(&bars.k_full[r % C::NK], (r / C::NK) & 1) &&
                 globaltimer_ns() - t0 < 100000000ull) {
          }
        for (uint32_t r = nk > (uint32_t)C::NV ? nk - C::NV : 0; r < nk; ++r)
          while (!mbar_try_wait(&bars.v_full[r % C::NV], (r / C::NV) & 1) &&
                 globaltimer_ns() - t0 < 100000000ull) {
          }
        for (int x = 0; x < kStreams; ++x)
          while (nq[x] > 0 && !mbar_try_wait(&bars.q_full[x], (nq[x] - 1) & 1) &&
                 globaltimer_ns() - t0 < 100000000ull) {
          }
        __syncwarp();
      }
    } else if (warp == kMmaWarp) {
      // -------------------------------------------------------------------- MMA issuer
      constexpr uint32_t fmt = is_bf16<T>() ? 1u : 0u;
      constexpr uint32_t ab = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(kBQ >> 4) << 24);
      constexpr uint32_t idesc_s = ab | ((uint32_t)(kBK >> 3) << 17);
      constexpr uint32_t idesc_o = ab | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // V is MN-major
      // a tile's descriptor is its address in 16-byte units in a constant pattern
      const uint64_t q_desc = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(smem_u32(sV), kBK * 128, 1024);
      uint32_t nk = 0, nv = 0;  // tiles taken so far
      int items[kStreams] = {0, 0};
      uint32_t p_count[kStreams] = {0, 0};
      bool ok = true;
      auto issue_s = [&](int x, uint32_t slot) {  // by the elected lane
        const uint64_t a0 = q_desc + (uint64_t)(x * (C::QBYTES >> 4));
        const uint64_t b0 = k_desc + (uint64_t)(slot * (C::SLOT >> 4));
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = (uint64_t)(((k / 4) * (kBQ * 128) + (k % 4) * 32) >> 4);
          mma_ss(tmem + C::S_COL(x), a0 + off, b0 + off, idesc_s, k > 0 ? 1u : 0u);
        }
        mma_commit(&bars.s_full[x]);
      };
      for (int i = blockIdx.x; i < p.n_items && ok; i += gridDim.x) {
        const Item it = item_of(p, i);
        if (it.n == 0) continue;
        const int ns = it.two ? 2 : 1;
        // the first scores: the last item's products, issued before, have taken P from where
        // these go; its epilogue still reads O
        ok = mbar_wait_warp(&bars.k_full[nk % C::NK], (nk / C::NK) & 1, abort_flag, p.wait_ns) &&
             (!kKeyMask || mbar_wait_warp(&bars.k_clear[nk % C::NK], (nk / C::NK) & 1, abort_flag,
                                          p.wait_ns));
#pragma unroll
        for (int x = 0; x < kStreams; ++x) {
          if (x >= ns || !ok) break;
          ok = mbar_wait_warp(&bars.q_full[x], items[x] & 1, abort_flag, p.wait_ns);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            issue_s(x, nk % C::NK);
            if (it.n == 1) mma_commit(&bars.q_empty[x]);
          }
          __syncwarp();
          ++items[x];
        }
        if (!ok) break;
        if (elect_one()) mma_commit(&bars.k_empty[nk % C::NK]);
        __syncwarp();
        ++nk;
        for (int t = 0; t < it.n && ok; ++t) {
          const bool more = t + 1 < it.n;
          const uint32_t vs = nv % C::NV, ks = nk % C::NK;
          const uint32_t v_par = (nv / C::NV) & 1, k_par = (nk / C::NK) & 1;
#pragma unroll
          for (int x = 0; x < kStreams; ++x) {
            if (x >= ns || !ok) break;
            // P of the first 64 keys is written; V(t) and K(t + 1), cleared of what is masked where
            // there are masks; the stream's last epilogue has read O. All are tested at once: a
            // test takes 107 cycles even of a barrier long complete. (Products from half of P on,
            // and this, took 16384 x 512 keys from 170 to 163 us.)
            const bool first = x == 0, o_wait = t == 0 && items[x] > 1;
            const uint32_t p_par = p_count[x] & 1, o_par = (items[x] - 2) & 1;
            bool ready = mbar_try_wait(&bars.p_half[x], p_par);
            if (first) ready &= mbar_try_wait(&bars.v_full[vs], v_par);
            if (first && clearing) ready &= mbar_try_wait(&bars.v_clear[vs], v_par);
            if (first && more) ready &= mbar_try_wait(&bars.k_full[ks], k_par);
            if (first && more && kKeyMask) ready &= mbar_try_wait(&bars.k_clear[ks], k_par);
            if (o_wait) ready &= mbar_try_wait(&bars.o_free[x], o_par);
            if (!__all_sync(0xffffffffu, ready))
              ok = (!first ||
                    (mbar_wait_warp(&bars.v_full[vs], v_par, abort_flag, p.wait_ns) &&
                     (!clearing ||
                      mbar_wait_warp(&bars.v_clear[vs], v_par, abort_flag, p.wait_ns)) &&
                     (!more || mbar_wait_warp(&bars.k_full[ks], k_par, abort_flag, p.wait_ns)) &&
                     (!more || !kKeyMask ||
                      mbar_wait_warp(&bars.k_clear[ks], k_par, abort_flag, p.wait_ns)))) &&
                   (!o_wait || mbar_wait_warp(&bars.o_free[x], o_par, abort_flag, p.wait_ns)) &&
                   mbar_wait_warp(&bars.p_half[x], p_par, abort_flag, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b0 = v_desc + (uint64_t)(vs * (C::SLOT >> 4));
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kBK / 32; ++k)  // the first half of P
                mma_ts(tmem + C::O_COL(x), tmem + C::S_COL(x) + k * 8, b0 + (uint64_t)(k * 128),
                       idesc_o, t > 0 || k > 0 ? 1u : 0u);
            }
            __syncwarp();
            ok = mbar_wait_warp(&bars.p_full[x], p_count[x] & 1, abort_flag, p.wait_ns);
            if (!ok) break;
            ++p_count[x];
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = kBK / 32; k < kBK / 16; ++k)
                mma_ts(tmem + C::O_COL(x), tmem + C::S_COL(x) + k * 8, b0 + (uint64_t)(k * 128),
                       idesc_o, t > 0 || k > 0 ? 1u : 0u);
              if (!more) mma_commit(&bars.o_final[x]);
              if (x + 1 == ns) mma_commit(&bars.v_empty[vs]);
              if (more) issue_s(x, ks);
              if (more && x + 1 == ns) mma_commit(&bars.k_empty[ks]);
              if (t + 2 == it.n) mma_commit(&bars.q_empty[x]);
            }
            __syncwarp();
          }
          if (!ok) break;
          ++nv;
          nk += more;
        }
      }
      // every issued MMA must complete before TMEM is released
      if (elect_one()) mma_commit(&bars.done);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&bars.done, 0) && globaltimer_ns() - t0 < 100000000ull) {
      }
      __syncwarp();
    } else {
      // --------------------------------- rows of K and of V that are not real keys (a warp each)
      // Every tile passes here, masked or not, so that a warp and its ring's barriers are never
      // more than one phase apart.
      const bool is_k = warp == kClearKWarp;
      const uint32_t ring = is_k ? C::NK : C::NV;
      uint64_t* full = is_k ? bars.k_full : bars.v_full;
      uint64_t* cleared = is_k ? bars.k_clear : bars.v_clear;
      uint32_t n = 0;
      bool ok = is_k ? kKeyMask : clearing;
      for (int i = blockIdx.x; i < p.n_items && ok; i += gridDim.x) {
        const Item it = item_of(p, i);
        uint32_t next = kKeyMask ? excluded(p, it, 0, lane) : 0;  // asked for a tile ahead
        if (!is_k && p.key_len != nullptr && lane == 0) {
          const int len = __ldg(p.key_len + it.b);
          if (len < 0 || len > p.Lk) report(p.status, BSA_ERR_BAD_PADDING);
        }
        for (int t = 0; t < it.n && ok; ++t, ++n) {
          const uint32_t out = next;
          if (kKeyMask) next = excluded(p, it, t + 1, lane);
          const uint32_t slot = n % ring;
          ok = mbar_wait_warp(&full[slot], (n / ring) & 1, abort_flag, p.wait_ns);
          if (!ok) break;
          if (kKeyMask && is_k) {  // for the softmax
            const uint32_t gone = __reduce_add_sync(0xffffffffu, __popc(out));
            auto term = [&](int j) { return (out >> j) & 1u ? -INFINITY : 0.f; };
            reinterpret_cast<float4*>(term_sh[n % kTermRing])[lane] =
                make_float4(term(0), term(1), term(2), term(3));
            if (lane == 0) gone_sh[n % kTermRing] = gone;
          }
          if (tile_masked(p, it, t)) {
            // A row is 128 bytes in each of the D / 64 sub-tiles. Eight lanes clear it, the warp
            // four rows at a time; rows behind the last key are zeros as they come.
            const int inside = min(kBK, p.Lk - (it.t0 + t) * kBK);
            uint32_t rows = 0;  // bit i: row 4 i + lane / 8
            if (!kKeyMask) {
              const int from = it.len - (it.t0 + t) * kBK;
              for (int i = 0; i < kBK / 4; ++i) {
                const int row = 4 * i + lane / 8;
                if (row >= from && row < inside) rows |= 1u << i;
              }
            } else {
              const int mine = max(0, min(4, inside - 4 * lane));
              const uint32_t there = out & ((1u << mine) - 1u);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t word = __ballot_sync(0xffffffffu, (there >> j) & 1u);
                if (lane / 8 == j) rows = word;
              }
            }
            unsigned char* at = (is_k ? sK : sV) + slot * C::SLOT + lane * 16;
#pragma unroll
            for (int i = 0; i < kBK / 4; ++i)
              if ((rows >> i) & 1u)
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                  *reinterpret_cast<uint4*>(at + h * (kBK * 128) + i * 512) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
          }
          mbar_arrive(&cleared[slot]);
        }
      }
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ------------------------------------------------------- softmax + epilogue (per stream)
    // P in fp16 is kept 2^7 times larger (at most 2^15, after the lazy rescale's 2^8), so that
    // keys up to 2^-31 below the row's largest still count
    constexpr float kLift = is_bf16<T>() ? 0.f : 7.f;
    const int x = warp / 4, quad = warp % 4;
    const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
    const uint32_t s_base = tmem + lane_addr + C::S_COL(x);
    const uint32_t o_base = tmem + lane_addr + C::O_COL(x);
    unsigned char* out = sV + C::NV * C::SLOT + warp * C::OUT;
    uint32_t tiles = 0, finals = 0, all = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < p.n_items; i += gridDim.x) {
      const Item it = item_of(p, i);
      const uint32_t first = all;  // of the item's tiles, in the count of the K ring
      all += it.n;
      if (x == 1 && !it.two) continue;
      float m_run = -INFINITY, l = 0.f;
      for (int t = 0; t < it.n; ++t) {
        ok = mbar_wait(&bars.s_full[x], tiles & 1, abort_flag, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++tiles;
        tc_fence_after();
        uint32_t r[kBK];
        tmem_ld32(s_base, *reinterpret_cast<uint32_t(*)[32]>(r));
        tmem_ld32(s_base + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
        tmem_ld32(s_base + 64, *reinterpret_cast<uint32_t(*)[32]>(r + 64));
        tmem_ld32(s_base + 96, *reinterpret_cast<uint32_t(*)[32]>(r + 96));
        tmem_wait_ld();
        const uint32_t entry = (first + t) % kTermRing;
        bool gone = false;
        if (!kKeyMask) {
          if (tile_masked(p, it, t)) {
            const int real = it.len - (it.t0 + t) * kBK;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int first = max(0, min(32, real - 32 * w));
              const uint32_t word = first == 32 ? 0u : 0xffffffffu << first;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if ((word >> e) & 1u) r[32 * w + e] = __float_as_uint(-INFINITY);
            }
          }
        } else {
          gone = gone_sh[entry] != 0;
          if (gone) {
            const float4* term = reinterpret_cast<const float4*>(term_sh[entry]);
#pragma unroll
            for (int e = 0; e < kBK; e += 4) {
              const float4 u = term[e / 4];
              const float2 a = add2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])),
                                    make_float2(u.x, u.y));
              const float2 b = add2(make_float2(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])),
                                    make_float2(u.z, u.w));
              r[e] = __float_as_uint(a.x);
              r[e + 1] = __float_as_uint(a.y);
              r[e + 2] = __float_as_uint(b.x);
              r[e + 3] = __float_as_uint(b.y);
            }
          }
        }
        float mx = row_max(r) * p.scale_log2;
        if (kKeyMask && gone && __any_sync(0xffffffffu, mx != mx)) {
          // a query that is not finite: its products with the zeros are NaN, and so the sums
#pragma unroll
          for (int e = 0; e < kBK; ++e)
            if (term_sh[entry][e] != 0.f) r[e] = __float_as_uint(-INFINITY);
          mx = row_max(r) * p.scale_log2;
        }
        const bool need = mx > m_run + kRescaleLog2;
        if (__any_sync(0xffffffffu, need)) {
          const float m_new = need ? mx : m_run;
          const float factor = need ? ex2(m_run - m_new) : 1.0f;
          if (t > 0) {
            // PV(t-1) was issued before S(t), so it has completed: rescale O in TMEM
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t ro[16];
              tmem_ld16(o_base + c, ro);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) ro[e] = __float_as_uint(__uint_as_float(ro[e]) * factor);
              tmem_st16(o_base + c, ro);
            }
          }
          l *= factor;
          m_run = m_new;
        }
        const float m_ref = m_run == -INFINITY ? 0.f : m_run - kLift;
        // NaN and +inf only come out right on the special-function unit
        const bool sfu = __any_sync(0xffffffffu, !(mx < INFINITY));
        if (sfu)
          l += row_exp<T, 0>(r, p.scale_log2, m_ref, s_base, &bars.p_half[x]);
        else
          l += row_exp<T, kPolyOf8>(r, p.scale_log2, m_ref, s_base, &bars.p_half[x]);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars.p_full[x]);
      }
      if (!ok) break;

      // ------------------------------------------------------------------ epilogue
      // (what a row without a real key has summed is what the polynomial makes of -inf)
      if (m_run == -INFINITY && l < 1.f) l = 0.f;
      const float inv_l = l == 0.f ? 0.f : 1.0f / l;  // no real key: zeros; NaN stays NaN
      const int row_w = it.qt * 2 * kBQ + x * kBQ + quad * 32, row_g = row_w + lane;
      const bool write = row_g < p.Lq;
      const int64_t row_of = ((int64_t)it.b * p.H + it.h) * p.Lq + row_g;
      if (it.n > 0) {
        ok = mbar_wait(&bars.o_final[x], finals++ & 1, abort_flag, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      if (p.splits > 1) {
        const int64_t at = (int64_t)it.split * p.Bt * p.H * p.Lq + row_of;
        if (write) p.part_ml[at] = make_float2(m_run - kLift, l);
#pragma unroll 1
        for (int c = 0; c < D && it.n > 0; c += 32) {
          uint32_t ro[32];
          tmem_ld32(o_base + c, ro);
          tmem_wait_ld();
          if (write)
#pragma unroll
            for (int e = 0; e < 32; e += 8) store8(p.part_o + at * D + c + e, ro + e);
        }
        tc_fence_before();
        if (it.n > 0) mbar_arrive(&bars.o_free[x]);
      } else {
#pragma unroll
        for (int c = 0; c < D; c += 64) {
          uint32_t ro[64] = {}, pk[32];
          if (it.n > 0) {
            tmem_ld32(o_base + c, *reinterpret_cast<uint32_t(*)[32]>(ro));
            tmem_ld32(o_base + c + 32, *reinterpret_cast<uint32_t(*)[32]>(ro + 32));
            tmem_wait_ld();
            if (c + 64 == D) {
              tc_fence_before();
              mbar_arrive(&bars.o_free[x]);
            }
          }
#pragma unroll
          for (int e = 0; e < 32; ++e)
            pk[e] = pack2<T>(__uint_as_float(ro[2 * e]) * inv_l,
                             __uint_as_float(ro[2 * e + 1]) * inv_l);
          // 32 rows of 64 columns, in the 128-byte swizzle of the store's box
          if (lane == 0) bulk_wait_read_all();  // the last store has read the buffer
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(out + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row_w < p.Lq) {  // rows past Lq are not written
            tma_store_5d(&tmO, out, 0, row_w, c / 64, it.h, it.b);
            bulk_commit_group();
          }
        }
        if (write && p.lse != nullptr)
          p.lse[row_of] = l == 0.f ? -INFINITY : (m_run - kLift + log2f(l)) * 0.69314718055994531f;
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && abort_sh) report(p.status, BSA_ERR_TIMEOUT);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct JoinParams {
  const float* part_o;
  const float2* part_ml;
  int64_t rows;
  int H, Lq;
  int parts;  // of every row; 0: as sh shares them
  Shares sh;
  bsa_strides os;
  float* lse;
};

// The parts of one row, joined in a fixed order: m = max m_i, o = sum 2^(m_i - m) o_i / l with
// l = sum 2^(m_i - m) l_i. W warps per row, each with its own run of parts, whose lanes take the
// parts' m and l, 32 at a time; eight parts of O are asked for together.
template <typename T, int D, int W>
__global__ void __launch_bounds__(128)
k_join(const __grid_constant__ JoinParams p, T* o) {
  constexpr int V = D / 32;
  __shared__ float acc_sh[W][D], l_sh[W];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, w = warp % W;
  const int64_t row = (int64_t)blockIdx.x * (4 / W) + warp / W;
  if (row >= p.rows) return;  // whole rows: W = 4 has one row per CTA
  const int t = (int)(row % p.Lq), h = (int)(row / p.Lq % p.H), b = (int)(row / p.Lq / p.H);
  const int parts = p.parts > 0 ? p.parts : ceil_div(p.sh.rounds(b), rounds_per_cta(p.sh));
  const int s1 = ceil_div(parts, W) * (w + 1), end = min(s1, parts);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float m = -INFINITY;
  for (int s = lane; s < parts; s += 32) {
    const float2 ml = p.part_ml[s * p.rows + row];
    if (ml.y != 0.f) m = fmaxf(m, ml.x);
  }
  m = warp_max(m);
  float acc[V] = {}, l = 0.f;
  for (int s0 = s1 - ceil_div(parts, W); s0 < end; s0 += 32) {
    float weight = 0.f;
    if (s0 + lane < end) {
      const float2 ml = p.part_ml[(s0 + lane) * p.rows + row];
      if (ml.y != 0.f) {
        weight = exp2f(ml.x - m);
        l += weight * ml.y;
      }
    }
    const int n = min(32, end - s0);
    for (int s = 0; s < n; s += 8) {
      Pack<float, V> part[8];
      float ws[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ws[j] = __shfl_sync(0xffffffffu, weight, s + j);
        if (ws[j] != 0.f)  // else there is no such part, or it has no real key and no O
          part[j] = *reinterpret_cast<const Pack<float, V>*>(
              p.part_o + ((s0 + s + j) * p.rows + row) * D + lane * V);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (ws[j] != 0.f)
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] += ws[j] * part[j].v[e];
    }
  }
  l = warp_sum(l);
  if constexpr (W > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) acc_sh[w][lane * V + e] = acc[e];
    if (lane == 0) l_sh[w] = l;
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int i = 1; i < W; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += acc_sh[i][lane * V + e];
      l += l_sh[i];
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  Pack<T, V> out;
#pragma unroll
  for (int e = 0; e < V; ++e) out.v[e] = from_f32<T>(acc[e] * inv);
  *reinterpret_cast<Pack<T, V>*>(o + b * p.os.batch + h * p.os.head + t * p.os.row + lane * V) = out;
  if (lane == 0 && p.lse != nullptr)
    p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ host side
// [Bt, H, L, D] as a 5-D map (64 columns, L, D / 64 column groups, H, Bt) with boxes of
// box_rows rows of box_groups column groups of one head: swizzled [box_rows x 64] sub-tiles,
// one behind the other.
template <typename T>
bool map_5d(CUtensorMap* m, const void* ptr, int D, int L, int H, int Bt, const bsa_strides& s,
            int box_rows, int box_groups) {
  fwdtiles::EncodeTiledFn enc = fwdtiles::encode_fn();
  if (!enc) return false;
  auto bytes = [](int64_t v) { return (cuuint64_t)(v > 0 ? v * 2 : 16); };
  cuuint64_t dims[5] = {64, (cuuint64_t)L, (cuuint64_t)(D / 64), (cuuint64_t)(s.head ? H : 1),
                        (cuuint64_t)(s.batch ? Bt : 1)};
  cuuint64_t strides[4] = {bytes(s.row), 128, bytes(s.head), bytes(s.batch)};
  cuuint32_t box[5] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_groups, 1, 1};
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(m, is_bf16<T>() ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
             const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call is run: by k_cross_few or k_cross; `parts` per row (1 of k_cross: it writes O), or
// (k_cross_few, ctas > 0) up to `parts`, as the key counts share `ctas` CTAs.
struct Plan {
  bool few;
  int parts, ctas;
};
// see plan_of; the bytes are those of a row's part in fp32, between d = 64 and 128
constexpr double kTileUs = 1.3, kItemUs = 2.5, kJoinUs = 4.0, kPartBytes = 400;
Plan plan_of(int Bt, int H, int Hkv, int Lq, int Lk) {
  const int sms = fwdtiles::sm_count();
  if (Lk > 0 && (int64_t)H / Hkv * Lq <= kMostRows) {
    const int64_t heads = (int64_t)Bt * Hkv, wave = (int64_t)kFewPerSm * sms;
    const int most = std::max(1, Lk / 256);  // 256 keys per CTA at least
    if (2 * heads <= wave && heads * ceil_div(Lk, 32) < 1 << 25) {
      const int ctas = (int)std::min(wave, 2 * heads * most);
      return Plan{true, std::min(ctas / Hkv, ceil_div(Lk, 32)), ctas};
    }
    // many heads: the runs per head that leave least of the last wave of CTAs empty
    Plan best{true, 1, 0};
    double cost = 1e300;
    for (int s = 1; s <= std::min<int64_t>(most, std::max<int64_t>(1, 4 * wave / heads)); ++s) {
      const double c = (double)((heads * s + wave - 1) / wave) / s + 1e-4 * s;
      if (c < cost) {
        cost = c;
        best.parts = s;
      }
    }
    return best;
  }
  // Runs of key tiles per row tile, four tiles each at least: those that make the SMs' longest
  // time least, in us from measured times of a tile, of an item beside its tiles, and of the join
  // of the parts (and their bytes, written and read). 6 x 16 heads x 28 queries x 5870 keys x 64,
  // masked: 75 us in 3 runs, 97 in one; 4 x 16 x 385 x 8741: one run, 109.
  const int64_t items = (int64_t)Bt * H * ceil_div(Lq, 2 * kBQ);
  const int tiles = std::max(1, ceil_div(Lk, kBK));
  const double joined = 2.0 * Bt * H * Lq * kPartBytes / 5e6;
  Plan best{false, 1, 0};
  double cost = 1e300;
  for (int s = 1; s <= std::max(1, tiles / 4) && s <= sms; ++s) {
    const int per = ceil_div(tiles, s);
    if (ceil_div(tiles, per) != s) continue;  // the same runs with a part less
    const double c = (double)((items * s + sms - 1) / sms) * (kTileUs * per + kItemUs) +
                     (s > 1 ? kJoinUs + s * joined : 0.0);
    if (c < cost) {
      cost = c;
      best.parts = s;
    }
  }
  return best;
}

Shares shares_of(const CrossArgs& a, const Plan& plan) {
  return Shares{a.key_len, a.Bt, a.Hkv, a.Lk, few_round(a.d, a.H / a.Hkv * a.Lq), plan.ctas, plan.parts};
}

template <typename T, int D>
cudaError_t join(const CrossArgs& a, const Plan& plan, const float* part_o, const float2* part_ml,
                 cudaStream_t st) {
  JoinParams p;
  p.part_o = part_o;
  p.part_ml = part_ml;
  p.rows = (int64_t)a.Bt * a.H * a.Lq;
  p.H = a.H;
  p.Lq = a.Lq;
  p.parts = plan.ctas > 0 ? 0 : plan.parts;
  p.sh = shares_of(a, plan);
  p.os = a.os;
  p.lse = a.lse;
  // four warps per row where the rows are too few to fill the SMs with a warp each
  const bool wide = p.rows <= 2048;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(wide ? p.rows : (p.rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, wide ? k_join<T, D, 4> : k_join<T, D, 1>, p, static_cast<T*>(a.O));
}

template <typename T, int D, bool kKeyMask>
cudaError_t run(const CrossArgs& a, cudaStream_t st) {
  using C = Cfg<D>;
  const Plan plan = plan_of(a.Bt, a.H, a.Hkv, a.Lq, a.Lk);
  const int64_t rows = (int64_t)a.Bt * a.H * a.Lq;
  float* part_o = align32(a.ws);
  float2* part_ml = reinterpret_cast<float2*>(part_o + plan.parts * rows * D);
  if (plan.few) {
    const cudaError_t e = run_few(a, shares_of(a, plan), part_o, part_ml, st);
    return e != cudaSuccess ? e : join<T, D>(a, plan, part_o, part_ml, st);
  }
  Params p;
  p.Bt = a.Bt;
  p.H = a.H;
  p.share = a.H / a.Hkv;
  p.Lq = a.Lq;
  p.Lk = a.Lk;
  p.q_tiles = ceil_div(a.Lq, 2 * kBQ);
  p.splits = plan.parts;
  p.tiles_per_split = ceil_div(std::max(ceil_div(a.Lk, kBK), 1), p.splits);
  p.n_items = a.Bt * a.H * p.q_tiles * p.splits;
  p.qb = a.qs.batch != 0;
  p.qh = a.qs.head != 0;
  p.kb = a.ks.batch != 0;
  p.kh = a.ks.head != 0;
  p.vb = a.vs.batch != 0;
  p.vh = a.vs.head != 0;
  p.key_len = a.key_len;
  p.key_mask = a.key_mask;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.lse = a.lse;
  p.part_o = part_o;
  p.part_ml = part_ml;
  p.status = a.status;
  p.wait_ns = a.wait_ns > 0 ? a.wait_ns : kWaitTimeoutNs;
  CUtensorMap tmQ, tmK, tmV, tmO;
  bool ok = map_5d<T>(&tmQ, a.Q, D, a.Lq, a.H, a.Bt, a.qs, kBQ, D / 64) &&
            map_5d<T>(&tmO, a.O, D, a.Lq, a.H, a.Bt, a.os, 32, 1);
  if (a.Lk > 0)
    ok = ok && map_5d<T>(&tmK, a.K, D, a.Lk, a.Hkv, a.Bt, a.ks, kBK, D / 64) &&
         map_5d<T>(&tmV, a.V, D, a.Lk, a.Hkv, a.Bt, a.vs, kBK, D / 64);
  else tmK = tmV = tmQ;  // no tile is loaded
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(k_cross<T, D, kKeyMask>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::SMEM);
  if (e != cudaSuccess) return e;
  // setmaxnreg.inc waits for registers that the launch must hold
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, k_cross<T, D, kKeyMask>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * kThreads < 128 * kRegsControl + 256 * kRegsSoftmax)
    return cudaErrorInvalidConfiguration;
  k_cross<T, D, kKeyMask><<<std::min(p.n_items, fwdtiles::sm_count()), kThreads, C::SMEM, st>>>(
      tmQ, tmK, tmV, tmO, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  return join<T, D>(a, plan, part_o, part_ml, st);
}

template <typename T>
cudaError_t by_shape(const CrossArgs& a, cudaStream_t st) {
  if (a.d == 64) return a.key_mask ? run<T, 64, true>(a, st) : run<T, 64, false>(a, st);
  return a.key_mask ? run<T, 128, true>(a, st) : run<T, 128, false>(a, st);
}

}  // namespace cross

// Where the query heads of a key head lie so that (head, row) steps evenly through both Q and O,
// they are taken as one head of H / Hkv * Lq rows: their tiles then read K and V once for all.
static bool folds(int H, int Hkv, int Lq, const bsa_strides& s) {
  return H > Hkv && s.head > 0 && s.head <= ((int64_t)1 << 38) / (H / Hkv) &&
         (int64_t)H / Hkv * Lq < 1 << 30 && (Lq == 1 || s.head == Lq * s.row);
}

static size_t workspace_of(int Bt, int H, int Hkv, int Lq, int Lk, int d) {
  const cross::Plan plan = cross::plan_of(Bt, H, Hkv, Lq, Lk);
  if (!plan.few && plan.parts == 1) return 0;
  const size_t rows = (size_t)Bt * H * Lq;
  return plan.parts * rows * (d + 2) * sizeof(float) + kAlignSlack;
}

size_t cross_workspace(int Bt, int H, int Hkv, int Lq, int Lk, int d) {
  // enough either way: the strides are not known here
  const int64_t rows = (int64_t)H / Hkv * Lq;
  const size_t plain = workspace_of(Bt, H, Hkv, Lq, Lk, d);
  return rows >= 1 << 30 ? plain : std::max(plain, workspace_of(Bt, Hkv, Hkv, (int)rows, Lk, d));
}

cudaError_t launch_cross(const CrossArgs& args, cudaStream_t st) {
  CrossArgs a = args;
  if (folds(a.H, a.Hkv, a.Lq, a.qs) && folds(a.H, a.Hkv, a.Lq, a.os)) {
    const int share = a.H / a.Hkv;
    for (bsa_strides* s : {&a.qs, &a.os}) {
      if (a.Lq == 1) s->row = s->head;
      s->head *= share;
    }
    a.Lq *= share;
    a.H = a.Hkv;
  }
  if (a.type == BSA_TYPE_BF16) return cross::by_shape<__nv_bfloat16>(a, st);
  return cross::by_shape<__half>(a, st);
}

}  // namespace bsa
