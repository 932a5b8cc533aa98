// bsa_linear: Y = R + g * act(X W^T + bias) on the 5th-generation tensor cores (tcgen05 +
// TMEM + TMA), sm_100a.
//
// X is read either as rows of K contiguous columns or head by head ([Bt, H, L, d], K = H d:
// the attention's output), and Y (and R) are addressed the same two ways ([Bt, H, L, d] is
// the layout the attention takes), so the projections around the attention need no copy.
//
// k_linear: one persistent CTA pair (cluster of two, tcgen05 cta_group::2) per two SMs,
// computing tiles of 256 rows x BN columns. Of every 64-deep step each CTA loads 128 rows of
// X and BN / 2 rows of W (both 128-byte swizzled) and the leader's MMA thread multiplies the
// pair's 256 x 64 by 64 x BN; each CTA accumulates its own 128 rows in its own TMEM. Sharing
// W over the pair halves the bytes of W that each SM reads per flop: 32 KB per 512 cycles of
// tensor work at BN = 256, where a CTA on its own would read 48 KB.
//   warp 0     TMA producer (each CTA its half; both report to the leader's barrier);
//   warp 1     MMA issuer (leader), TMEM allocation;
//   warps 2..  epilogue: up to four warps per TMEM lane quadrant, each with its own columns.
//              Per chunk of 32 columns: accumulators to registers, bias, activation,
//              gate and residual in fp32, one rounding, then through a swizzled staging
//              buffer to a TMA store (or coalesced 2-byte stores where Y's strides rule TMA
//              out). Two TMEM accumulators, so the epilogue of one tile runs under the
//              products of the next.
// Every mbarrier wait is bounded; on a timeout the pair drains, frees TMEM and reports
// BSA_ERR_TIMEOUT.
#include <algorithm>

#include "common.cuh"
#include "forward_tiles.cuh"
#include "internal.h"
#include "sm100_pair.cuh"
#include "types.cuh"

namespace bsa {
namespace linear {

using namespace sm100;

constexpr int kBM = 128;      // rows per CTA (256 per pair)
constexpr int kBK = 64;       // columns of X and W per step: one 128-byte swizzled row
constexpr int kCW = 32;        // columns per epilogue chunk: rows of 64 bytes in the staging buffer
constexpr int kRowGroup = 8;  // row tiles that a sweep over the columns shares (L2 reuse)

// What the epilogue needs of a [Bt, H, L, d] operand with H * d = N columns.
struct View {
  int64_t batch, head, row;
  int cols;  // d
};

template <typename T>
struct Params {
  int Bt, L, K, N;
  int gate_rows;        // rows of an entry that share one gate vector
  int x_steps;          // 64-column steps per head of X
  int xb, xh;           // 0 where X's batch or head stride is 0 (one copy for all)
  int k_steps, row_tiles, m_tiles, n_tiles;
  const T* bias;
  const T* gate;
  const T* res;
  T* y;
  View rv, yv;
  int tma_out;          // Y's base and strides allow TMA stores
  int vec_res;          // R's base and strides allow 16-byte loads
  int32_t* status;
  uint64_t wait_ns;
};

// z / (1 + 2^-w) for a pair
__device__ __forceinline__ float2 sigmoid_times(float2 z, float2 w) {
  return make_float2(__fdividef(z.x, 1.0f + ex2(-w.x)), __fdividef(z.y, 1.0f + ex2(-w.y)));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  return fma2(a, b, make_float2(-0.f, -0.f));
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
  if (kAct == BSA_ACT_GELU_ERF)  // the complementary form keeps the tail of negative z
    return make_float2(0.5f * z.x * erfcf(-0.70710678118654752f * z.x),
                       0.5f * z.y * erfcf(-0.70710678118654752f * z.y));
  if (kAct == BSA_ACT_SILU) return sigmoid_times(z, mul2(z, make_float2(kLog2e, kLog2e)));
  return z;
}

template <int BN>
struct Cfg {
  static constexpr int A_BYTES = kBM * 128;
  static constexpr int B_BYTES = BN / 2 * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  // epilogue warps: four (one per TMEM lane quadrant) for each of PARTS column ranges
  static constexpr int PARTS = BN / kCW < 4 ? BN / kCW : 4;
  static constexpr int COLS = BN / PARTS;
  static constexpr int EPI = 4 * PARTS;
  static constexpr int THREADS = 64 + 32 * EPI;
  static constexpr int OUT = 32 * kCW * 2;  // staging bytes per epilogue warp: one chunk
  static constexpr int NSTAGE = BN == 256 ? 5 : BN == 128 ? 6 : 9;
  static constexpr int SMEM = NSTAGE * STAGE + EPI * OUT + 1024;
  static constexpr uint32_t TMEM = 2 * BN;              // two accumulators
};

constexpr int kMaxStages = 9;
struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t done;
};

// Row and column tile of work item t: groups of kRowGroup row tiles, within a group column
// by column, so that the pairs at work at one time share both X's and W's tiles.
template <typename P>
__device__ __forceinline__ void tile_of(const P& p, int t, int& m, int& n) {
  const int per = kRowGroup * p.n_tiles;
  const int g = t / per, r = t % per;
  const int rows = min(kRowGroup, p.m_tiles - g * kRowGroup);
  m = g * kRowGroup + r % rows;
  n = r / rows;
}

template <typename T, int BN, int kAct>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<BN>::THREADS, 1)
k_linear(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
         const __grid_constant__ CUtensorMap tmY, const __grid_constant__ Params<T> p) {
  using C = Cfg<BN>;
  extern __shared__ unsigned char smem_raw[];
  // the same offset in both CTAs: the window's base is the same for the whole grid
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Barriers bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ __align__(16) float bias_sh[C::EPI][kCW], gate_sh[C::EPI][kCW];  // of a chunk

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    abort_sh = 0;
    for (int i = 0; i < C::NSTAGE; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], 2 * C::EPI);
    }
    mbar_init(&bars.done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_base_sh, C::TMEM);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmW);
    if (p.tma_out) prefetch_tensormap(&tmY);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  volatile int* abort_flag = &abort_sh;
  const int tiles = p.m_tiles * p.n_tiles;
  const int first = blockIdx.x / 2, step = gridDim.x / 2;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        int m, n;
        tile_of(p, t, m, n);
        const int b = m / p.row_tiles;
        const int row = (m % p.row_tiles) * 2 * kBM + (int)rank * kBM;
        const int wrow = n * BN + (int)rank * (BN / 2);
        int z = 0, x = 0;  // head and column of X at this step
        for (int k = 0; k < p.k_steps; ++k) {
          ok = mbar_wait(&bars.empty[stage], phase ^ 1, abort_flag, p.wait_ns);
          if (!ok) break;
          const uint32_t bar = cluster_addr(&bars.full[stage], 0);
          if (rank == 0) mbar_arrive_expect_tx(&bars.full[stage], 2 * C::STAGE);
          unsigned char* dst = smem + stage * C::STAGE;
          tma_load_4d_pair(dst, &tmX, bar, x * kBK, row, z * p.xh, b * p.xb);
          tma_load_2d_pair(dst + C::A_BYTES, &tmW, bar, k * kBK, wrow);
          ++issued;
          if (++x == p.x_steps) {
            x = 0;
            ++z;
          }
          if (++stage == C::NSTAGE) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // The peer's copies report to the leader, whose last waits below see them land; the
      // cluster barrier at the end keeps the peer until then.
      if (!ok && rank == 0) {
        const uint64_t t0 = globaltimer_ns();
        const uint32_t from = issued > (uint32_t)C::NSTAGE ? issued - C::NSTAGE : 0;
        for (uint32_t r = from; r < issued; ++r)
          while (!mbar_try_wait(&bars.full[r % C::NSTAGE], (r / C::NSTAGE) & 1) &&
                 globaltimer_ns() - t0 < 100000000ull) {
          }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank == 0) {
      // D fp32; A and B both T, K-major; M = 256 over the pair
      constexpr uint32_t fmt = sizeof(T) == 2 && is_bf16<T>() ? 1u : 0u;
      constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(BN >> 3) << 17) |
                                 ((uint32_t)(2 * kBM >> 4) << 24);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step, ++it) {
        const int acc = it & 1;
        if (it >= 2) ok = mbar_wait(&bars.acc_empty[acc], (it / 2 - 1) & 1, abort_flag, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        for (int k = 0; k < p.k_steps; ++k) {
          ok = mbar_wait(&bars.full[stage], phase, abort_flag, p.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint32_t addr = smem_u32(smem + stage * C::STAGE);
          const uint64_t a0 = smem_desc_sw128(addr, 16, 1024);
          const uint64_t b0 = smem_desc_sw128(addr + C::A_BYTES, 16, 1024);
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j)
            mma_ss_pair(tmem + acc * BN, a0 + j * 2, b0 + j * 2, idesc, (k | j) ? 1u : 0u);
          mma_commit_pair(&bars.empty[stage]);
          if (++stage == C::NSTAGE) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) mma_commit_pair(&bars.acc_full[acc]);
      }
      if (!ok) {
        // the MMAs already issued end before TMEM is freed
        mma_commit_pair(&bars.done);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&bars.done, 0) && globaltimer_ns() - t0 < 100000000ull) {
        }
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------------- epilogue
    const int e = warp - 2;
    const int quad = warp % 4;                     // TMEM lane quadrant of this warp
    const int part = e / 4;                        // its range of the columns
    unsigned char* out = smem + C::NSTAGE * C::STAGE + e * C::OUT;
    const uint32_t empty_addr[2] = {cluster_addr(&bars.acc_empty[0], 0),
                                    cluster_addr(&bars.acc_empty[1], 0)};
    bool ok = true;
    int it = 0;
    for (int t = first; t < tiles; t += step, ++it) {
      int m, n;
      tile_of(p, t, m, n);
      const int b = m / p.row_tiles;
      const int row0 = (m % p.row_tiles) * 2 * kBM + (int)rank * kBM + quad * 32;
      const int row = row0 + lane;
      const bool live = row < p.L;
      const int acc = it & 1;
      const int tile_col = n * BN + part * C::COLS;
      // gate vector of this row (entries merged into one run of rows have several)
      const int gate_of = p.gate != nullptr ? (b * p.L + min(row, p.L - 1)) / p.gate_rows : 0;
      const bool one_gate = __all_sync(0xffffffffu, gate_of == __shfl_sync(0xffffffffu, gate_of, 0));
      const T* gate = p.gate + (int64_t)gate_of * p.N;
      const T* res_row = p.res + b * p.rv.batch + row * p.rv.row;
      // what a chunk needs besides the accumulators: one column's bias and (shared) gate per
      // lane, and 32 columns of the row's residual; asked for a chunk ahead
      struct Ahead {
        T bias, gate;
        Pack<T, 8> res[kCW / 8];
      } ahead;
      auto fetch = [&](int col0) {
        const bool in = col0 + lane < p.N;
        ahead.bias = in && p.bias != nullptr ? p.bias[col0 + lane] : from_f32<T>(0.f);
        ahead.gate = in && p.gate != nullptr && one_gate ? gate[col0 + lane] : from_f32<T>(1.f);
      };
      auto fetch_res = [&](int col) -> Pack<T, 8> {
        const int head = col / p.rv.cols;
        return *reinterpret_cast<const Pack<T, 8>*>(res_row + head * p.rv.head +
                                                    (col - head * p.rv.cols));
      };
      const bool vec_res = p.vec_res && live;  // then 8 columns are all there or all not
      const bool rows_here = row0 < p.L;
      if (rows_here && tile_col < p.N) {
        fetch(tile_col);
#pragma unroll
        for (int g = 0; g < kCW / 8; ++g)
          if (vec_res && tile_col + g * 8 < p.N) ahead.res[g] = fetch_res(tile_col + g * 8);
      }
      ok = mbar_wait(&bars.acc_full[acc], (it / 2) & 1, abort_flag, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < C::COLS; c += kCW) {
        const int col0 = tile_col + c;
        if (col0 >= p.N || !rows_here) break;
        uint32_t r[kCW];
        tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16) + acc * BN + part * C::COLS + c, r);
        bias_sh[e][lane] = to_f32(ahead.bias);
        gate_sh[e][lane] = to_f32(ahead.gate);
        const bool more = c + kCW < C::COLS && col0 + kCW < p.N;
        if (more) fetch(col0 + kCW);
        if (lane == 0) bulk_wait_read_all();  // the staging buffer's last store has read it
        __syncwarp();
        if (p.res != nullptr && !p.vec_res) {
          // a residual that 16-byte loads cannot take comes through the staging buffer, a
          // row at a time across the lanes (places past the end repeat the last)
          const int head = col0 / p.rv.cols;
          const T* at = p.res + b * p.rv.batch + head * p.rv.head +
                        (min(col0 + lane, p.N - 1) - head * p.rv.cols);
#pragma unroll 8
          for (int rr = 0; rr < 32; ++rr)
            *reinterpret_cast<T*>(out + rr * kCW * 2 + ((lane / 8) ^ ((rr >> 1) & 3)) * 16 +
                                  lane % 8 * 2) = at[min(row0 + rr, p.L - 1) * p.rv.row];
          __syncwarp();
        }
        tmem_wait_ld();
#pragma unroll
        for (int g = 0; g < kCW / 8; ++g) {
          const int col = col0 + g * 8;
          // the 64-byte swizzle of the store's box: 16-byte piece g of row r sits at
          // g ^ (r / 2 % 4)
          Pack<T, 8>* slot = reinterpret_cast<Pack<T, 8>*>(out + lane * kCW * 2 +
                                                           (g ^ ((lane >> 1) & 3)) * 16);
          float2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = activate<kAct>(add2(make_float2(__uint_as_float(r[g * 8 + 2 * i]),
                                                   __uint_as_float(r[g * 8 + 2 * i + 1])),
                                       *reinterpret_cast<float2*>(&bias_sh[e][g * 8 + 2 * i])));
          if (p.gate != nullptr) {
            if (one_gate) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                v[i] = mul2(v[i], *reinterpret_cast<float2*>(&gate_sh[e][g * 8 + 2 * i]));
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                v[i] = mul2(v[i], make_float2(to_f32(gate[min(col + 2 * i, p.N - 1)]),
                                              to_f32(gate[min(col + 2 * i + 1, p.N - 1)])));
            }
          }
          if (p.res != nullptr) {
            const Pack<T, 8> w = p.vec_res ? ahead.res[g] : *slot;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[i] = add2(v[i], make_float2(to_f32(w.v[2 * i]), to_f32(w.v[2 * i + 1])));
            if (more && vec_res && col + kCW < p.N) ahead.res[g] = fetch_res(col + kCW);
          }
          Pack<T, 8> o;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o.v[2 * i] = from_f32<T>(v[i].x);
            o.v[2 * i + 1] = from_f32<T>(v[i].y);
          }
          *slot = o;
        }
        const int yhead = col0 / p.yv.cols, yc = col0 - yhead * p.yv.cols;
        if (p.tma_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_4d(&tmY, out, yc, row0, yhead, b);
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          T* y = p.y + b * p.yv.batch + yhead * p.yv.head + yc;
          if (col0 + lane < p.N)
            for (int rr = 0; rr < 32 && row0 + rr < p.L; ++rr)
              y[(row0 + rr) * p.yv.row + lane] = *reinterpret_cast<const T*>(
                  out + rr * kCW * 2 + ((lane / 8) ^ ((rr >> 1) & 3)) * 16 + lane % 8 * 2);
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(empty_addr[acc]);
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (threadIdx.x == 0 && abort_sh) report(p.status, BSA_ERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::TMEM);
  }
}

// ------------------------------------------------------------------ host side
// A [Bt][H][L][d] operand as a 4-D map with boxes of box_cols x box_rows.
template <typename T>
bool map_4d(CUtensorMap* m, const void* ptr, int d, int L, int H, int Bt, const bsa_strides& s,
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
bool map_w(CUtensorMap* m, const void* ptr, int K, int N, int64_t row, int box_rows) {
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

bool whole16(const void* ptr, const bsa_strides& s) {
  return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0 && s.batch % 8 == 0 && s.head % 8 == 0 &&
         s.row % 8 == 0;
}

template <typename T, int BN, int kAct>
cudaError_t run(const LinearArgs& a, cudaStream_t st) {
  using C = Cfg<BN>;
  Params<T> p;
  p.Bt = a.Bt;
  p.L = a.L;
  p.K = a.K;
  p.N = a.N;
  p.gate_rows = a.gate_rows;
  const int dx = a.K / a.x_heads, dy = a.N / a.y_heads;
  p.x_steps = ceil_div(dx, kBK);
  p.xb = a.xs.batch != 0;
  p.xh = a.xs.head != 0;
  p.k_steps = p.x_steps * a.x_heads;
  p.row_tiles = ceil_div(a.L, 2 * kBM);
  p.m_tiles = a.Bt * p.row_tiles;
  p.n_tiles = ceil_div(a.N, BN);
  p.bias = static_cast<const T*>(a.bias);
  p.gate = static_cast<const T*>(a.gate);
  p.res = static_cast<const T*>(a.R);
  p.y = static_cast<T*>(a.Y);
  p.rv = View{a.rs.batch, a.rs.head, a.rs.row, dy};
  p.yv = View{a.ys.batch, a.ys.head, a.ys.row, dy};
  p.tma_out = whole16(a.Y, a.ys);
  p.vec_res = a.R != nullptr && a.N % 8 == 0 && whole16(a.R, a.rs);
  p.status = a.status;
  p.wait_ns = kWaitTimeoutNs;
  CUtensorMap tmX, tmW, tmY;
  bool ok = map_4d<T>(&tmX, a.X, dx, a.L, a.x_heads, a.Bt, a.xs, kBK, kBM) &&
            map_w<T>(&tmW, a.W, a.K, a.N, a.w_row, BN / 2);
  if (p.tma_out) ok = ok && map_4d<T>(&tmY, a.Y, dy, a.L, a.y_heads, a.Bt, a.ys, kCW, 32);
  else tmY = tmX;
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(k_linear<T, BN, kAct>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
  const int pairs = (int)std::min<int64_t>(tiles, fwdtiles::sm_count() / 2);
  k_linear<T, BN, kAct><<<2 * pairs, C::THREADS, C::SMEM, st>>>(tmX, tmW, tmY, p);
  return cudaGetLastError();
}

template <typename T, int kAct>
cudaError_t by_width(const LinearArgs& a, cudaStream_t st) {
  const int pairs = fwdtiles::sm_count() / 2;
  const int64_t m = (int64_t)a.Bt * ceil_div(a.L, 2 * kBM);
  // the widest tile that still gives every pair of SMs one
  if (m * ceil_div(a.N, 256) >= pairs) return run<T, 256, kAct>(a, st);
  if (m * ceil_div(a.N, 128) >= pairs) return run<T, 128, kAct>(a, st);
  return run<T, 64, kAct>(a, st);
}

template <typename T>
cudaError_t dispatch(const LinearArgs& a, cudaStream_t st) {
  if (a.act == BSA_ACT_GELU_TANH) return by_width<T, BSA_ACT_GELU_TANH>(a, st);
  if (a.act == BSA_ACT_GELU_ERF) return by_width<T, BSA_ACT_GELU_ERF>(a, st);
  if (a.act == BSA_ACT_SILU) return by_width<T, BSA_ACT_SILU>(a, st);
  return by_width<T, BSA_ACT_NONE>(a, st);
}

}  // namespace linear

size_t linear_workspace(int, int, int, int) { return 0; }

cudaError_t launch_linear(const LinearArgs& in, cudaStream_t st) {
  LinearArgs a = in;
  // heads that lie next to one another are plain columns
  if (a.x_heads > 1 && a.xs.head == a.K / a.x_heads) {
    a.x_heads = 1;
    a.xs.head = 0;
  }
  auto flat = [&](const bsa_strides& s) { return a.L == 1 || s.batch == a.L * s.row; };
  a.gate_rows = a.L;
  // (a stride of 0 repeats X, whose rows then are not a run)
  if (a.Bt > 1 && a.xs.batch > 0 && flat(a.xs) && flat(a.ys) && (a.R == nullptr || flat(a.rs))) {
    // every entry's rows follow the last one's: one run of Bt * L rows
    auto merge = [&](bsa_strides& s) {
      if (a.L == 1) s.row = s.batch;
      s.batch = 0;
    };
    merge(a.xs);
    merge(a.ys);
    merge(a.rs);
    a.L *= a.Bt;
    a.Bt = 1;
  }
  return a.type == BSA_TYPE_BF16 ? linear::dispatch<__nv_bfloat16>(a, st)
                                 : linear::dispatch<__half>(a, st);
}

}  // namespace bsa
