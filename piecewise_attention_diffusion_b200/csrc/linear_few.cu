// bsa_linear for few rows (at most 128 of an entry): the weight is what is read, once, so the
// roles of the operands are exchanged. Tiles are 128 rows of W (128 columns of Y) by all rows
// of X: D[n][m] = sum_k W[n][k] X[m][k], with W as the 128-row operand of tcgen05.mma and X as
// the narrow one (16, 32, 64 or 128 wide), so that no tensor work is spent on rows that are not
// there and a CTA's shared memory holds little but W.
//
// One CTA per SM; the CTAs share (tile, step) units evenly, so that all of them stream W to the
// end: a ring of 6 to 11 stages keeps up to 176 KB of W in flight per SM. Warp 0: TMA, warp 1:
// MMA, warps 2-5: epilogue. TMEM lane n holds column n of Y, so a warp writes 32 consecutive
// columns of a row at a time whatever Y's alignment. Bound by memory: W is N K values for 2 M N K
// operations.
#include "linear_common.cuh"

namespace bsa {
namespace linear {

constexpr int kCols = 128;
constexpr int kFewThreads = 192;

template <int R>
struct FewCfg {
  static constexpr int STAGE = kCols * 128 + R * 128;
  static constexpr int NSTAGE = R == 16 ? 11 : R == 32 ? 10 : R == 64 ? 8 : 6;
  static constexpr int SMEM = NSTAGE * STAGE + 1024;
  static constexpr uint32_t TMEM = 2 * R;
};

struct FewBarriers {
  uint64_t full[11], empty[11];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t done;
};

template <typename T, int R, int kAct>
__global__ void __launch_bounds__(kFewThreads, 1)
k_linear_few(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
             const __grid_constant__ Params<T> p) {
  using C = FewCfg<R>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ FewBarriers bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    abort_sh = 0;
    for (int i = 0; i < C::NSTAGE; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], 4);
    }
    mbar_init(&bars.done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, C::TMEM);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmW);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  volatile int* abort_flag = &abort_sh;
  const int group = blockIdx.x, groups = gridDim.x;
  // k_finish may take its place now; it waits for this grid before it reads a sum
  if (p.split) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    WorkIter iter(p, group, groups);
    for (Work w; ok && iter.next(p, w);) {
      const int n = w.tile / p.m_tiles, b = w.tile % p.m_tiles;
      int z = w.k0 / p.x_steps, x = w.k0 % p.x_steps;  // head and column step of X
      for (int k = w.k0; k < w.k1; ++k) {
        ok = mbar_wait_warp(&bars.empty[stage], phase ^ 1, abort_flag, p.wait_ns);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&bars.full[stage], C::STAGE);
          unsigned char* dst = smem + stage * C::STAGE;
          tma_load_2d(dst, &tmW, &bars.full[stage], k * kBK, n * kCols);
          tma_load_4d(dst + kCols * 128, &tmX, &bars.full[stage], x * kBK, 0, z * p.xh, b * p.xb);
        }
        __syncwarp();
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
    if (!ok) {
      // drain: wait (bounded, ignoring the abort flag) for copies still in flight
      const uint64_t t0 = globaltimer_ns();
      const uint32_t from = issued > (uint32_t)C::NSTAGE ? issued - C::NSTAGE : 0;
      for (uint32_t r = from; r < issued; ++r)
        while (!mbar_try_wait(&bars.full[r % C::NSTAGE], (r / C::NSTAGE) & 1) &&
               globaltimer_ns() - t0 < 100000000ull) {
        }
      __syncwarp();
    }
  } else if (warp == 1) {
    constexpr uint32_t fmt = is_bf16<T>() ? 1u : 0u;
    constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(R >> 3) << 17) |
                               ((uint32_t)(kCols >> 4) << 24);
    const uint64_t desc0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
    int stage = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true;
    WorkIter iter(p, group, groups);
    for (Work w; ok && iter.next(p, w); ++it) {
      const int acc = it & 1;
      if (it >= 2)
        ok = mbar_wait_warp(&bars.acc_empty[acc], (it / 2 - 1) & 1, abort_flag, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      for (int k = w.k0; k < w.k1; ++k) {
        ok = mbar_wait_warp(&bars.full[stage], phase, abort_flag, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a0 = desc0 + (uint64_t)(stage * (C::STAGE >> 4));
          const uint64_t b0 = a0 + (kCols * 128 >> 4);
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j)
            mma_ss(tmem + acc * R, a0 + j * 2, b0 + j * 2, idesc, k > w.k0 || j > 0 ? 1u : 0u);
          mma_commit(&bars.empty[stage]);
          if (k + 1 == w.k1) mma_commit(&bars.acc_full[acc]);
        }
        __syncwarp();
        if (++stage == C::NSTAGE) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      // the MMAs already issued end before TMEM is freed
      if (elect_one()) mma_commit(&bars.done);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&bars.done, 0) && globaltimer_ns() - t0 < 100000000ull) {
      }
      __syncwarp();
    }
  } else {
    const int quad = warp % 4;
    bool ok = true;
    int it = 0;
    WorkIter iter(p, group, groups);
    for (Work w; iter.next(p, w); ++it) {
      const int n = w.tile / p.m_tiles, b = w.tile % p.m_tiles;
      const int c = quad * 32 + lane, col = n * kCols + c;
      const int acc = it & 1;
      const bool whole = !partial(p, w), in = col < p.N;
      const float bias = whole && in && p.bias != nullptr ? to_f32(p.bias[col]) : 0.f;
      const int rhead = col / p.rv.cols, yhead = col / p.yv.cols;
      const T* at_res = p.res + b * p.rv.batch + rhead * p.rv.head + (col - rhead * p.rv.cols);
      T* y = p.y + b * p.yv.batch + yhead * p.yv.head + (col - yhead * p.yv.cols);
      float* part = whole ? nullptr : slot_of(p, w, group, kCols) + c;
      ok = mbar_wait(&bars.acc_full[acc], (it / 2) & 1, abort_flag, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int m0 = 0; m0 < R && m0 < p.L; m0 += 16) {
        // residuals and gates of 16 rows, all asked for before the first is used
        T res[16], gate[16];
        const bool use = whole && in;
        if (use && p.res != nullptr) {
          const T* at = at_res + m0 * p.rv.row;
#pragma unroll
          for (int i = 0; i < 16; ++i, at += p.rv.row)
            if (m0 + i < p.L) res[i] = *at;
        }
        if (use && p.gate != nullptr) {
          const int first = (b * p.L + m0) / p.gate_rows;
          const T* at = p.gate + (int64_t)first * p.N + col;
          int left = p.gate_rows - (b * p.L + m0 - first * p.gate_rows);  // rows of this vector
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (m0 + i < p.L) gate[i] = *at;
            if (--left == 0) {
              at += p.N;
              left = p.gate_rows;
            }
          }
        }
        uint32_t r[16];
        tmem_ld16(tmem + ((uint32_t)(quad * 32) << 16) + acc * R + m0, r);
        tmem_wait_ld();
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (m0 + i < p.L) part[(m0 + i) * kCols] = __uint_as_float(r[i]);
          continue;
        }
        if (!in) continue;
        T* at = y + m0 * p.yv.row;
#pragma unroll
        for (int i = 0; i < 16; ++i, at += p.yv.row) {
          if (m0 + i >= p.L) break;
          float z = __uint_as_float(r[i]) + bias;
          z = activate<kAct>(make_float2(z, z)).x;
          if (p.gate != nullptr) z *= to_f32(gate[i]);
          if (p.res != nullptr) z += to_f32(res[i]);
          *at = from_f32<T>(z);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.acc_empty[acc]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && abort_sh) report(p.status, BSA_ERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
}

template <typename T, int R, int kAct>
cudaError_t launch_few(const LinearArgs& a, const Plan& plan, cudaStream_t st) {
  using C = FewCfg<R>;
  const Params<T> p = params_of<T>(a, plan);
  CUtensorMap tmX, tmW;
  if (!map_4d<T>(&tmX, a.X, a.K / a.x_heads, a.L, a.x_heads, a.Bt, a.xs, kBK, R) ||
      !map_w<T>(&tmW, a.W, a.K, a.N, a.w_row, kCols))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(k_linear_few<T, R, kAct>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  k_linear_few<T, R, kAct><<<plan.groups, kFewThreads, C::SMEM, st>>>(tmX, tmW, p);
  return cudaGetLastError();
}

template <typename T, int kAct>
cudaError_t by_rows(const LinearArgs& a, const Plan& plan, cudaStream_t st) {
  if (plan.rows == 16) return launch_few<T, 16, kAct>(a, plan, st);
  if (plan.rows == 32) return launch_few<T, 32, kAct>(a, plan, st);
  if (plan.rows == 64) return launch_few<T, 64, kAct>(a, plan, st);
  return launch_few<T, 128, kAct>(a, plan, st);
}

template <typename T>
cudaError_t run_few(const LinearArgs& a, const Plan& plan, cudaStream_t st) {
  if (a.act == BSA_ACT_GELU_TANH) return by_rows<T, BSA_ACT_GELU_TANH>(a, plan, st);
  if (a.act == BSA_ACT_GELU_ERF) return by_rows<T, BSA_ACT_GELU_ERF>(a, plan, st);
  if (a.act == BSA_ACT_SILU) return by_rows<T, BSA_ACT_SILU>(a, plan, st);
  return by_rows<T, BSA_ACT_NONE>(a, plan, st);
}

template cudaError_t run_few<__nv_bfloat16>(const LinearArgs&, const Plan&, cudaStream_t);
template cudaError_t run_few<__half>(const LinearArgs&, const Plan&, cudaStream_t);

}  // namespace linear
}  // namespace bsa
