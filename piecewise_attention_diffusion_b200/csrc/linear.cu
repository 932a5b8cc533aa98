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
//              The residual comes by TMA into the warp's staging buffer while the products
//              run; then per chunk of 32 columns: accumulators to registers, bias, activation,
//              gate and residual in fp32, one rounding, back into the buffer, and a TMA store.
//              (Where strides rule TMA out: coalesced 2-byte accesses, 16 rows at a time.) Two
//              TMEM accumulators, so the epilogue of one tile runs under the products of the next.
// Measured out of L2, bf16: 16384 x 5120 x 5120 with bias, gate and residual 585 us after idle time
// and 690 call after call, where the power limit holds the SMs at 1.24 GHz of 1.965 (1.24-1.47
// PFLOP/s), the tensor pipe at 93%; 9216 x 1024 x 4096 with GELU (fp16) 66 and 78 us (1.4 GHz), the
// tensor pipe at 69%: a tile takes 11500 cycles, of which 8200 are products, as the epilogue's warps
// wait on one latency after the other; 23240 x 400 x 2560 with
// GELU (erf), gate and residual 109 us (177 with CUDA's erfcf); 2928 x 168 x 19968 with a residual
// 83 us where 16-byte loads of it by the lanes that own its rows took 126. Chunks are 32 columns
// because boxes of 64 (128-byte rows), stored once per tile, delay the operands' loads: 2.3% more
// time at K = 5120.
// Every mbarrier wait is bounded; on a timeout the pair drains, frees TMEM and reports
// BSA_ERR_TIMEOUT.
#include <algorithm>

#include "linear_common.cuh"
#include "sm100_pair.cuh"

namespace bsa {
namespace linear {

constexpr int kBM = 128;      // rows per CTA (256 per pair)
constexpr int kCW = 32;       // columns per epilogue chunk
constexpr int kRowGroup = 8;  // row tiles that a sweep over the columns shares (L2 reuse)

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
  static constexpr int OUT = 32 * COLS * 2;  // staging bytes per epilogue warp: its columns
  static constexpr int NSTAGE = BN == 256 ? 5 : BN == 128 ? 6 : 9;
  static constexpr uint32_t TMEM = 2 * BN;              // two accumulators
};

constexpr int kMaxStages = 9, kMaxEpilogue = 16;
struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t res_full[kMaxEpilogue];
  uint64_t done;
};
// What lies behind the stages and the staging buffers in shared memory.
template <typename T>
struct Small {
  T bias[kMaxEpilogue][kCW], gate[kMaxEpilogue][kCW];  // of a chunk
  Barriers bars;
  uint32_t tmem_base;
  int abort;
};
template <typename T, int BN>
constexpr int kSmem = Cfg<BN>::NSTAGE * Cfg<BN>::STAGE + Cfg<BN>::EPI * Cfg<BN>::OUT + (int)sizeof(Small<T>);

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
         const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmR,
         const __grid_constant__ Params<T> p) {
  using C = Cfg<BN>;
  // all of it, so that the base is the window's, with no room to spare for aligning it
  extern __shared__ __align__(1024) unsigned char smem[];
  if (smem_u32(smem) % 1024 != 0) {  // alike in both CTAs
    if (threadIdx.x == 0) report(p.status, BSA_ERR_CUDA);
    return;
  }
  Small<T>& small = *reinterpret_cast<Small<T>*>(smem + C::NSTAGE * C::STAGE + C::EPI * C::OUT);
  Barriers& bars = small.bars;
  int& abort_sh = small.abort;

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
    for (int i = 0; i < C::EPI; ++i) mbar_init(&bars.res_full[i], 1);
    mbar_init(&bars.done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&small.tmem_base, C::TMEM);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmW);
    if (p.tma_out) prefetch_tensormap(&tmY);
    if (p.tma_res) prefetch_tensormap(&tmR);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = small.tmem_base;
  volatile int* abort_flag = &abort_sh;
  const int group = blockIdx.x / 2, groups = gridDim.x / 2;
  // k_finish may take its place now; it waits for this grid before it reads a sum
  if (p.split) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    const uint32_t full0 = cluster_addr(&bars.full[0], 0);  // the leader's barriers
    WorkIter iter(p, group, groups);
    for (Work w; ok && iter.next(p, w);) {
      int m, n;
      tile_of(p, w.tile, m, n);
      const int b = m / p.row_tiles;
      const int row = (m % p.row_tiles) * 2 * kBM + (int)rank * kBM;
      const int wrow = n * BN + (int)rank * (BN / 2);
      int z = w.k0 / p.x_steps, x = w.k0 % p.x_steps;  // head and column step of X
      for (int k = w.k0; k < w.k1; ++k) {
        ok = mbar_wait_warp(&bars.empty[stage], phase ^ 1, abort_flag, p.wait_ns);
        if (!ok) break;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&bars.full[stage], 2 * C::STAGE);
          unsigned char* dst = smem + stage * C::STAGE;
          tma_load_4d_pair(dst, &tmX, full0 + stage * 8, x * kBK, row, z * p.xh, b * p.xb);
          tma_load_2d_pair(dst + C::A_BYTES, &tmW, full0 + stage * 8, k * kBK, wrow);
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
      // Drain. Both CTAs' copies report to the leader, which waits for those it expected; one
      // CTA may be ahead of the other by a few, which nobody expected: both leave them a
      // millisecond, and the cluster barrier at the end keeps both CTAs until then.
      const uint64_t t0 = globaltimer_ns();
      const uint32_t from = issued > (uint32_t)C::NSTAGE ? issued - C::NSTAGE : 0;
      for (uint32_t r = from; r < issued && rank == 0; ++r)
        while (!mbar_try_wait(&bars.full[r % C::NSTAGE], (r / C::NSTAGE) & 1) &&
               globaltimer_ns() - t0 < 100000000ull) {
        }
      while (globaltimer_ns() - t0 < 1000000ull) {
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      // D fp32; A and B both T, K-major; M = 256 over the pair
      constexpr uint32_t fmt = sizeof(T) == 2 && is_bf16<T>() ? 1u : 0u;
      constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(BN >> 3) << 17) |
                                 ((uint32_t)(2 * kBM >> 4) << 24);
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
            const uint64_t b0 = a0 + (C::A_BYTES >> 4);
#pragma unroll
            for (int j = 0; j < kBK / 16; ++j)
              mma_ss_pair(tmem + acc * BN, a0 + j * 2, b0 + j * 2, idesc, k > w.k0 || j > 0 ? 1u : 0u);
            mma_commit_pair(&bars.empty[stage]);
            if (k + 1 == w.k1) mma_commit_pair(&bars.acc_full[acc]);
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
        if (elect_one()) mma_commit_pair(&bars.done);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&bars.done, 0) && globaltimer_ns() - t0 < 100000000ull) {
        }
        __syncwarp();
      }
    }
  } else {
    // -------------------------------------------------------------------- epilogue
    const int e = warp - 2;
    const int quad = warp % 4;                     // TMEM lane quadrant of this warp
    const int part = e / 4;                        // its range of the columns
    unsigned char* out = smem + C::NSTAGE * C::STAGE + e * C::OUT;
    const uint32_t empty_addr[2] = {cluster_addr(&bars.acc_empty[0], 0),
                                    cluster_addr(&bars.acc_empty[1], 0)};
    // 16-byte piece g of row r of the staging buffer, which holds a chunk after the other, each of
    // 64-byte rows in that width's swizzle
    auto piece = [&](int r, int g) {
      return out + g / 4 * (32 * kCW * 2) + r * kCW * 2 + (g % 4 ^ ((r >> 1) & 3)) * 16;
    };
    auto staged = [&](int r, int col) {
      return reinterpret_cast<uint16_t*>(piece(r, col / 8) + col % 8 * 2);
    };
    bool ok = true;
    int it = 0;
    uint32_t residuals = 0;  // loaded by TMA
    WorkIter iter(p, group, groups);
    for (Work w; iter.next(p, w); ++it) {
      int m, n;
      tile_of(p, w.tile, m, n);
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
      const bool here = row0 < p.L && tile_col < p.N;  // this warp has outputs in this tile
      const bool whole = !partial(p, w);
      // a chunk's bias and (shared) gate, a column per lane, asked for a chunk ahead
      T bias_ahead, gate_ahead;
      auto fetch = [&](int col0) {
        const bool in = col0 + lane < p.N;
        bias_ahead = in && p.bias != nullptr ? p.bias[col0 + lane] : from_f32<T>(0.f);
        gate_ahead = in && p.gate != nullptr && one_gate ? gate[col0 + lane] : from_f32<T>(1.f);
      };
      if (whole && here) {
        fetch(tile_col);
        // R lands where Y is staged, and is replaced by it piece by piece
        if (lane == 0) bulk_wait_read_all();  // the last store has read the buffer
        __syncwarp();
        if (p.tma_res) {
          if (lane == 0) {
            const int head = tile_col / p.rv.cols;
            mbar_arrive_expect_tx(&bars.res_full[e], C::OUT);
            for (int c = 0; c < C::COLS; c += kCW)
              tma_load_4d(out + c * 64, &tmR, &bars.res_full[e], tile_col + c - head * p.rv.cols, row0,
                          head * p.rh, b * p.rb);
          }
          ++residuals;
        } else if (p.res != nullptr) {
          // a row at a time across the lanes (places past the end repeat the last)
#pragma unroll 1
          for (int c = 0; c < C::COLS && tile_col + c < p.N; c += kCW) {
            const int head = (tile_col + c) / p.rv.cols;
            const T* at = p.res + b * p.rv.batch + head * p.rv.head + row0 * p.rv.row +
                          (min(tile_col + c + lane, p.N - 1) - head * p.rv.cols);
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += 16) {
              uint16_t words[16];  // all asked for before the first is used
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                words[i] = __ldg(reinterpret_cast<const uint16_t*>(at));
                if (row0 + r0 + i + 1 < p.L) at += p.rv.row;
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) *staged(r0 + i, c + lane) = words[i];
            }
          }
          __syncwarp();
        }
      }
      ok = mbar_wait(&bars.acc_full[acc], (it / 2) & 1, abort_flag, p.wait_ns);
      if (whole && here && p.tma_res && ok)
        ok = mbar_wait(&bars.res_full[e], (residuals - 1) & 1, abort_flag, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < C::COLS; c += kCW) {
        const int col0 = tile_col + c;
        if (col0 >= p.N || !here) break;
        uint32_t r[kCW];
        tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16) + acc * BN + part * C::COLS + c, r);
        if (!whole) {  // a partial sum: 128 bytes of the slot's row
          tmem_wait_ld();
          float* at = slot_of(p, w, group, BN) +
                      (int64_t)(row - (m % p.row_tiles) * 2 * kBM) * BN + part * C::COLS + c;
          if (live)
#pragma unroll
            for (int i = 0; i < kCW; i += 8)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at + i),
                           "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]),
                           "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
                           : "memory");
          continue;
        }
        small.bias[e][lane] = bias_ahead;
        small.gate[e][lane] = gate_ahead;
        if (c + kCW < C::COLS && col0 + kCW < p.N) fetch(col0 + kCW);
        __syncwarp();
        tmem_wait_ld();
#pragma unroll
        for (int g = 0; g < kCW / 8; ++g) {
          const int col = col0 + g * 8;
          uint4* slot = reinterpret_cast<uint4*>(piece(lane, c / 8 + g));
          const uint4 bias8 = *reinterpret_cast<const uint4*>(&small.bias[e][g * 8]);
          const uint32_t biases[4] = {bias8.x, bias8.y, bias8.z, bias8.w};
          float2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = activate<kAct>(add2(make_float2(__uint_as_float(r[g * 8 + 2 * i]),
                                                   __uint_as_float(r[g * 8 + 2 * i + 1])),
                                       unpack2<T>(biases[i])));
          if (p.gate != nullptr) {
            if (one_gate) {
              const uint4 gate8 = *reinterpret_cast<const uint4*>(&small.gate[e][g * 8]);
              const uint32_t gates[4] = {gate8.x, gate8.y, gate8.z, gate8.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], unpack2<T>(gates[i]));
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                v[i] = mul2(v[i], make_float2(to_f32(gate[min(col + 2 * i, p.N - 1)]),
                                              to_f32(gate[min(col + 2 * i + 1, p.N - 1)])));
            }
          }
          if (p.res != nullptr) {
            const uint4 res8 = *slot;
            const uint32_t words[4] = {res8.x, res8.y, res8.z, res8.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = add2(v[i], unpack2<T>(words[i]));
          }
          *slot = make_uint4(pack2<T>(v[0].x, v[0].y), pack2<T>(v[1].x, v[1].y),
                             pack2<T>(v[2].x, v[2].y), pack2<T>(v[3].x, v[3].y));
        }
        if (p.tma_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int head = tile_col / p.yv.cols;
            tma_store_4d(&tmY, out + c * 64, col0 - head * p.yv.cols, row0, head, b);
            bulk_commit_group();
          }
        }
        __syncwarp();  // the next chunk's bias goes where this one's was
      }
      if (whole && here) {
        if (!p.tma_out) {
#pragma unroll 1
          for (int c = 0; c < C::COLS && tile_col + c < p.N; c += kCW) {
            const int head = (tile_col + c) / p.yv.cols;
            T* y = p.y + b * p.yv.batch + head * p.yv.head + row0 * p.yv.row +
                   (tile_col + c + lane - head * p.yv.cols);
            const bool in = tile_col + c + lane < p.N;
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += 16) {
              uint16_t words[16];  // all read before the first is stored
#pragma unroll
              for (int i = 0; i < 16; ++i) words[i] = *staged(r0 + i, c + lane);
#pragma unroll
              for (int i = 0; i < 16; ++i, y += p.yv.row)
                if (in && row0 + r0 + i < p.L) *reinterpret_cast<uint16_t*>(y) = words[i];
            }
          }
          fence_proxy_async_smem();  // R's next rows are written by TMA
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(empty_addr[acc]);
    }
    if (!ok && residuals > 0) {  // its copy lands before the CTA ends
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&bars.res_full[e], (residuals - 1) & 1) && globaltimer_ns() - t0 < 100000000ull) {
      }
      __syncwarp();
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

// The tiles whose sums several groups share: slots added in the order of the steps, then the
// same epilogue. A thread takes four columns of a row; tiles that one group summed whole are
// already written.
template <typename T, int kAct>
__global__ void __launch_bounds__(256)
k_finish(const Params<T> p, int few, int groups, int cols, int rows) {
  // the groups [g0, g1) that share this block's tile
  const int tile = blockIdx.x, units = p.m_tiles * p.n_tiles * p.k_steps;
  const int u0 = tile * p.k_steps, u1 = u0 + p.k_steps;
  int g0 = min((int)((int64_t)u0 * groups / units), groups - 1);
  while (first_unit(units, groups, g0) > u0) --g0;
  while (first_unit(units, groups, g0 + 1) <= u0) ++g0;
  int g1 = g0 + 1;
  while (first_unit(units, groups, g1) < u1) ++g1;
  int m, n;
  if (few) {
    n = tile / p.m_tiles;
    m = tile % p.m_tiles;
  } else {
    tile_of(p, tile, m, n);
  }
  const int id = blockIdx.y * 256 + threadIdx.x;
  const int r = id / (cols / 4), c = id % (cols / 4) * 4;
  const int b = m / p.row_tiles, row = (m % p.row_tiles) * rows + r, col = n * cols + c;
  const bool mine = g1 - g0 > 1 && r < p.part_rows && row < p.L && col < p.N;
  const int live = min(4, p.N - col);
  float bias[4] = {}, gate[4], res[4] = {};
  const T* at_gate = p.gate + (int64_t)((b * p.L + row) / p.gate_rows) * p.N + col;
  const int rhead = col / p.rv.cols, yhead = col / p.yv.cols;
  const T* at_res = p.res + b * p.rv.batch + rhead * p.rv.head + row * p.rv.row + (col - rhead * p.rv.cols);
  T* y = p.y + b * p.yv.batch + yhead * p.yv.head + row * p.yv.row + (col - yhead * p.yv.cols);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool in = mine && i < live;
    if (in && p.bias != nullptr) bias[i] = to_f32(p.bias[col + i]);
    gate[i] = in && p.gate != nullptr ? to_f32(at_gate[i]) : 1.f;
    if (in && p.res != nullptr) res[i] = to_f32(at_res[i]);
  }
  // every block waits, also one with nothing to add: this grid must not end before the one
  // that sums
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine) return;
  const float* at = p.part + ((int64_t)2 * g0 * p.part_rows + r) * cols + c;
  const int64_t slot = (int64_t)p.part_rows * cols;
  // the first group's slot is its second one (its run begins at or before the tile), a later
  // group's its first one, as slot_of has it
  float4 sum = *reinterpret_cast<const float4*>(at + slot);
#pragma unroll 4
  for (int g = 1; g < g1 - g0; ++g) {
    const float4 v = *reinterpret_cast<const float4*>(at + 2 * g * slot);
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float z = v[i] + bias[i];
    if (i < live)
      y[i] = from_f32<T>(activate<kAct>(make_float2(z, z)).x * gate[i] + res[i]);
  }
}

// ------------------------------------------------------------------ host side
template <typename T, int BN, int kAct>
cudaError_t run_pair(const LinearArgs& a, const Plan& plan, cudaStream_t st) {
  const Params<T> p = params_of<T>(a, plan);
  const int dx = a.K / a.x_heads, dy = a.N / a.y_heads;
  CUtensorMap tmX, tmW, tmY, tmR;
  bool ok = map_4d<T>(&tmX, a.X, dx, a.L, a.x_heads, a.Bt, a.xs, kBK, kBM) &&
            map_w<T>(&tmW, a.W, a.K, a.N, a.w_row, BN / 2);
  if (p.tma_out) ok = ok && map_4d<T>(&tmY, a.Y, dy, a.L, a.y_heads, a.Bt, a.ys, kCW, 32);
  else tmY = tmX;
  if (p.tma_res) ok = ok && map_4d<T>(&tmR, a.R, dy, a.L, a.y_heads, a.Bt, a.rs, kCW, 32);
  else tmR = tmX;
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(k_linear<T, BN, kAct>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<T, BN>);
  if (e != cudaSuccess) return e;
  k_linear<T, BN, kAct><<<2 * plan.groups, Cfg<BN>::THREADS, kSmem<T, BN>, st>>>(tmX, tmW, tmY, tmR, p);
  return cudaGetLastError();
}

template <typename T, int kAct>
cudaError_t run(const LinearArgs& a, const Plan& plan, cudaStream_t st) {
  cudaError_t e = plan.few           ? run_few<T>(a, plan, st)
                  : plan.cols == 256 ? run_pair<T, 256, kAct>(a, plan, st)
                  : plan.cols == 128 ? run_pair<T, 128, kAct>(a, plan, st)
                                     : run_pair<T, 64, kAct>(a, plan, st);
  if (e != cudaSuccess || !plan.split) return e;
  const Params<T> p = params_of<T>(a, plan);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.m_tiles * p.n_tiles),
                     (unsigned)ceil_div(p.part_rows * (plan.cols / 4), 256));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_finish<T, kAct>, p, (int)plan.few, plan.groups, plan.cols,
                            plan.rows);
}

template <typename T>
cudaError_t dispatch(const LinearArgs& a, cudaStream_t st) {
  const int k_steps = ceil_div(a.K / a.x_heads, kBK) * a.x_heads;
  const Plan plan = plan_of(a.Bt, a.L, k_steps, a.N);
  if (a.act == BSA_ACT_GELU_TANH) return run<T, BSA_ACT_GELU_TANH>(a, plan, st);
  if (a.act == BSA_ACT_GELU_ERF) return run<T, BSA_ACT_GELU_ERF>(a, plan, st);
  if (a.act == BSA_ACT_SILU) return run<T, BSA_ACT_SILU>(a, plan, st);
  return run<T, BSA_ACT_NONE>(a, plan, st);
}

// The plan of least estimated time, in microseconds. The constants were fitted to calls of 4 to
// 4096 rows, K 1024 to 10240 and N 1024 to 16384 (each plan timed on each size): a step of a
// tile, what a tile and a call cost besides, and for sums shared between groups the second
// kernel and its traffic per output. Whole tiles win where they fill the SMs (1024 x 1024 x
// 16384, 4 rows: 6.8 against 7.9), sharing where they do not (5120 x 5120, 4 rows: 13.1 against
// 20.9; 256 rows, K 10240, N 1024: 18 against 34) or where a last wave would be nearly empty
// and the output is small.
Plan plan_of(int Bt, int L, int k_steps, int N) {
  const int sms = fwdtiles::sm_count();
  Plan best{};
  double cost = 1e300;
  auto consider = [&](bool few, int rows, int cols, double call, double tile, double step) {
    const int most = few ? sms : sms / 2;
    const int64_t tiles = (int64_t)Bt * ceil_div(L, rows) * ceil_div(N, cols);
    const int whole = (int)std::min<int64_t>(tiles, most);
    const double c0 = call + (double)((tiles + whole - 1) / whole) * (k_steps * step + tile);
    if (c0 < cost) {
      cost = c0;
      best = Plan{few, cols, rows, whole, false};
    }
    // below 16 (6) steps per group the slots cost more than the SMs gained save
    const int64_t units = tiles * k_steps;
    const int shared = (int)std::min<int64_t>(most, units / (few ? 6 : 16));
    if (shared < 2 || tiles > 4 * most || units >= INT32_MAX) return;
    const double outputs = 1e-6 * Bt * L * N;
    const double c1 = call + tile + (double)units / shared * step +
                      (few ? 3.0 + 4.0 * outputs : 6.0 + 6.3 * outputs);
    if (c1 < cost) {
      cost = c1;
      best = Plan{few, cols, rows, shared, true};
    }
  };
  if (L <= 16) consider(true, 16, 128, 5.2, 0.4, 0.195);
  else if (L <= 32) consider(true, 32, 128, 5.5, 0.4, 0.20);
  else if (L <= 64) consider(true, 64, 128, 6.2, 0.4, 0.21);
  else if (L <= 128) consider(true, 128, 128, 8.0, 0.4, 0.224);
  consider(false, 256, 256, 6.2, 2.6, 0.285);
  consider(false, 256, 128, 6.0, 1.5, 0.185);
  consider(false, 256, 64, 6.0, 1.0, 0.165);
  return best;
}

}  // namespace linear

size_t linear_workspace(int Bt, int L, int K, int N) {
  const int k_steps = ceil_div(K, linear::kBK);
  const size_t apart = linear::plan_of(Bt, L, k_steps, N).workspace(L);
  const size_t merged = linear::plan_of(1, Bt * L, k_steps, N).workspace(Bt * L);
  return std::max(apart, merged);  // the strides say which; the larger serves both
}

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
