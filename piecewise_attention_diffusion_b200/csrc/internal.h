// Internal launcher interface between the C ABI (api.cu) and the kernels.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/bsattn.h"

namespace bsa {

struct Shape {
  int Bt, H, L, d, block;
  const int32_t* key_valid = nullptr;  // real tokens per block (device int32 [M]), or null
  int BH() const { return Bt * H; }
  int M() const { return L / block; }
};

// Workspace size of each call (bytes); 0 if none.
size_t precompute_workspace(const Shape& s);
size_t forward_workspace(const Shape& s);

cudaError_t launch_build_mask(const bsa_mask_desc& desc, int M, int32_t* row_ptr,
                              int32_t* col_idx, int64_t cap, int32_t* status,
                              cudaStream_t st);

cudaError_t launch_precompute(const Shape& s, const void* K, const void* V, float* kbar,
                              float* vsum, float* Hbar, float* Mnorm, float* Hblk,
                              void* ws, int32_t* status, cudaStream_t st);

// Routing workspace: the column sums of every 32-row segment of Q (fp32 [BH, L/32, d]).
size_t route_workspace(const Shape& s);

cudaError_t launch_route(const Shape& s, const void* Q, const float* kbar,
                         const float* Mnorm, int k_top, float lambda, float scale,
                         int32_t* row_ptr, int32_t* col_idx, float* scores, void* ws,
                         int32_t* status, cudaStream_t st);

struct ForwardArgs {
  Shape s;
  const void *Q, *K, *V;
  const int32_t *row_ptr, *col_idx;
  int64_t nnz_total;
  int csr_per_head;
  int mode;
  const float *kbar, *vsum, *Hbar;
  float scale;
  void* O;
  float* lse;
  void* ws;
  int32_t* status;
  uint64_t wait_ns = 0;  // limit of the attention kernel's bounded waits; 0: the default
};

// bsa_forward's arguments as one record (the scale as given; 0 is resolved at launch).
ForwardArgs forward_args(const void* Q, const void* K, const void* V, int Bt, int H, int L, int d,
                         int block, const int32_t* key_valid, const int32_t* row_ptr,
                         const int32_t* col_idx, int64_t nnz_total, int csr_per_head, int mode,
                         const float* kbar, const float* vsum, const float* Hbar, float scale,
                         void* O, float* lse, void* ws, int32_t* status);

// Host-side checks of bsa_forward's arguments, all but the workspace: shapes, pointers,
// alignment, list sizes, mode, scale. BSA_OK or the status to return.
bsa_status check_forward_args(const ForwardArgs& a);

// The scale a forward call uses: `scale`, or 1/sqrt(d) when it is 0.
float forward_scale(float scale, int d);

cudaError_t launch_forward(const ForwardArgs& a, cudaStream_t st);

// Tensor-core attention kernel (forward_tc.cu); `flag` is the validation result, the
// first word of the forward workspace.
size_t forward_tc_workspace(const Shape& s);
cudaError_t launch_forward_tc(const ForwardArgs& a, const int32_t* flag, cudaStream_t st);

// The attention kernel of the keep-or-drop and PISA modes at head dim 64
// (forward_pair.cu): kb16, vs16 [BH, Mp, d] and hb16 [BH, d, d] are the bf16 statistics
// (PISA only).
cudaError_t launch_forward_pair(const ForwardArgs& a, const int32_t* flag, const void* kb16,
                                const void* vs16, const void* hb16, int Mp, cudaStream_t st);

// The first 32-byte boundary of a workspace: callers give 16-byte aligned ones, the kernels'
// 32-byte stores want more. Sizes count kAlignSlack for it.
constexpr size_t kAlignSlack = 16;
inline float* align32(void* ws) {
  return reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(ws) + 31) & ~uintptr_t(31));
}

struct RotaryArgs {
  const void* X;
  bsa_strides xs;
  void* Y;
  bsa_strides ys;
  int type, Bt, H, L, d;
  const float* pos;
  int pos_per_batch, n_axes;
  const int32_t* axis_dim;
  double base;
  int pairing, inverse;
};
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t st);

struct LinearArgs {
  const void* X;
  bsa_strides xs;
  int x_heads;
  const void* W;
  int64_t w_row;
  const void* bias;
  int act;
  const void* gate;
  const void* R;
  bsa_strides rs;
  void* Y;
  bsa_strides ys;
  int y_heads, type, Bt, L, K, N;
  void* ws;
  int32_t* status;
  int gate_rows;         // set at launch: rows that share one gate vector
  uint64_t wait_ns = 0;  // limit of the kernels' bounded waits; 0: the default
};
size_t linear_workspace(int Bt, int L, int K, int N);
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t st);

struct CrossArgs {
  const void* Q;
  bsa_strides qs;
  const void* K;
  bsa_strides ks;
  const void* V;
  bsa_strides vs;
  int type, Bt, H, Hkv, Lq, Lk, d;
  const int32_t* key_len;
  const uint8_t* key_mask;
  float scale;
  void* O;
  bsa_strides os;
  float* lse;
  void* ws;
  int32_t* status;
  uint64_t wait_ns = 0;  // limit of the kernel's bounded waits; 0: the default
};
namespace cross {
// The kernel for few query rows (cross_few.cu): a key head's query heads times Lq at most
// kMostRows; kFewPerSm CTAs share an SM. The CTAs are shared as `shares` says (cross_share.cuh);
// each leaves a part for k_join.
constexpr int kMostRows = 4, kFewPerSm = 2, kFewWarps = 8;
// Keys per round of a CTA: what its run of keys is counted in.
constexpr int few_round(int d, int rows) { return kFewWarps * (256 / d) * (rows <= 2 ? 4 : 2); }
struct Shares;
cudaError_t run_few(const CrossArgs& a, const Shares& shares, float* part_o, float2* part_ml,
                    cudaStream_t st);
}  // namespace cross
size_t cross_workspace(int Bt, int H, int Hkv, int Lq, int Lk, int d);
cudaError_t launch_cross(const CrossArgs& a, cudaStream_t st);

}  // namespace bsa
