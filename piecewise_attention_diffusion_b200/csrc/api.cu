// C ABI of libbsattn: host-side argument validation, then asynchronous launches on the
// caller's stream. No call allocates, frees or synchronises.
#include <stdint.h>

#include "../../include/bsattn.h"
#include "internal.h"

namespace {

using bsa::Shape;

constexpr int kMaxBlocks = 2048;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shape checks shared by precompute / route / forward.
bsa_status check_shape(const Shape& s) {
  if (s.Bt <= 0 || s.H <= 0 || s.L <= 0 || s.d <= 0 || s.block <= 0)
    return BSA_ERR_INVALID_ARG;
  if (s.d != 64 && s.d != 128) return BSA_ERR_UNSUPPORTED;
  if (s.block != 64 && s.block != 128) return BSA_ERR_UNSUPPORTED;
  if (s.L % s.block != 0) return BSA_ERR_UNSUPPORTED;
  if (s.M() > kMaxBlocks) return BSA_ERR_UNSUPPORTED;
  if ((int64_t)s.Bt * s.H * s.L * s.d >= (int64_t)1 << 40) return BSA_ERR_UNSUPPORTED;
  if ((int64_t)s.Bt * s.H > 65535) return BSA_ERR_UNSUPPORTED;  // grid.y limit
  if ((reinterpret_cast<uintptr_t>(s.key_valid) & 3u) != 0) return BSA_ERR_INVALID_ARG;
  return BSA_OK;
}

bsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA; }

bool workspace_ok(size_t need, const void* ws, size_t ws_bytes) {
  return need == 0 || (ws != nullptr && ws_bytes >= need && aligned16(ws));
}

int mask_blocks(const bsa_mask_desc* d) {
  if (d == nullptr) return -1;
  if (d->n_text_blocks < 0 || d->grid_h < 0 || d->grid_w < 0 || d->radius < 0 ||
      d->global_stride < 0)
    return -1;
  if ((d->grid_h == 0) != (d->grid_w == 0)) return -1;
  const int64_t m = (int64_t)d->n_text_blocks + (int64_t)d->grid_h * d->grid_w;
  if (m <= 0 || m > kMaxBlocks) return -1;
  return (int)m;
}

// The strides of a [Bt, H, L, d] tensor: as given, or contiguous where there are none. A
// dimension of size 1 is never stepped over, so its stride becomes 0.
bsa_strides strides_of(const bsa_strides* s, int Bt, int H, int L, int d) {
  bsa_strides r = s != nullptr ? *s : bsa_strides{(int64_t)H * L * d, (int64_t)L * d, d};
  if (Bt == 1) r.batch = 0;
  if (H == 1) r.head = 0;
  if (L == 1) r.row = 0;
  return r;
}

// Whole 16-byte steps, and no step or sum of steps that could pass 2^62 bytes.
bsa_status check_strides(const bsa_strides& s, int elem_bytes) {
  for (const int64_t v : {s.batch, s.head, s.row}) {
    if (v < 0 || v >= (int64_t)1 << 40) return BSA_ERR_INVALID_ARG;
    if (v * elem_bytes % 16 != 0) return BSA_ERR_UNSUPPORTED;
  }
  return BSA_OK;
}

// Rows, columns and tiles of a product are counted in 32 bits. (Sizes > 0.)
bool linear_sizes_fit(int Bt, int L, int K, int N) {
  return (int64_t)Bt * L < (int64_t)1 << 30 && K < 1 << 30 && N < 1 << 30 &&
         (((int64_t)L + 255) / 256 * Bt) * (((int64_t)N + 63) / 64) < INT32_MAX;
}

bsa_status check_cross(int Bt, int H, int Hkv, int Lq, int Lk, int d) {
  if (Bt <= 0 || H <= 0 || Hkv <= 0 || Lq <= 0 || Lk < 0) return BSA_ERR_INVALID_ARG;
  if (H % Hkv != 0) return BSA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return BSA_ERR_UNSUPPORTED;
  // rows, keys and work items are counted in 32 bits, with room for tiles past the end
  if ((int64_t)Bt * H >= (int64_t)1 << 24 || Lq >= 1 << 30 || Lk >= 1 << 30 ||
      (int64_t)Bt * H * (((int64_t)Lq + 255) / 256) >= (int64_t)1 << 22)
    return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}

}  // namespace

namespace bsa {

float forward_scale(float scale, int d) { return scale > 0.f ? scale : 1.0f / sqrtf((float)d); }

ForwardArgs forward_args(const void* Q, const void* K, const void* V, int Bt, int H, int L, int d,
                         int block, const int32_t* key_valid, const int32_t* row_ptr,
                         const int32_t* col_idx, int64_t nnz_total, int csr_per_head, int mode,
                         const float* kbar, const float* vsum, const float* Hbar, float scale,
                         void* O, float* lse, void* ws, int32_t* status) {
  ForwardArgs a;
  a.s = Shape{Bt, H, L, d, block, key_valid};
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.row_ptr = row_ptr;
  a.col_idx = col_idx;
  a.nnz_total = nnz_total;
  a.csr_per_head = csr_per_head;
  a.mode = mode;
  a.kbar = kbar;
  a.vsum = vsum;
  a.Hbar = Hbar;
  a.scale = scale;
  a.O = O;
  a.lse = lse;
  a.ws = ws;
  a.status = status;
  return a;
}

bsa_status check_forward_args(const ForwardArgs& a) {
  bsa_status r = check_shape(a.s);
  if (r != BSA_OK) return r;
  if (!a.Q || !a.K || !a.V || !a.O || !a.row_ptr) return BSA_ERR_INVALID_ARG;
  if (a.nnz_total < 0 || (a.nnz_total > 0 && a.col_idx == nullptr)) return BSA_ERR_INVALID_ARG;
  if (a.nnz_total >= INT32_MAX) return BSA_ERR_UNSUPPORTED;
  if (!aligned16(a.Q) || !aligned16(a.K) || !aligned16(a.V) || !aligned16(a.O))
    return BSA_ERR_INVALID_ARG;
  if (a.csr_per_head != 0 && a.csr_per_head != 1) return BSA_ERR_INVALID_ARG;
  if (a.mode != BSA_MODE_KEEP_OR_DROP && a.mode != BSA_MODE_PISA &&
      a.mode != BSA_MODE_PISA_BLOCK)
    return BSA_ERR_INVALID_ARG;
  if (a.mode == BSA_MODE_PISA && (!a.kbar || !a.vsum || !a.Hbar)) return BSA_ERR_INVALID_ARG;
  if (!(a.scale >= 0.f)) return BSA_ERR_INVALID_ARG;
  return BSA_OK;
}

}  // namespace bsa

extern "C" {

int32_t bsa_version(void) { return 200; }

const char* bsa_status_string(int32_t code) {
  switch (code) {
    case BSA_OK: return "BSA_OK";
    case BSA_ERR_INVALID_ARG: return "BSA_ERR_INVALID_ARG";
    case BSA_ERR_UNSUPPORTED: return "BSA_ERR_UNSUPPORTED";
    case BSA_ERR_CUDA: return "BSA_ERR_CUDA";
    case BSA_ERR_BAD_CSR: return "BSA_ERR_BAD_CSR";
    case BSA_ERR_TIMEOUT: return "BSA_ERR_TIMEOUT";
    case BSA_ERR_WORKSPACE: return "BSA_ERR_WORKSPACE";
    case BSA_ERR_CAPACITY: return "BSA_ERR_CAPACITY";
    case BSA_ERR_SCRATCH_LIMIT: return "BSA_ERR_SCRATCH_LIMIT";
    case BSA_ERR_BAD_PADDING: return "BSA_ERR_BAD_PADDING";
    default: return "BSA_UNKNOWN_STATUS";
  }
}

int32_t bsa_mask_blocks(const bsa_mask_desc* desc) { return mask_blocks(desc); }

size_t bsa_workspace_bytes(int32_t call, int32_t Bt, int32_t H, int32_t L, int32_t d,
                           int32_t block) {
  const Shape s{Bt, H, L, d, block};
  if (call == BSA_CALL_BUILD_MASK) return 0;
  if (check_shape(s) != BSA_OK) return 0;
  if (call == BSA_CALL_PRECOMPUTE) return bsa::precompute_workspace(s);
  if (call == BSA_CALL_ROUTE) return bsa::route_workspace(s);
  if (call == BSA_CALL_FORWARD) return bsa::forward_workspace(s);
  return 0;
}

bsa_status bsa_build_mask(const bsa_mask_desc* desc, int32_t* row_ptr, int32_t* col_idx,
                          int64_t col_capacity, int32_t* status, void* stream) {
  const int M = mask_blocks(desc);
  if (M < 0) return BSA_ERR_INVALID_ARG;
  if (row_ptr == nullptr || col_idx == nullptr || col_capacity < 0) return BSA_ERR_INVALID_ARG;
  return from_cuda(bsa::launch_build_mask(*desc, M, row_ptr, col_idx, col_capacity, status,
                                          static_cast<cudaStream_t>(stream)));
}

bsa_status bsa_precompute(const void* K, const void* V, int32_t Bt, int32_t H, int32_t L,
                          int32_t d, int32_t block, const int32_t* key_valid, float* kbar,
                          float* vsum, float* Hbar, float* Mnorm, float* Hblk,
                          void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  const Shape s{Bt, H, L, d, block, key_valid};
  bsa_status r = check_shape(s);
  if (r != BSA_OK) return r;
  if (!K || !V || !kbar || !vsum || !Hbar || !Mnorm) return BSA_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V)) return BSA_ERR_INVALID_ARG;
  if (!workspace_ok(bsa::precompute_workspace(s), workspace, ws_bytes)) return BSA_ERR_WORKSPACE;
  return from_cuda(bsa::launch_precompute(s, K, V, kbar, vsum, Hbar, Mnorm, Hblk, workspace,
                                          status, static_cast<cudaStream_t>(stream)));
}

bsa_status bsa_route(const void* Q, const float* kbar, const float* Mnorm, int32_t Bt,
                     int32_t H, int32_t L, int32_t d, int32_t block, const int32_t* key_valid,
                     int32_t k_top, float lambda, float scale, int32_t* row_ptr,
                     int32_t* col_idx, float* scores, void* workspace, size_t ws_bytes,
                     int32_t* status, void* stream) {
  const Shape s{Bt, H, L, d, block, key_valid};
  bsa_status r = check_shape(s);
  if (r != BSA_OK) return r;
  if (!Q || !kbar || !Mnorm || !row_ptr || !col_idx) return BSA_ERR_INVALID_ARG;
  if (!aligned16(Q)) return BSA_ERR_INVALID_ARG;
  if (k_top < 1 || k_top > s.M()) return BSA_ERR_INVALID_ARG;
  if ((int64_t)s.BH() * s.M() * k_top >= INT32_MAX) return BSA_ERR_UNSUPPORTED;
  if (!(lambda >= 0.f) || !(scale >= 0.f)) return BSA_ERR_INVALID_ARG;
  if (!workspace_ok(bsa::route_workspace(s), workspace, ws_bytes)) return BSA_ERR_WORKSPACE;
  const float sc = bsa::forward_scale(scale, d);
  return from_cuda(bsa::launch_route(s, Q, kbar, Mnorm, k_top, lambda, sc, row_ptr, col_idx,
                                     scores, workspace, status,
                                     static_cast<cudaStream_t>(stream)));
}

bsa_status bsa_forward(const void* Q, const void* K, const void* V, int32_t Bt, int32_t H,
                       int32_t L, int32_t d, int32_t block, const int32_t* key_valid,
                       const int32_t* row_ptr,
                       const int32_t* col_idx, int64_t nnz_total, int32_t csr_per_head,
                       int32_t mode, const float* kbar, const float* vsum,
                       const float* Hbar, float scale, void* O, float* lse,
                       void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  const bsa::ForwardArgs a = bsa::forward_args(Q, K, V, Bt, H, L, d, block, key_valid, row_ptr,
                                               col_idx, nnz_total, csr_per_head, mode, kbar,
                                               vsum, Hbar, scale, O, lse, workspace, status);
  const bsa_status r = bsa::check_forward_args(a);
  if (r != BSA_OK) return r;
  if (!workspace_ok(bsa::forward_workspace(a.s), workspace, ws_bytes)) return BSA_ERR_WORKSPACE;
  return from_cuda(bsa::launch_forward(a, static_cast<cudaStream_t>(stream)));
}

bsa_status bsa_selftest_forward_timeout(const void* Q, const void* K, const void* V, int32_t Bt,
                                        int32_t H, int32_t L, int32_t d, int32_t block,
                                        const int32_t* row_ptr, const int32_t* col_idx,
                                        int64_t nnz_total, int32_t mode, const float* kbar,
                                        const float* vsum, const float* Hbar, void* O,
                                        void* workspace, size_t ws_bytes, int64_t wait_ns,
                                        int32_t* status, void* stream) {
  if (status == nullptr || wait_ns < 1 || wait_ns > 10000000000ll) return BSA_ERR_INVALID_ARG;
  bsa::ForwardArgs a = bsa::forward_args(Q, K, V, Bt, H, L, d, block, nullptr, row_ptr, col_idx,
                                         nnz_total, 1, mode, kbar, vsum, Hbar, 0.f, O, nullptr,
                                         workspace, status);
  const bsa_status r = bsa::check_forward_args(a);
  if (r != BSA_OK) return r;
  if (!workspace_ok(bsa::forward_workspace(a.s), workspace, ws_bytes)) return BSA_ERR_WORKSPACE;
  a.wait_ns = static_cast<uint64_t>(wait_ns);
  return from_cuda(bsa::launch_forward(a, static_cast<cudaStream_t>(stream)));
}

bsa_status bsa_rotary(const void* X, const bsa_strides* xs, void* Y, const bsa_strides* ys,
                      int32_t type, int32_t Bt, int32_t H, int32_t L, int32_t d,
                      const float* pos, int32_t pos_per_batch, int32_t n_axes,
                      const int32_t* axis_dim, double base, int32_t pairing, int32_t inverse,
                      void* stream) {
  if (!X || !Y || !pos || !axis_dim) return BSA_ERR_INVALID_ARG;
  if (Bt <= 0 || H <= 0 || L <= 0 || d <= 0) return BSA_ERR_INVALID_ARG;
  if (type != BSA_TYPE_BF16 && type != BSA_TYPE_FP16 && type != BSA_TYPE_FP32)
    return BSA_ERR_INVALID_ARG;
  if (pairing != BSA_PAIR_ADJACENT && pairing != BSA_PAIR_HALVES) return BSA_ERR_INVALID_ARG;
  if (n_axes < 1 || n_axes > 4 || !(base > 1.0) || !(base <= 1e30)) return BSA_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > 256) return BSA_ERR_UNSUPPORTED;
  if (H > 65535 || (int64_t)Bt * L > INT32_MAX) return BSA_ERR_UNSUPPORTED;
  int64_t turned = 0;
  for (int i = 0; i < n_axes; ++i) {
    if (axis_dim[i] < 2 || axis_dim[i] % 2 != 0) return BSA_ERR_INVALID_ARG;
    turned += axis_dim[i];
  }
  if (turned > d) return BSA_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Y) || (reinterpret_cast<uintptr_t>(pos) & 3u) != 0)
    return BSA_ERR_INVALID_ARG;
  const bsa::RotaryArgs a{X, strides_of(xs, Bt, H, L, d), Y, strides_of(ys, Bt, H, L, d), type, Bt,
                          H, L, d, pos, pos_per_batch, n_axes, axis_dim, base, pairing, inverse};
  const int elem = type == BSA_TYPE_FP32 ? 4 : 2;
  bsa_status r = check_strides(a.xs, elem);
  if (r == BSA_OK) r = check_strides(a.ys, elem);
  if (r != BSA_OK) return r;
  // a step of 0 would have several threads write one place
  if ((Bt > 1 && a.ys.batch == 0) || (H > 1 && a.ys.head == 0) || (L > 1 && a.ys.row == 0))
    return BSA_ERR_INVALID_ARG;
  return from_cuda(bsa::launch_rotary(a, static_cast<cudaStream_t>(stream)));
}

size_t bsa_linear_workspace_bytes(int32_t Bt, int32_t L, int32_t K, int32_t N) {
  if (Bt <= 0 || L <= 0 || K <= 0 || N <= 0 || !linear_sizes_fit(Bt, L, K, N)) return 0;
  return bsa::linear_workspace(Bt, L, K, N);
}

static bsa_status linear_call(uint64_t wait_ns, const void* X, const bsa_strides* xs,
                              int32_t x_heads, const void* W, int64_t w_row, const void* bias,
                              int32_t act, const void* gate, const void* R, const bsa_strides* rs,
                              void* Y, const bsa_strides* ys, int32_t y_heads, int32_t type,
                              int32_t Bt, int32_t L, int32_t K, int32_t N, void* workspace,
                              size_t ws_bytes, int32_t* status, void* stream) {
  if (!X || !W || !Y) return BSA_ERR_INVALID_ARG;
  if (Bt <= 0 || L <= 0 || K <= 0 || N <= 0 || x_heads <= 0 || y_heads <= 0)
    return BSA_ERR_INVALID_ARG;
  if (K % x_heads != 0 || N % y_heads != 0 || w_row < 0) return BSA_ERR_INVALID_ARG;
  if (act < BSA_ACT_NONE || act > BSA_ACT_SILU) return BSA_ERR_INVALID_ARG;
  if (type != BSA_TYPE_BF16 && type != BSA_TYPE_FP16)
    return type == BSA_TYPE_FP32 ? BSA_ERR_UNSUPPORTED : BSA_ERR_INVALID_ARG;
  if ((x_heads > 1 && K / x_heads % 64 != 0) || (y_heads > 1 && N / y_heads % 64 != 0))
    return BSA_ERR_UNSUPPORTED;
  if (!linear_sizes_fit(Bt, L, K, N)) return BSA_ERR_UNSUPPORTED;
  if (!aligned16(X) || !aligned16(W)) return BSA_ERR_INVALID_ARG;
  for (const void* v : {bias, gate, R, static_cast<const void*>(Y)})
    if ((reinterpret_cast<uintptr_t>(v) & 1u) != 0) return BSA_ERR_INVALID_ARG;
  bsa::LinearArgs a{X, strides_of(xs, Bt, x_heads, L, K / x_heads), x_heads, W,
                          w_row == 0 ? K : w_row, bias, act, gate, R,
                          strides_of(rs, Bt, y_heads, L, N / y_heads), Y,
                          strides_of(ys, Bt, y_heads, L, N / y_heads), y_heads, type, Bt, L, K, N,
                          workspace, status, 0, wait_ns};
  if (a.w_row < K || a.w_row >= (int64_t)1 << 39) return BSA_ERR_INVALID_ARG;
  if (N > 1 && a.w_row % 8 != 0) return BSA_ERR_UNSUPPORTED;
  const bsa_status r = check_strides(a.xs, 2);
  if (r != BSA_OK) return r;
  if (a.xs.batch >= (int64_t)1 << 39 || a.xs.head >= (int64_t)1 << 39 ||
      a.xs.row >= (int64_t)1 << 39)
    return BSA_ERR_UNSUPPORTED;  // a tensor map's stride is below 2^40 bytes
  if (L > 1 && a.xs.row == 0) return BSA_ERR_INVALID_ARG;
  for (const int64_t v : {a.ys.batch, a.ys.head, a.ys.row, a.rs.batch, a.rs.head, a.rs.row})
    if (v < 0 || v >= (int64_t)1 << 39) return BSA_ERR_INVALID_ARG;
  if ((Bt > 1 && a.ys.batch == 0) || (y_heads > 1 && a.ys.head == 0) || (L > 1 && a.ys.row == 0))
    return BSA_ERR_INVALID_ARG;
  if (!workspace_ok(bsa::linear_workspace(Bt, L, K, N), workspace, ws_bytes))
    return BSA_ERR_WORKSPACE;
  return from_cuda(bsa::launch_linear(a, static_cast<cudaStream_t>(stream)));
}

bsa_status bsa_linear(const void* X, const bsa_strides* xs, int32_t x_heads, const void* W,
                      int64_t w_row, const void* bias, int32_t act, const void* gate,
                      const void* R, const bsa_strides* rs, void* Y, const bsa_strides* ys,
                      int32_t y_heads, int32_t type, int32_t Bt, int32_t L, int32_t K, int32_t N,
                      void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  return linear_call(0, X, xs, x_heads, W, w_row, bias, act, gate, R, rs, Y, ys, y_heads, type, Bt, L,
                     K, N, workspace, ws_bytes, status, stream);
}

size_t bsa_cross_workspace_bytes(int32_t Bt, int32_t H, int32_t Hkv, int32_t Lq, int32_t Lk,
                                 int32_t d) {
  if (check_cross(Bt, H, Hkv, Lq, Lk, d) != BSA_OK) return 0;
  return bsa::cross_workspace(Bt, H, Hkv, Lq, Lk, d);
}

static bsa_status cross_call(uint64_t wait_ns, const void* Q, const bsa_strides* qs, const void* K,
                             const bsa_strides* ks, const void* V, const bsa_strides* vs,
                             int32_t type, int32_t Bt, int32_t H, int32_t Hkv, int32_t Lq,
                             int32_t Lk, int32_t d, const int32_t* key_len,
                             const uint8_t* key_mask, float scale, void* O, const bsa_strides* os,
                             float* lse, void* workspace, size_t ws_bytes, int32_t* status,
                             void* stream) {
  bsa_status r = check_cross(Bt, H, Hkv, Lq, Lk, d);
  if (r != BSA_OK) return r;
  if (!Q || !O || (Lk > 0 && (!K || !V))) return BSA_ERR_INVALID_ARG;
  if (type != BSA_TYPE_BF16 && type != BSA_TYPE_FP16)
    return type == BSA_TYPE_FP32 ? BSA_ERR_UNSUPPORTED : BSA_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return BSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(key_len) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return BSA_ERR_INVALID_ARG;
  if (!(scale >= 0.f) || !(scale <= 1e30f)) return BSA_ERR_INVALID_ARG;
  bsa::CrossArgs a{Q, strides_of(qs, Bt, H, Lq, d), K, strides_of(ks, Bt, Hkv, Lk, d), V,
                   strides_of(vs, Bt, Hkv, Lk, d), type, Bt, H, Hkv, Lq, Lk, d, key_len, key_mask,
                   bsa::forward_scale(scale, d), O, strides_of(os, Bt, H, Lq, d), lse, workspace,
                   status, wait_ns};
  for (const bsa_strides& s : {a.qs, a.ks, a.vs, a.os}) {
    r = check_strides(s, 2);
    if (r != BSA_OK) return r;
    if (s.batch >= (int64_t)1 << 39 || s.head >= (int64_t)1 << 39 || s.row >= (int64_t)1 << 39)
      return BSA_ERR_UNSUPPORTED;  // a tensor map's stride is below 2^40 bytes
  }
  if ((Lq > 1 && (a.qs.row == 0 || a.os.row == 0)) || (Lk > 1 && (a.ks.row == 0 || a.vs.row == 0)))
    return BSA_ERR_INVALID_ARG;
  if ((Bt > 1 && a.os.batch == 0) || (H > 1 && a.os.head == 0)) return BSA_ERR_INVALID_ARG;
  if (!workspace_ok(bsa::cross_workspace(Bt, H, Hkv, Lq, Lk, d), workspace, ws_bytes))
    return BSA_ERR_WORKSPACE;
  return from_cuda(bsa::launch_cross(a, static_cast<cudaStream_t>(stream)));
}

bsa_status bsa_cross_forward(const void* Q, const bsa_strides* qs, const void* K,
                             const bsa_strides* ks, const void* V, const bsa_strides* vs,
                             int32_t type, int32_t Bt, int32_t H, int32_t Hkv, int32_t Lq,
                             int32_t Lk, int32_t d, const int32_t* key_len,
                             const uint8_t* key_mask, float scale, void* O, const bsa_strides* os,
                             float* lse, void* workspace, size_t ws_bytes, int32_t* status,
                             void* stream) {
  return cross_call(0, Q, qs, K, ks, V, vs, type, Bt, H, Hkv, Lq, Lk, d, key_len, key_mask, scale, O,
                    os, lse, workspace, ws_bytes, status, stream);
}

bsa_status bsa_selftest_linear_timeout(const void* X, const void* W, void* Y, int32_t type,
                                       int32_t L, int32_t K, int32_t N, void* workspace,
                                       size_t ws_bytes, int64_t wait_ns, int32_t* status,
                                       void* stream) {
  if (status == nullptr || wait_ns < 1 || wait_ns > 10000000000ll) return BSA_ERR_INVALID_ARG;
  return linear_call(static_cast<uint64_t>(wait_ns), X, nullptr, 1, W, 0, nullptr, BSA_ACT_NONE,
                     nullptr, nullptr, nullptr, Y, nullptr, 1, type, 1, L, K, N, workspace, ws_bytes,
                     status, stream);
}

bsa_status bsa_selftest_cross_timeout(const void* Q, const void* K, const void* V, void* O,
                                      int32_t type, int32_t H, int32_t Lq, int32_t Lk, int32_t d,
                                      const int32_t* key_len, void* workspace, size_t ws_bytes,
                                      int64_t wait_ns, int32_t* status, void* stream) {
  return bsa_selftest_cross_mask_timeout(Q, K, V, O, type, H, Lq, Lk, d, key_len, nullptr, workspace,
                                         ws_bytes, wait_ns, status, stream);
}

bsa_status bsa_selftest_cross_mask_timeout(const void* Q, const void* K, const void* V, void* O,
                                           int32_t type, int32_t H, int32_t Lq, int32_t Lk, int32_t d,
                                           const int32_t* key_len, const uint8_t* key_mask,
                                           void* workspace, size_t ws_bytes, int64_t wait_ns,
                                           int32_t* status, void* stream) {
  if (status == nullptr || wait_ns < 1 || wait_ns > 10000000000ll) return BSA_ERR_INVALID_ARG;
  return cross_call(static_cast<uint64_t>(wait_ns), Q, nullptr, K, nullptr, V, nullptr, type, 1, H, H,
                    Lq, Lk, d, key_len, key_mask, 0.f, O, nullptr, nullptr, workspace, ws_bytes,
                    status, stream);
}

}  // extern "C"
