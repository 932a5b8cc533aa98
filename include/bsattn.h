/*
 * libbsattn — block-sparse (keep-or-drop) and piecewise (PISA) attention for
 * diffusion transformers on one NVIDIA B200 (sm_100a).
 *
 * Sources (page title and section):
 *   [BSA]  "多模态 DiT 上的块稀疏 Attention" (block-sparse attention on multimodal DiT,
 *          dpshk.com engineering blog): §3.3 block-sparse output formula, §4.1 block
 *          layout (text first, image after, each padded to a block multiple), §4.2 the
 *          multimodal fixed pattern, §4.3/§4.4 the per-query-block loop with online
 *          softmax, §5.4 index lists instead of a dense mask, §8.1 build once / reuse.
 *   [PISA] "PISA: Piecewise Sparse Attention Is Wiser for Efficient Diffusion
 *          Transformers" (gist.science summary of arXiv 2602.01077), technical summary
 *          §2: exact-or-approximate split S_i / U_i, o_t = N_t / D_t, zeroth-order
 *          centroid terms alpha_{t,j}, global first-order correction with H-bar,
 *          covariance-aware routing with M_j = ||H_j - H-bar||, and the fused pipeline
 *          (precompute -> exact stage -> zeroth-order sweep -> first-order correction).
 *
 * Conventions shared by every call
 *   - Tensors are contiguous, row-major [Bt, H, L, d] (page [BSA] §4.3 uses
 *     q, k, v: [B, H, N, D]); Q, K, V and O are bf16; statistics are fp32.
 *     "BH" below is Bt * H, "M" is L / block.
 *   - Every pointer except `desc`, bsa_strides and `axis_dim`, which are read on the host
 *     during the call, is a DEVICE pointer the caller allocated; the
 *     library never allocates, frees or synchronises. Device buffers must be 16-byte
 *     aligned.
 *   - Every call is asynchronous on `stream` (a cudaStream_t, NULL = legacy default
 *     stream). The return value reports host-side argument validation and launch
 *     errors only.
 *   - `status` (nullable) is one device int32 the caller zeroes. Kernels that detect
 *     a data error (malformed block lists, overflowing capacity, a wait that timed
 *     out) write the first such bsa_status code there and never trap. A call whose
 *     inputs were found malformed leaves its outputs unwritten.
 *   - Supported: d in {64, 128}; block in {64, 128}; L % block == 0; M <= 2048.
 *     Anything else returns BSA_ERR_UNSUPPORTED. (The calls around the block attention,
 *     bsa_rotary, bsa_cross_forward and bsa_linear, take other shapes, types and
 *     strided tensors: each says which.)
 *   - Token padding ([BSA] §4.1 pads the text segment to a multiple of the block size;
 *     §7.3 gives a timestep token its own block): `key_valid` (nullable, device int32
 *     [M], shared by every (batch, head)) is the number of leading real tokens of each
 *     block, 1..block; the rest of the block is padding. NULL means no padding. Padded
 *     keys receive no attention weight; centroids, value sums, H_j and pooled queries
 *     are taken over real tokens only; an unselected block's Taylor-tail weight is its
 *     real-token count; a padded block is always computed exactly: bsa_route places it
 *     in every list, and bsa_forward in the PISA modes reports BSA_ERR_BAD_PADDING for a
 *     list that lacks one. Padded query rows are computed like any other row. Values
 *     outside 1..block report BSA_ERR_BAD_PADDING (and are clamped). A key_valid
 *     pointer that is not 4-byte aligned returns BSA_ERR_INVALID_ARG.
 */
#ifndef BSATTN_H
#define BSATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define BSA_API __attribute__((visibility("default")))
#else
#define BSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  BSA_OK = 0,
  BSA_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, non-positive size, ...     */
  BSA_ERR_UNSUPPORTED = 2,   /* valid request outside the supported shapes          */
  BSA_ERR_CUDA = 3,          /* a CUDA runtime call or kernel launch failed          */
  BSA_ERR_BAD_CSR = 4,       /* block lists malformed (device-detected)              */
  BSA_ERR_TIMEOUT = 5,       /* a bounded device-side wait gave up (device-detected) */
  BSA_ERR_WORKSPACE = 6,     /* workspace null or smaller than bsa_workspace_bytes   */
  BSA_ERR_CAPACITY = 7,      /* an output list would exceed its capacity (device)    */
  BSA_ERR_SCRATCH_LIMIT = 8, /* bsa_forward_noalloc: the shape needs more scratch than
                                BSA_NOALLOC_SCRATCH_BYTES                            */
  BSA_ERR_BAD_PADDING = 9    /* key_valid out of range, or a padded block missing from a
                                PISA list (device-detected)                          */
} bsa_status;

/* Size of the device scratch array built into the library for bsa_forward_noalloc. */
#define BSA_NOALLOC_SCRATCH_BYTES (16u << 20)

typedef enum {
  BSA_MODE_KEEP_OR_DROP = 0, /* [BSA] §3.3: softmax over the selected blocks only      */
  BSA_MODE_PISA = 1,         /* [PISA] §2: exact S_i + Taylor-approximated U_i         */
  BSA_MODE_PISA_BLOCK = 2    /* [PISA] §2, first order with each block's own H_j       */
} bsa_mode;

typedef enum {
  BSA_CALL_BUILD_MASK = 0,
  BSA_CALL_PRECOMPUTE = 1,
  BSA_CALL_ROUTE = 2,
  BSA_CALL_FORWARD = 3
} bsa_call;

/* Multimodal fixed pattern, [BSA] §4.2, generalised from the page's 1-D image
 * sequence to a 2-D grid of image blocks.
 *   n_text_blocks    text blocks at the front of the sequence ([BSA] §4.1 puts text
 *                    first, each modality padded to a block multiple);
 *   grid_h, grid_w   image blocks form a grid_h x grid_w grid, row-major;
 *   radius           image block a keeps image block b when the Chebyshev distance
 *                    of their grid positions is <= radius (radius 1 = 3x3 window;
 *                    grid_h 1 reproduces the page's |i - j| <= window_size);
 *   global_stride    image block b is global (kept by every image row) when
 *                    b % global_stride == 0; 0 disables global blocks;
 *   global_rows_full nonzero: global image blocks also keep every block.
 * Text rows and text columns are always full. M = n_text_blocks + grid_h*grid_w. */
typedef struct {
  int32_t n_text_blocks;
  int32_t grid_h;
  int32_t grid_w;
  int32_t radius;
  int32_t global_stride;
  int32_t global_rows_full;
} bsa_mask_desc;

/* Library version (major * 10000 + minor * 100 + patch). */
BSA_API int32_t bsa_version(void);

/* Human-readable name of a bsa_status code (static string, never NULL). */
BSA_API const char* bsa_status_string(int32_t code);

/* Number of blocks M of a mask descriptor, or -1 if the descriptor is invalid. */
BSA_API int32_t bsa_mask_blocks(const bsa_mask_desc* desc);

/* Bytes of device workspace a call needs for the given shape (0 = none). `call` is
 * a bsa_call; the sizes are those of the corresponding call. Returns 0 for an
 * unsupported shape. */
BSA_API size_t bsa_workspace_bytes(int32_t call, int32_t Bt, int32_t H, int32_t L, int32_t d,
                           int32_t block);

/* bsa_build_mask — the multimodal fixed pattern as CSR block lists ([BSA] §4.2,
 * stored as index lists per [BSA] §5.4; built once and reused per [BSA] §8.1).
 *   desc      host pointer to the pattern descriptor;
 *   row_ptr   device int32[M + 1]: row i's key blocks are col_idx[row_ptr[i] ..
 *             row_ptr[i+1]); row_ptr[0] = 0;
 *   col_idx   device int32[col_capacity], written strictly ascending per row;
 *             M*M always suffices;
 *   status    see conventions; BSA_ERR_CAPACITY if nnz > col_capacity (then only
 *             row_ptr is written).
 * One shared list serves every (batch, head) ([BSA] §8.2). */
BSA_API bsa_status bsa_build_mask(const bsa_mask_desc* desc, int32_t* row_ptr, int32_t* col_idx,
                          int64_t col_capacity, int32_t* status, void* stream);

/* bsa_precompute — per-block statistics of [PISA] §2 ("precompute" stage):
 *   kbar_j = (1/B_j) sum_n k_{j,n}                   -> kbar  fp32 [BH, M, d]
 *   vsum_j = sum_n v_{j,n}                           -> vsum  fp32 [BH, M, d]
 *   H_j    = sum_n (k_{j,n} - kbar_j)^T v_{j,n}      (d_k rows x d_v cols)
 *   Hbar   = (1/M) sum_j H_j  (mean over all blocks of the head) -> Hbar fp32 [BH, d, d]
 *   Mnorm_j = ||H_j - Hbar||_F (Frobenius)           -> Mnorm fp32 [BH, M]
 *   Hblk (nullable) receives every H_j              -> fp32 [BH, M, d, d]
 *   (sums over the B_j real tokens of block j: B_j = key_valid[j], or B)
 * K, V are bf16 [Bt, H, L, d]. workspace: device, >= bsa_workspace_bytes(
 * BSA_CALL_PRECOMPUTE, ...) bytes, contents scratch. */
BSA_API bsa_status bsa_precompute(const void* K, const void* V, int32_t Bt, int32_t H, int32_t L,
                          int32_t d, int32_t block, const int32_t* key_valid, float* kbar,
                          float* vsum, float* Hbar, float* Mnorm, float* Hblk,
                          void* workspace, size_t ws_bytes, int32_t* status, void* stream);

/* bsa_route — covariance-aware top-k block selection ([PISA] §2, routing).
 *   qbar_i   = mean of the (real) queries of block i;
 *   p_ij     = softmax_j(scale * qbar_i . kbar_j) over all M key blocks;
 *   score_ij = p_ij + lambda * Mnorm_j / sum_j' Mnorm_j'  (term is 0 if the sum is 0);
 *   S_i      = the padded blocks, then the highest scores up to k_top, ties to the
 *              smaller j, written ascending (BSA_ERR_BAD_PADDING if k_top is smaller
 *              than the number of padded blocks).
 * (The pages say the score "combines" the attention score with M_j without a
 * formula; this mix of two distributions is this library's reading.)
 *   Q        bf16 [Bt, H, L, d];  kbar fp32 [BH, M, d];  Mnorm fp32 [BH, M];
 *   scale    score scale; 0 selects 1/sqrt(d);
 *   row_ptr  device int32 [BH, M + 1]: absolute offsets into col_idx; head h row i is
 *            col_idx[row_ptr[h*(M+1)+i] .. row_ptr[h*(M+1)+i+1]) = h*M*k_top + i*k_top ..;
 *   col_idx  device int32 [BH, M * k_top];
 *   scores   nullable fp32 [BH, M, M] receives score_ij;
 *   workspace  device, >= bsa_workspace_bytes(BSA_CALL_ROUTE, ...) bytes (the column sums
 *            of every 32-row segment of Q, BH * L/32 * d floats), contents scratch.
 * 1 <= k_top <= M. */
BSA_API bsa_status bsa_route(const void* Q, const float* kbar, const float* Mnorm, int32_t Bt,
                     int32_t H, int32_t L, int32_t d, int32_t block, const int32_t* key_valid,
                     int32_t k_top, float lambda, float scale, int32_t* row_ptr,
                     int32_t* col_idx, float* scores, void* workspace, size_t ws_bytes,
                     int32_t* status, void* stream);

/* bsa_forward — fused online-softmax attention over block lists.
 *   mode BSA_MODE_KEEP_OR_DROP ([BSA] §3.3):
 *     o_t = sum_{j in S_i} sum_n e^{s q.k_{j,n}} v_{j,n} / sum_{j in S_i} sum_n e^{s q.k_{j,n}}
 *     A row with an empty list outputs zeros and lse = -inf.
 *   mode BSA_MODE_PISA ([PISA] §2), with alpha_tj = e^{s q_t.kbar_j}:
 *     N_t = sum_{S_i} sum_n e^{s q.k} v + sum_{U_i} alpha_tj vsum_j
 *           + s (q_t Hbar) sum_{U_i} alpha_tj
 *     D_t = sum_{S_i} sum_n e^{s q.k} + sum_{U_i} block * alpha_tj;   o_t = N_t / D_t
 *     (every exponent is shifted by a running row maximum, which cancels).
 *   mode BSA_MODE_PISA_BLOCK ([PISA] §2, the per-block first-order term, of which the
 *     Hbar form above is the global approximation):
 *     N_t = sum_{S_i} sum_n e^{s q.k} v + sum_{U_i} alpha_tj (vsum_j + s q_t H_j)
 *     D_t as for BSA_MODE_PISA. Because kbar_j is the mean key of block j, s q_t.kbar_j
 *     is the mean of the row's exact scores over the block, and
 *     alpha_tj (vsum_j + s q_t H_j) = sum_n alpha_tj (1 + s q_t.(k_{j,n} - kbar_j)) v_{j,n}:
 *     every unselected block is computed as a tile whose weights are the first-order
 *     expansion of e^{s q.k} about its centroid. No statistics are read (kbar, vsum,
 *     Hbar may be NULL); every block of every query block is a tile, so the tensor
 *     work is that of dense attention: an accuracy reference, not a fast path.
 *   Q, K, V      bf16 [Bt, H, L, d];   O bf16 [Bt, H, L, d] (written);
 *   row_ptr/col_idx  block lists, each row strictly ascending in [0, M);
 *     csr_per_head 0: one list of M rows (row_ptr int32[M+1]) shared by every head;
 *     csr_per_head 1: per-head lists laid out as bsa_route writes them;
 *   nnz_total    number of entries in col_idx (bounds every row_ptr value);
 *   kbar, vsum, Hbar  bsa_precompute outputs (PISA only; ignored, may be NULL, for
 *                keep-or-drop);
 *   scale        0 selects 1/sqrt(d);
 *   lse          nullable fp32 [BH, L]: natural-log denominator, m_t + log D_t;
 *   workspace    device, >= bsa_workspace_bytes(BSA_CALL_FORWARD, ...) bytes.
 *   key_valid    see the conventions: padded keys are masked; in the PISA modes every
 *                padded block must be in every list.
 * Malformed lists set BSA_ERR_BAD_CSR (a missing padded block BSA_ERR_BAD_PADDING) in
 * *status and leave O unwritten. */
BSA_API bsa_status bsa_forward(const void* Q, const void* K, const void* V, int32_t Bt, int32_t H,
                       int32_t L, int32_t d, int32_t block, const int32_t* key_valid,
                       const int32_t* row_ptr,
                       const int32_t* col_idx, int64_t nnz_total, int32_t csr_per_head,
                       int32_t mode, const float* kbar, const float* vsum,
                       const float* Hbar, float scale, void* O, float* lse,
                       void* workspace, size_t ws_bytes, int32_t* status, void* stream);

/* bsa_forward_noalloc — bsa_forward for callers that cannot allocate device memory.
 * (No counterpart in the pages: this is a deployment variant of bsa_forward.)
 * Some callers cannot call cudaMalloc: a host whose memory pool owns the whole device
 * and forbids allocations from plug-ins, a serving loop that cannot take cudaMalloc's
 * implicit synchronisation, an embedded runtime with a memory budget fixed at load time.
 * This call takes the same arguments as bsa_forward minus the workspace and computes
 * the same result; its scratch is one __device__ array of BSA_NOALLOC_SCRATCH_BYTES
 * inside the library, which every GPU that loads the library keeps until the process
 * exits. It calls no allocating routine.
 *   - The scratch address is looked up on the current device at every call (the device
 *     of the stream); the first call on a device may load the library's device code, so
 *     make it before any stream capture.
 *   - Every call shares the one array (per device) and leaves its contents behind; calls
 *     whose kernels overlap on the GPU (different streams or host threads) race on it,
 *     so serialise them.
 *   - Returns BSA_ERR_SCRATCH_LIMIT when the shape needs more scratch than the array
 *     holds: PISA needs 256 + 2*BH*Mp*d*2 + BH*d*d*2 bytes (Mp = M rounded up to 128,
 *     each term rounded up to 256), the other modes 256 bytes. Other errors as bsa_forward. */
BSA_API bsa_status bsa_forward_noalloc(const void* Q, const void* K, const void* V, int32_t Bt,
                                       int32_t H, int32_t L, int32_t d, int32_t block,
                                       const int32_t* key_valid, const int32_t* row_ptr,
                                       const int32_t* col_idx,
                                       int64_t nnz_total, int32_t csr_per_head, int32_t mode,
                                       const float* kbar, const float* vsum, const float* Hbar,
                                       float scale, void* O, float* lse, int32_t* status,
                                       void* stream);

/* bsa_selftest_wait_timeout — the failure path of every kernel, exercised without a fault.
 * (No counterpart in the pages.) Every wait of the library's kernels is bounded: a wait
 * that runs out sets a CTA-wide abort flag, the kernel drains and returns, and
 * BSA_ERR_TIMEOUT is written to *status, leaving the context usable. This call launches
 * one CTA whose thread waits, with that same bounded wait and a limit of timeout_ns, on
 * an mbarrier that nothing ever completes; the wait runs out and the kernel reports.
 *   timeout_ns  1 .. 10^10 (10 s); status: device int32, written with BSA_ERR_TIMEOUT.
 * Returns BSA_ERR_INVALID_ARG for a null status or a limit out of range. */
BSA_API bsa_status bsa_selftest_wait_timeout(int64_t timeout_ns, int32_t* status, void* stream);

/* bsa_selftest_forward_timeout — the attention kernel's own abort path, run without a fault.
 * (No counterpart in the pages.) The same launch sequence as bsa_forward (per-head lists,
 * no token padding, default scale, no lse), with every bounded wait of the attention
 * kernel limited to wait_ns instead of its 2 s default. With a limit far below the time
 * the kernel's copies and MMAs take, a wait runs out while TMA copies and tensor-core work
 * are in flight: the CTA raises its abort flag, every role leaves its loop, the producer
 * drains its copies, the MMA thread waits for its issued MMAs, TMEM is freed and
 * BSA_ERR_TIMEOUT is written to *status. O is then partly written (unspecified); the
 * context stays usable.
 *   wait_ns  1 .. 10^10; status: device int32 the caller zeroes (required); other
 *            arguments as bsa_forward. */
BSA_API bsa_status bsa_selftest_forward_timeout(const void* Q, const void* K, const void* V,
                                                int32_t Bt, int32_t H, int32_t L, int32_t d,
                                                int32_t block, const int32_t* row_ptr,
                                                const int32_t* col_idx, int64_t nnz_total,
                                                int32_t mode, const float* kbar,
                                                const float* vsum, const float* Hbar, void* O,
                                                void* workspace, size_t ws_bytes,
                                                int64_t wait_ns, int32_t* status, void* stream);

/* ---------------------------------------------------------------------------------
 * Calls around the block attention. (No counterpart in the pages: a diffusion
 * transformer's block also projects its tokens, rotates q and k by their positions and
 * attends to an encoder's states.) They share the conventions at the top of this file
 * but for the shapes: tensors are [Bt, H, L, d] with the head dimension contiguous and
 * any batch, head and row strides. */

/* Strides of a [Bt, H, L, d] tensor in elements. Every stride is >= 0 and, where its
 * dimension is larger than 1, a multiple of 16 bytes (else BSA_ERR_UNSUPPORTED). A NULL
 * pointer means contiguous. A projection's [Bt, L, H, d] is {L*H*d, d, H*d}. */
typedef struct {
  int64_t batch;
  int64_t head;
  int64_t row;
} bsa_strides;

typedef enum {
  BSA_TYPE_BF16 = 0,
  BSA_TYPE_FP16 = 1,
  BSA_TYPE_FP32 = 2
} bsa_type;

/* Which two components of an axis's section of d turn together: 2i and 2i + 1, or i and
 * i + (section / 2). */
typedef enum {
  BSA_PAIR_ADJACENT = 0,
  BSA_PAIR_HALVES = 1
} bsa_pairing;

/* bsa_rotary — rotary positions with one to four axes (time, height, width of a video's
 * or an image's tokens) on queries or keys, before bsa_precompute / bsa_route /
 * bsa_forward.
 *   The head dimension is cut into consecutive sections of axis_dim[0], axis_dim[1], ...
 *   components, one per axis; what is left of d is copied. Pair i of axis a turns by
 *     phi = pos[t][a] * base^(-2 i / axis_dim[a]):
 *     y_lo = x_lo cos phi - x_hi sin phi,   y_hi = x_lo sin phi + x_hi cos phi.
 *   inverse nonzero turns by -phi: the transposed map, which takes a gradient of y to
 *   the gradient of x.
 *   X, Y     [Bt, H, L, d] of `type` (bf16, fp16 or fp32), with strides xs, ys. Y may be
 *            X with the same strides (in place); any other overlap is undefined;
 *   d        a multiple of 8, at most 256;
 *   pos      device fp32 [L, n_axes], or [Bt, L, n_axes] with pos_per_batch nonzero; a
 *            text token at position 0 of every axis is left as it is. Angles are formed
 *            and reduced in 64 bits: besides the rounding of a sine to fp32, an angle is off
 *            by less than |pos| 2^-50 radians (up to positions of 2^26 less than that
 *            rounding; at 2^40 up to 2^-10). A position that is not finite makes its
 *            token's rotated components NaN;
 *   axis_dim host int32[n_axes], each even and >= 2, their sum at most d; 1 <= n_axes <= 4;
 *   base     > 1, finite.
 * Arithmetic is fp32, rounded once to `type`. */
BSA_API bsa_status bsa_rotary(const void* X, const bsa_strides* xs, void* Y,
                              const bsa_strides* ys, int32_t type, int32_t Bt, int32_t H,
                              int32_t L, int32_t d, const float* pos, int32_t pos_per_batch,
                              int32_t n_axes, const int32_t* axis_dim, double base,
                              int32_t pairing, int32_t inverse, void* stream);

typedef enum {
  BSA_ACT_NONE = 0,
  BSA_ACT_GELU_TANH = 1, /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
  BSA_ACT_GELU_ERF = 2,  /* z (1 + erf(z / sqrt 2)) / 2                      */
  BSA_ACT_SILU = 3       /* z / (1 + e^-z)                                    */
} bsa_act;

/* Bytes of device workspace bsa_linear needs on the current device (how the work is split depends
 * on its SMs); 0 if none, or for sizes that it refuses. */
BSA_API size_t bsa_linear_workspace_bytes(int32_t Bt, int32_t L, int32_t K, int32_t N);

/* bsa_linear — matrix product with bias, activation, gate and residual:
 *     Y[b, t, n] = R[b, t, n] + gate[b, n] * act(sum_k X[b, t, k] W[n, k] + bias[n]).
 * The projections into and out of the attention, the feed-forward and the modulation
 * layers. X's K columns and Y's N columns may be cut into heads, so that a projection
 * writes the [Bt, H, L, d] that bsa_precompute / bsa_route / bsa_forward read, and the
 * output projection reads the O that bsa_forward writes.
 *   X        `type` [Bt, x_heads, L, K / x_heads] with strides xs, 16-byte aligned;
 *            x_heads 1: plain [Bt, L, K]. With x_heads > 1, K / x_heads is a multiple of
 *            64. A batch or head stride of 0 repeats one tensor; the row stride is not 0
 *            (unless L is 1);
 *   W        `type` [N, K], rows w_row elements apart (0: K), w_row a multiple of 8;
 *            16-byte aligned;
 *   bias     nullable `type` [N];   gate  nullable `type` [Bt, N], contiguous;
 *   R        nullable `type` [Bt, y_heads, L, N / y_heads] with strides rs, any (a stride
 *            of 0 repeats);
 *   Y        `type`, the shape of R, strides ys: any that step over no place twice (with
 *            bases and strides of whole 16 bytes it is written by TMA); with y_heads > 1,
 *            N / y_heads is a multiple of 64. Y may be R with the same strides; it must
 *            not overlap the other inputs;
 *   type     bf16 or fp16; sums are fp32, rounded once after the residual;
 *   workspace  device, >= bsa_linear_workspace_bytes(Bt, L, K, N) bytes, contents scratch
 *            (NULL and 0 where that is 0);
 *   status   see the conventions (BSA_ERR_TIMEOUT).
 * Results are the same bits on every run on one kind of GPU: no atomics. */
BSA_API bsa_status bsa_linear(const void* X, const bsa_strides* xs, int32_t x_heads,
                              const void* W, int64_t w_row, const void* bias, int32_t act,
                              const void* gate, const void* R, const bsa_strides* rs, void* Y,
                              const bsa_strides* ys, int32_t y_heads, int32_t type, int32_t Bt,
                              int32_t L, int32_t K, int32_t N, void* workspace,
                              size_t ws_bytes, int32_t* status, void* stream);

/* Bytes of device workspace bsa_cross_forward needs on the current device (as for bsa_linear); 0
 * if none, or for sizes that it refuses. */
BSA_API size_t bsa_cross_workspace_bytes(int32_t Bt, int32_t H, int32_t Hkv, int32_t Lq,
                                         int32_t Lk, int32_t d);

/* bsa_cross_forward — attention of the image or video tokens over an encoder's states, whose
 * length is another.
 *     o_t = sum_n e^{s q_t.k_n} v_n / sum_n e^{s q_t.k_n}  over the real keys n
 *   Q        `type` [Bt, H, Lq, d], strides qs;   O  the same shape, strides os (written);
 *   K, V     `type` [Bt, Hkv, Lk, d], strides ks, vs. H is a multiple of Hkv; query head h
 *            reads key head h / (H / Hkv). Lk may be 0 (K, V may then be NULL). In Q, K and V
 *            a batch or head stride of 0 repeats one tensor;
 *   type     bf16 or fp16; d 64 or 128; bases 16-byte aligned. Scores, the running maximum
 *            and sum, and the output's sum are fp32; the weights of a tile are rounded to
 *            `type` for the second product;
 *   key_len  nullable device int32 [Bt]: entry b's real keys are its first key_len[b], 0..Lk
 *            (values outside report BSA_ERR_BAD_PADDING and are clamped);
 *   key_mask nullable device uint8 [Bt, Lk]: a key whose byte is 0 is not real. With both, a
 *            key is real if both say so. What K and V hold where a key is not real (NaN, say)
 *            never matters;
 *   scale    0 selects 1/sqrt(d);
 *   lse      nullable fp32 [Bt, H, Lq]: the natural logarithm of the denominator.
 * A row without a real key outputs zeros and lse = -inf, as does one whose real keys all have the
 * score -inf. O must not overlap Q, K or V.
 *   workspace  device, >= bsa_cross_workspace_bytes(...) bytes, contents scratch: with few
 *            query rows the keys are split over the GPU and their parts joined (always in one
 *            order: the same bits on every run);
 *   status   see the conventions. */
BSA_API bsa_status bsa_cross_forward(const void* Q, const bsa_strides* qs, const void* K,
                                     const bsa_strides* ks, const void* V, const bsa_strides* vs,
                                     int32_t type, int32_t Bt, int32_t H, int32_t Hkv, int32_t Lq,
                                     int32_t Lk, int32_t d, const int32_t* key_len,
                                     const uint8_t* key_mask, float scale, void* O,
                                     const bsa_strides* os, float* lse, void* workspace,
                                     size_t ws_bytes, int32_t* status, void* stream);

/* bsa_selftest_linear_timeout, bsa_selftest_cross_timeout, bsa_selftest_cross_mask_timeout — the
 * abort paths of bsa_linear's and bsa_cross_forward's kernels (the last one's that of the kernel
 * for a key_mask, uint8 [Lk]), run without a fault, as bsa_selftest_forward_timeout runs that of
 * bsa_forward: the same launch sequence on contiguous tensors (X [L, K], W [N, K], Y [L, N], no
 * bias, gate or residual; Q, O [H, Lq, d], K, V [H, Lk, d]) with every bounded wait limited to
 * wait_ns. With a limit far below the time of a copy a wait runs out while copies and products
 * are in flight: the kernel drains, frees TMEM and writes BSA_ERR_TIMEOUT to *status. The output
 * is then unspecified; the context stays usable.
 *   wait_ns  1 .. 10^10; status: device int32 the caller zeroes (required). (The kernel of
 *            bsa_cross_forward for at most four query rows of a key head has no waits.) */
BSA_API bsa_status bsa_selftest_linear_timeout(const void* X, const void* W, void* Y, int32_t type,
                                               int32_t L, int32_t K, int32_t N, void* workspace,
                                               size_t ws_bytes, int64_t wait_ns, int32_t* status,
                                               void* stream);
BSA_API bsa_status bsa_selftest_cross_timeout(const void* Q, const void* K, const void* V, void* O,
                                              int32_t type, int32_t H, int32_t Lq, int32_t Lk,
                                              int32_t d, const int32_t* key_len, void* workspace,
                                              size_t ws_bytes, int64_t wait_ns, int32_t* status,
                                              void* stream);
BSA_API bsa_status bsa_selftest_cross_mask_timeout(const void* Q, const void* K, const void* V,
                                                   void* O, int32_t type, int32_t H, int32_t Lq,
                                                   int32_t Lk, int32_t d, const int32_t* key_len,
                                                   const uint8_t* key_mask, void* workspace,
                                                   size_t ws_bytes, int64_t wait_ns,
                                                   int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BSATTN_H */
