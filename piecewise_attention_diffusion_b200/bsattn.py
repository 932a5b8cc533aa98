"""Thin Python binding of libbsattn (include/bsattn.h).

Argument marshalling only: every step of the computation runs in the library's CUDA
kernels. torch supplies device memory and the current stream. The functions named
``bsa_*`` mirror the C entry points one to one and take torch tensors; the lower-case
helpers (``build_mask``, ``precompute``, ``route``, ``forward``; around the block attention
``rotary``, ``linear``, ``cross_forward``) allocate the outputs and workspace with torch and
call them.

If the shared library is missing or cannot be loaded, every call raises: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsattn.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_BAD_CSR, ERR_TIMEOUT, ERR_WORKSPACE, \
    ERR_CAPACITY, ERR_SCRATCH_LIMIT, ERR_BAD_PADDING = range(10)
NOALLOC_SCRATCH_BYTES = 16 << 20
MODE_KEEP_OR_DROP, MODE_PISA, MODE_PISA_BLOCK = 0, 1, 2
TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
PAIR_ADJACENT, PAIR_HALVES = 0, 1
ACT_NONE, ACT_GELU_TANH, ACT_GELU_ERF, ACT_SILU = range(4)
CALL_BUILD_MASK, CALL_PRECOMPUTE, CALL_ROUTE, CALL_FORWARD = 0, 1, 2, 3

# Every symbol include/bsattn.h declares, in header order.
EXPORTS = ("bsa_version", "bsa_status_string", "bsa_mask_blocks", "bsa_workspace_bytes",
           "bsa_build_mask", "bsa_precompute", "bsa_route", "bsa_forward",
           "bsa_forward_noalloc", "bsa_selftest_wait_timeout", "bsa_selftest_forward_timeout",
           "bsa_rotary", "bsa_linear_workspace_bytes", "bsa_linear",
           "bsa_cross_workspace_bytes", "bsa_cross_forward", "bsa_selftest_linear_timeout",
           "bsa_selftest_cross_timeout", "bsa_selftest_cross_mask_timeout")


class BsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


class MaskDesc(ctypes.Structure):
    _fields_ = [("n_text_blocks", ctypes.c_int32), ("grid_h", ctypes.c_int32),
                ("grid_w", ctypes.c_int32), ("radius", ctypes.c_int32),
                ("global_stride", ctypes.c_int32), ("global_rows_full", ctypes.c_int32)]


class Strides(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("head", ctypes.c_int64), ("row", ctypes.c_int64)]


_lib = None
_vp, _i32, _i64, _f32, _sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                              ctypes.c_float, ctypes.c_size_t)
_sp = ctypes.POINTER(Strides)
_SIGS = {
    "bsa_version": (_i32, []),
    "bsa_status_string": (ctypes.c_char_p, [_i32]),
    "bsa_mask_blocks": (_i32, [ctypes.POINTER(MaskDesc)]),
    "bsa_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "bsa_build_mask": (_i32, [ctypes.POINTER(MaskDesc), _vp, _vp, _i64, _vp, _vp]),
    "bsa_precompute": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                              _vp, _vp, _sz, _vp, _vp]),
    "bsa_route": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _i32, _f32, _f32,
                         _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "bsa_forward": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _i64,
                           _i32, _i32, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _sz, _vp, _vp]),
    "bsa_forward_noalloc": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp,
                                   _i64, _i32, _i32, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _vp]),
    "bsa_selftest_wait_timeout": (_i32, [_i64, _vp, _vp]),
    "bsa_selftest_forward_timeout": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp,
                                            _vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _sz,
                                            _i64, _vp, _vp]),
    "bsa_rotary": (_i32, [_vp, _sp, _vp, _sp, _i32, _i32, _i32, _i32, _i32, _vp, _i32, _i32,
                          ctypes.POINTER(_i32), ctypes.c_double, _i32, _i32, _vp]),
    "bsa_linear_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "bsa_linear": (_i32, [_vp, _sp, _i32, _vp, _i64, _vp, _i32, _vp, _vp, _sp, _vp, _sp, _i32,
                          _i32, _i32, _i32, _i32, _i32, _vp, _sz, _vp, _vp]),
    "bsa_cross_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "bsa_cross_forward": (_i32, [_vp, _sp, _vp, _sp, _vp, _sp, _i32, _i32, _i32, _i32, _i32, _i32,
                                 _i32, _vp, _vp, _f32, _vp, _sp, _vp, _vp, _sz, _vp, _vp]),
    "bsa_selftest_linear_timeout": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _sz, _i64,
                                           _vp, _vp]),
    "bsa_selftest_cross_timeout": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp,
                                          _vp, _sz, _i64, _vp, _vp]),
    "bsa_selftest_cross_mask_timeout": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                               _vp, _vp, _vp, _sz, _i64, _vp, _vp]),
}


def lib() -> ctypes.CDLL:
    """Load libbsattn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m piecewise_attention_diffusion_b200.build`")
        so = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(so, name)
            fn.restype = res
            fn.argtypes = args
        _lib = so
    return _lib


def status_string(code: int) -> str:
    return lib().bsa_status_string(int(code)).decode()


def _check(code: int, where: str):
    if code != OK:
        raise BsaError(code, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, dtype, name, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _desc(desc) -> MaskDesc:
    if isinstance(desc, MaskDesc):
        return desc
    return MaskDesc(int(desc["n_text_blocks"]), int(desc["grid_h"]), int(desc["grid_w"]),
                    int(desc["radius"]), int(desc["global_stride"]),
                    int(desc.get("global_rows_full", 0)))


# ------------------------------------------------------------------ C entry points
def bsa_version() -> int:
    return int(lib().bsa_version())


def bsa_mask_blocks(desc) -> int:
    d = _desc(desc)
    return int(lib().bsa_mask_blocks(ctypes.byref(d)))


def bsa_workspace_bytes(call: int, Bt: int, H: int, L: int, d: int, block: int) -> int:
    return int(lib().bsa_workspace_bytes(call, Bt, H, L, d, block))


def bsa_build_mask(desc, row_ptr, col_idx, status=None, stream=None):
    d = _desc(desc)
    _need(row_ptr, torch.int32, "row_ptr")
    _need(col_idx, torch.int32, "col_idx")
    _check(lib().bsa_build_mask(ctypes.byref(d), _ptr(row_ptr), _ptr(col_idx),
                                col_idx.numel(), _ptr(status), _stream(stream)),
           "bsa_build_mask")


def _bhld(x, name):
    _need(x, torch.bfloat16, name)
    if x.dim() != 4:
        raise ValueError(f"{name} must be [Bt, H, L, d]")
    return x.shape


def _key_valid(key_valid, L, block):
    """Check the per-block real-token counts (int32[L/block], shared by all heads)."""
    if key_valid is not None:
        _need(key_valid, torch.int32, "key_valid", (L // block,))
    return _ptr(key_valid)


def bsa_precompute(K, V, block, kbar, vsum, Hbar, Mnorm, Hblk=None, workspace=None,
                   status=None, stream=None, key_valid=None):
    Bt, H, L, d = _bhld(K, "K")
    _need(V, torch.bfloat16, "V", K.shape)
    M = L // block
    _need(kbar, torch.float32, "kbar", (Bt * H, M, d))
    _need(vsum, torch.float32, "vsum", (Bt * H, M, d))
    _need(Hbar, torch.float32, "Hbar", (Bt * H, d, d))
    _need(Mnorm, torch.float32, "Mnorm", (Bt * H, M))
    if Hblk is not None:
        _need(Hblk, torch.float32, "Hblk", (Bt * H, M, d, d))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().bsa_precompute(_ptr(K), _ptr(V), Bt, H, L, d, block,
                                _key_valid(key_valid, L, block), _ptr(kbar), _ptr(vsum),
                                _ptr(Hbar), _ptr(Mnorm), _ptr(Hblk), _ptr(workspace), ws_bytes,
                                _ptr(status), _stream(stream)), "bsa_precompute")


def bsa_route(Q, kbar, Mnorm, block, k_top, lam, scale, row_ptr, col_idx, scores=None,
              workspace=None, status=None, stream=None, key_valid=None):
    Bt, H, L, d = _bhld(Q, "Q")
    M = L // block
    _need(kbar, torch.float32, "kbar", (Bt * H, M, d))
    _need(Mnorm, torch.float32, "Mnorm", (Bt * H, M))
    _need(row_ptr, torch.int32, "row_ptr", (Bt * H * (M + 1),))
    _need(col_idx, torch.int32, "col_idx", (Bt * H * M * k_top,))
    if scores is not None:
        _need(scores, torch.float32, "scores", (Bt * H, M, M))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().bsa_route(_ptr(Q), _ptr(kbar), _ptr(Mnorm), Bt, H, L, d, block,
                           _key_valid(key_valid, L, block), k_top,
                           float(lam), float(scale), _ptr(row_ptr), _ptr(col_idx),
                           _ptr(scores), _ptr(workspace), ws_bytes, _ptr(status),
                           _stream(stream)), "bsa_route")


def bsa_forward(Q, K, V, block, row_ptr, col_idx, csr_per_head, mode, kbar, vsum, Hbar, scale,
                O, lse=None, workspace=None, status=None, stream=None, key_valid=None):
    Bt, H, L, d = _bhld(Q, "Q")
    _need(K, torch.bfloat16, "K", Q.shape)
    _need(V, torch.bfloat16, "V", Q.shape)
    _need(O, torch.bfloat16, "O", Q.shape)
    _need(row_ptr, torch.int32, "row_ptr")
    _need(col_idx, torch.int32, "col_idx")
    M = L // block
    if mode == MODE_PISA:
        _need(kbar, torch.float32, "kbar", (Bt * H, M, d))
        _need(vsum, torch.float32, "vsum", (Bt * H, M, d))
        _need(Hbar, torch.float32, "Hbar", (Bt * H, d, d))
    if lse is not None:
        _need(lse, torch.float32, "lse", (Bt * H, L))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().bsa_forward(_ptr(Q), _ptr(K), _ptr(V), Bt, H, L, d, block,
                             _key_valid(key_valid, L, block), _ptr(row_ptr), _ptr(col_idx),
                             col_idx.numel(), int(csr_per_head), int(mode),
                             _ptr(kbar), _ptr(vsum), _ptr(Hbar), float(scale), _ptr(O),
                             _ptr(lse), _ptr(workspace), ws_bytes, _ptr(status),
                             _stream(stream)), "bsa_forward")


def bsa_forward_noalloc(Q, K, V, block, row_ptr, col_idx, csr_per_head, mode, kbar, vsum, Hbar,
                        scale, O, lse=None, status=None, stream=None, key_valid=None):
    """bsa_forward without a workspace argument: the library's built-in device scratch
    array is used instead, for callers that cannot allocate device memory."""
    Bt, H, L, d = _bhld(Q, "Q")
    _need(K, torch.bfloat16, "K", Q.shape)
    _need(V, torch.bfloat16, "V", Q.shape)
    _need(O, torch.bfloat16, "O", Q.shape)
    _need(row_ptr, torch.int32, "row_ptr")
    _need(col_idx, torch.int32, "col_idx")
    M = L // block
    if mode == MODE_PISA:
        _need(kbar, torch.float32, "kbar", (Bt * H, M, d))
        _need(vsum, torch.float32, "vsum", (Bt * H, M, d))
        _need(Hbar, torch.float32, "Hbar", (Bt * H, d, d))
    if lse is not None:
        _need(lse, torch.float32, "lse", (Bt * H, L))
    _check(lib().bsa_forward_noalloc(_ptr(Q), _ptr(K), _ptr(V), Bt, H, L, d, block,
                                     _key_valid(key_valid, L, block), _ptr(row_ptr),
                                     _ptr(col_idx), col_idx.numel(),
                                     int(csr_per_head), int(mode), _ptr(kbar), _ptr(vsum),
                                     _ptr(Hbar), float(scale), _ptr(O), _ptr(lse),
                                     _ptr(status), _stream(stream)), "bsa_forward_noalloc")


def bsa_selftest_wait_timeout(timeout_ns, status, stream=None):
    """Launch the bounded-wait self-test: the kernel's wait runs out after timeout_ns and
    BSA_ERR_TIMEOUT is written to `status` (device int32)."""
    _need(status, torch.int32, "status")
    _check(lib().bsa_selftest_wait_timeout(int(timeout_ns), _ptr(status), _stream(stream)),
           "bsa_selftest_wait_timeout")


def bsa_selftest_forward_timeout(Q, K, V, block, row_ptr, col_idx, mode, kbar, vsum, Hbar, O,
                                 workspace, wait_ns, status, stream=None):
    """bsa_forward (per-head lists) with every bounded wait of the attention kernel limited
    to wait_ns: the kernel's abort and drain path, reported as BSA_ERR_TIMEOUT in `status`."""
    Bt, H, L, d = _bhld(Q, "Q")
    _need(K, torch.bfloat16, "K", Q.shape)
    _need(V, torch.bfloat16, "V", Q.shape)
    _need(O, torch.bfloat16, "O", Q.shape)
    _need(row_ptr, torch.int32, "row_ptr")
    _need(col_idx, torch.int32, "col_idx")
    _need(status, torch.int32, "status")
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().bsa_selftest_forward_timeout(
        _ptr(Q), _ptr(K), _ptr(V), Bt, H, L, d, block, _ptr(row_ptr), _ptr(col_idx),
        col_idx.numel(), int(mode), _ptr(kbar), _ptr(vsum), _ptr(Hbar), _ptr(O),
        _ptr(workspace), ws_bytes, int(wait_ns), _ptr(status), _stream(stream)),
        "bsa_selftest_forward_timeout")


# The calls around the block attention take strided tensors of several types; they run on
# the tensors' device, whichever device is current. Small ones last a few microseconds, so
# their wrappers pass plain integers and ask torch for little.
def _view(t, name, first=None, shape=None):
    """Check a [Bt, H, L, d] tensor (or [Bt, L, N] for a single head) whose last dimension is
    contiguous, of `first`'s type and device; its strides, None if it is contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if first is None:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype not in TYPES:
            raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    elif t.dtype != first.dtype or t.get_device() != first.get_device():
        raise ValueError(f"{name} must be {first.dtype} on {first.device}, "
                         f"got {t.dtype} on {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    n = len(st)
    if n != 4 and n != 3:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [Bt, H, L, d]")
    if t.is_contiguous():
        return None
    if st[-1] != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return Strides(st[0], st[1], st[2]) if n == 4 else Strides(st[0], 0, st[1])


def _plain(t, dtype, name, shape, index):
    """The address of a contiguous tensor of this type and shape on device `index`; None for
    None."""
    if t is None:
        return None
    _need(t, dtype, name, shape)
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected device {index}")
    return t.data_ptr()


def _workspace_of(ws, index):
    """(address, bytes) of a workspace tensor on device `index`, or of none."""
    if ws is None:
        return None, 0
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on device {index}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _call(fn, index, stream, *args):
    """lib().fn(*args, stream) with device `index` current; on its current stream if none is
    given."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on device {index}")
    else:
        raw = stream.cuda_stream
    f = getattr(_lib or lib(), fn)
    if index == torch._C._cuda_getDevice():
        code = f(*args, raw)
    else:
        with torch.cuda.device(index):
            code = f(*args, raw)
    if code:
        raise BsaError(code, fn)


@functools.lru_cache(maxsize=64)
def _int_array(values):
    return (_i32 * max(len(values), 1))(*map(int, values))


def _rotary(X, xs, Y, ys, pos, axis_dims, base, pairing, inverse, stream):
    Bt, H, L, d = X.shape
    n, index = len(axis_dims), X.get_device()
    per = pos.dim() == 3
    pos_ptr = _plain(pos, torch.float32, "pos", (Bt, L, n) if per else (L, n), index)
    _call("bsa_rotary", index, stream, X.data_ptr(), xs, Y.data_ptr(), ys, TYPES[X.dtype], Bt, H, L,
          d, pos_ptr, per, n, _int_array(tuple(axis_dims)), base, pairing, bool(inverse))


def _four(t, name):
    if t.dim() != 4:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [Bt, H, L, d]")


def bsa_rotary(X, Y, pos, axis_dims, base=10000.0, pairing=PAIR_ADJACENT, inverse=False,
               stream=None):
    xs = _view(X, "X")
    _four(X, "X")
    _rotary(X, xs, Y, xs if Y is X else _view(Y, "Y", X, X.shape), pos, axis_dims, base, pairing,
            inverse, stream)


def bsa_linear_workspace_bytes(Bt: int, L: int, K: int, N: int) -> int:
    return int(lib().bsa_linear_workspace_bytes(Bt, L, K, N))


def _linear_shape(X, W, y_heads):
    """(Bt, L, K, N, x_heads) of X [Bt, L, K] or [Bt, H, L, d] and W [N, K]."""
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise ValueError("W must be a [N, K] tensor")
    shape = X.shape
    x_heads = shape[1] if len(shape) == 4 else 1
    N, K = W.shape
    if K != x_heads * shape[-1]:
        raise ValueError(f"W has shape {tuple(W.shape)}, X {tuple(shape)}")
    if y_heads and N % y_heads:
        raise ValueError(f"{N} columns do not divide into {y_heads} heads")
    return shape[0], shape[-2], K, N, x_heads


def _linear(X, xs, W, Y, ys, y_heads, dims, bias, act, gate, R, ws, ws_bytes, status, stream):
    Bt, L, K, N, x_heads = dims
    index, dtype = X.get_device(), X.dtype
    if W.dtype != dtype or W.get_device() != index:
        raise ValueError(f"W must be {dtype} on {X.device}, got {W.dtype} on {W.device}")
    row, last = W.stride()
    if last != 1 and K > 1:
        raise ValueError("W's rows must be contiguous")
    rs = None if R is None else ys if R is Y else _view(R, "R", X, Y.shape)
    _call("bsa_linear", index, stream, X.data_ptr(), xs, x_heads, W.data_ptr(), row if N > 1 else 0,
          _plain(bias, dtype, "bias", (N,), index), act, _plain(gate, dtype, "gate", (Bt, N), index),
          None if R is None else R.data_ptr(), rs, Y.data_ptr(), ys, y_heads, TYPES[dtype], Bt, L, K,
          N, ws, ws_bytes, _plain(status, torch.int32, "status", (1,), index))


def bsa_linear(X, W, Y, bias=None, act=ACT_NONE, gate=None, R=None, workspace=None, status=None,
               stream=None):
    xs = _view(X, "X")
    ys = _view(Y, "Y", X)
    heads = Y.shape[1] if Y.dim() == 4 else 1
    dims = Bt, L, K, N, _ = _linear_shape(X, W, heads)
    want = (Bt, heads, L, N // heads) if Y.dim() == 4 else (Bt, L, N)
    if Y.shape != want:
        raise ValueError(f"Y has shape {tuple(Y.shape)}, expected {want}")
    ws, ws_bytes = _workspace_of(workspace, X.get_device())
    _linear(X, xs, W, Y, ys, heads, dims, bias, act, gate, R, ws, ws_bytes, status, stream)


def bsa_cross_workspace_bytes(Bt: int, H: int, Hkv: int, Lq: int, Lk: int, d: int) -> int:
    return int(lib().bsa_cross_workspace_bytes(Bt, H, Hkv, Lq, Lk, d))


def _cross(Q, qs, K, V, O, os_, key_len, key_mask, scale, lse, ws, ws_bytes, status, stream):
    ks = _view(K, "K", Q)
    vs = _view(V, "V", Q, K.shape)
    Bt, H, Lq, d = Q.shape
    if K.dim() != 4 or K.shape[0] != Bt or K.shape[3] != d:
        raise ValueError(f"K has shape {tuple(K.shape)}, Q {tuple(Q.shape)}")
    Hkv, Lk = K.shape[1], K.shape[2]
    index = Q.get_device()
    if isinstance(key_mask, torch.Tensor) and key_mask.dtype == torch.bool:
        key_mask = key_mask.view(torch.uint8)  # the same bytes
    _call("bsa_cross_forward", index, stream, Q.data_ptr(), qs, K.data_ptr(), ks, V.data_ptr(), vs,
          TYPES[Q.dtype], Bt, H, Hkv, Lq, Lk, d,
          _plain(key_len, torch.int32, "key_len", (Bt,), index),
          _plain(key_mask, torch.uint8, "key_mask", (Bt, Lk), index), scale, O.data_ptr(), os_,
          _plain(lse, torch.float32, "lse", (Bt, H, Lq), index), ws, ws_bytes,
          _plain(status, torch.int32, "status", (1,), index))


def bsa_cross_forward(Q, K, V, O, key_len=None, key_mask=None, scale=0.0, lse=None,
                      workspace=None, status=None, stream=None):
    qs = _view(Q, "Q")
    _four(Q, "Q")
    os_ = _view(O, "O", Q, Q.shape)
    ws, ws_bytes = _workspace_of(workspace, Q.get_device())
    _cross(Q, qs, K, V, O, os_, key_len, key_mask, scale, lse, ws, ws_bytes, status, stream)


def bsa_selftest_linear_timeout(X, W, Y, workspace, wait_ns, status, stream=None):
    """bsa_linear of X [L, K], W [N, K] with every bounded wait limited to wait_ns: the kernels'
    abort and drain path, reported as BSA_ERR_TIMEOUT in `status`."""
    dev = X.get_device()
    (L, K), N = X.shape, W.shape[0]
    ws, ws_bytes = _workspace_of(workspace, dev)
    _call("bsa_selftest_linear_timeout", dev, stream, _plain(X, X.dtype, "X", (L, K), dev),
          _plain(W, X.dtype, "W", (N, K), dev), _plain(Y, X.dtype, "Y", (L, N), dev),
          TYPES[X.dtype], L, K, N, ws, ws_bytes, int(wait_ns), _plain(status, torch.int32, "status", (1,), dev))


def bsa_selftest_cross_timeout(Q, K, V, O, workspace, wait_ns, status, key_len=None, stream=None):
    """bsa_cross_forward of Q [H, Lq, d], K, V [H, Lk, d] with every bounded wait limited to
    wait_ns: the kernel's abort and drain path, reported as BSA_ERR_TIMEOUT in `status`."""
    _cross_timeout("bsa_selftest_cross_timeout", Q, K, V, O, (), workspace, wait_ns, status, key_len,
                   stream)


def bsa_selftest_cross_mask_timeout(Q, K, V, O, key_mask, workspace, wait_ns, status, key_len=None,
                                    stream=None):
    """The same of the kernel for a key_mask, uint8 [Lk]."""
    mask = _plain(key_mask, torch.uint8, "key_mask", (K.shape[1],), Q.get_device())
    _cross_timeout("bsa_selftest_cross_mask_timeout", Q, K, V, O, (mask,), workspace, wait_ns, status,
                   key_len, stream)


def _cross_timeout(fn, Q, K, V, O, mask, workspace, wait_ns, status, key_len, stream):
    dev, dt = Q.get_device(), Q.dtype
    (H, Lq, d), Lk = Q.shape, K.shape[1]
    ws, ws_bytes = _workspace_of(workspace, dev)
    _call(fn, dev, stream, _plain(Q, dt, "Q", (H, Lq, d), dev),
          _plain(K, dt, "K", (H, Lk, d), dev), _plain(V, dt, "V", (H, Lk, d), dev),
          _plain(O, dt, "O", (H, Lq, d), dev), TYPES[dt], H, Lq, Lk, d,
          _plain(key_len, torch.int32, "key_len", (1,), dev), *mask, ws, ws_bytes, int(wait_ns),
          _plain(status, torch.int32, "status", (1,), dev))


# ------------------------------------------------------------ allocating helpers
def workspace(call, Bt, H, L, d, block, device="cuda"):
    n = bsa_workspace_bytes(call, Bt, H, L, d, block)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def build_mask(desc, device="cuda", status=None):
    """Return (row_ptr int32[M+1], col_idx int32[nnz]) on `device`."""
    M = bsa_mask_blocks(desc)
    if M < 0:
        raise BsaError(ERR_INVALID_ARG, "build_mask")
    row_ptr = torch.empty(M + 1, dtype=torch.int32, device=device)
    col_idx = torch.empty(M * M, dtype=torch.int32, device=device)
    bsa_build_mask(desc, row_ptr, col_idx, status=status)
    nnz = int(row_ptr[-1].item())
    return row_ptr, col_idx[:nnz].clone()


def precompute(K, V, block, want_blocks=False, status=None, ws=None, key_valid=None):
    Bt, H, L, d = K.shape
    BH, M = Bt * H, L // block
    f = dict(dtype=torch.float32, device=K.device)
    out = dict(kbar=torch.empty(BH, M, d, **f), vsum=torch.empty(BH, M, d, **f),
               Hbar=torch.empty(BH, d, d, **f), Mnorm=torch.empty(BH, M, **f))
    out["Hblk"] = torch.empty(BH, M, d, d, **f) if want_blocks else None
    if ws is None:
        ws = workspace(CALL_PRECOMPUTE, Bt, H, L, d, block, K.device)
    bsa_precompute(K, V, block, out["kbar"], out["vsum"], out["Hbar"], out["Mnorm"],
                   out["Hblk"], ws, status, key_valid=key_valid)
    return out


def route(Q, kbar, Mnorm, block, k_top, lam=1.0, scale=0.0, want_scores=False, status=None,
          key_valid=None, ws=None):
    Bt, H, L, d = Q.shape
    BH, M = Bt * H, L // block
    row_ptr = torch.empty(BH * (M + 1), dtype=torch.int32, device=Q.device)
    col_idx = torch.empty(BH * M * k_top, dtype=torch.int32, device=Q.device)
    scores = torch.empty(BH, M, M, dtype=torch.float32, device=Q.device) if want_scores \
        else None
    if ws is None:
        ws = workspace(CALL_ROUTE, Bt, H, L, d, block, Q.device)
    bsa_route(Q, kbar, Mnorm, block, k_top, lam, scale, row_ptr, col_idx, scores, ws, status,
              key_valid=key_valid)
    return row_ptr, col_idx, scores


def forward(Q, K, V, block, row_ptr, col_idx, csr_per_head, mode, stats=None, scale=0.0,
            want_lse=False, status=None, ws=None, out=None, key_valid=None):
    Bt, H, L, d = Q.shape
    O = torch.empty_like(Q) if out is None else out
    lse = torch.empty(Bt * H, L, dtype=torch.float32, device=Q.device) if want_lse else None
    if ws is None:
        ws = workspace(CALL_FORWARD, Bt, H, L, d, block, Q.device)
    st = stats or {}
    bsa_forward(Q, K, V, block, row_ptr, col_idx, csr_per_head, mode, st.get("kbar"),
                st.get("vsum"), st.get("Hbar"), scale, O, lse, ws, status, key_valid=key_valid)
    return O, lse


# With `stream` given, a helper's inputs have to be ready on that stream, and the caller orders the
# result's use after it.
def _empty(like, shape, stream, dtype=None):
    """What a helper gives back: memory that `stream`, or the current one, may write at once. A block
    of the current stream's pool may still be in use by what that stream has queued, so with a
    stream given the memory comes from that stream's pool; it is kept for the current stream too,
    where the caller has it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _given(out, stream):
    """A caller's output, kept until `stream` has written it even if the caller lets go of it."""
    if stream is not None:
        out.record_stream(stream)
    return out


def _bytes_on(index, query, *sizes):
    """What a size query answers for device `index`: the plans behind it count that device's SMs."""
    f = getattr(_lib or lib(), query)
    if index == torch._C._cuda_getDevice():
        return f(*sizes)
    with torch.cuda.device(index):
        return f(*sizes)


def _scratch(like, n, stream):
    """n bytes of workspace of `stream`, or of the current one; None for 0. Freed when the helper
    returns, it goes to work that the same stream does later."""
    if n == 0:
        return None
    if stream is None:
        return like.new_empty((n,), dtype=torch.uint8)
    with torch.cuda.stream(stream):
        return like.new_empty((n,), dtype=torch.uint8)


def rotary(X, pos, axis_dims, base=10000.0, pairing=PAIR_ADJACENT, inverse=False, out=None,
           stream=None):
    """Rotary positions on [Bt, H, L, d] queries or keys (any strides, such as a projection's
    [Bt, L, H, d] transposed): fp32 pos [L, n] or [Bt, L, n], one column per axis, whose
    sections of d are axis_dims. Returns a contiguous [Bt, H, L, d], or `out` (which may be X
    itself). inverse turns back, which also takes gradients through the rotation."""
    if out is not None:
        bsa_rotary(X, out, pos, axis_dims, base, pairing, inverse, stream)
        return _given(out, stream)
    xs = _view(X, "X")
    _four(X, "X")
    out = _empty(X, X.shape, stream)
    _rotary(X, xs, out, None, pos, axis_dims, base, pairing, inverse, stream)
    return out


def linear(X, W, bias=None, act=ACT_NONE, gate=None, residual=None, heads=0, status=None, ws=None,
           out=None, stream=None):
    """residual + gate * act(X W^T + bias): X [Bt, L, K], or [Bt, H, L, d] whose heads side by
    side are the K columns; W [N, K]; gate [Bt, N]. Returns [Bt, L, N], with `heads` the
    [Bt, heads, L, N / heads] that the attention takes, or `out` (which may be the residual)."""
    xs = _view(X, "X")
    dims = Bt, L, K, N, _ = _linear_shape(X, W, heads)
    if ws is None:
        ws = _scratch(X, _bytes_on(X.get_device(), "bsa_linear_workspace_bytes", Bt, L, K, N), stream)
    if out is not None:
        bsa_linear(X, W, out, bias, act, gate, residual, ws, status, stream)
        return _given(out, stream)
    out = _empty(X, (Bt, heads, L, N // heads) if heads else (Bt, L, N), stream)
    ptr, ws_bytes = _workspace_of(ws, X.get_device())
    _linear(X, xs, W, out, None, heads or 1, dims, bias, act, gate, residual, ptr, ws_bytes, status,
            stream)
    return out


def cross_forward(Q, K, V, key_len=None, key_mask=None, scale=0.0, want_lse=False, status=None,
                  ws=None, out=None, stream=None):
    """Attention of Q [Bt, H, Lq, d] over K, V [Bt, Hkv, Lk, d] (any strides; H a multiple of
    Hkv): the first key_len[b] (int32 [Bt]) keys of each entry, those whose key_mask (uint8 or
    bool [Bt, Lk]) is not 0, or all. Returns (O contiguous or `out`, lse fp32 [Bt, H, Lq] or None)."""
    qs = _view(Q, "Q")
    _four(Q, "Q")
    if not isinstance(K, torch.Tensor) or K.dim() != 4:
        raise ValueError("K must be a [Bt, Hkv, Lk, d] tensor")
    Bt, H, Lq, d = Q.shape
    O, os_ = (_empty(Q, Q.shape, stream), None) if out is None else (out, _view(out, "out", Q, Q.shape))
    lse = _empty(Q, (Bt, H, Lq), stream, torch.float32) if want_lse else None
    if ws is None:
        ws = _scratch(Q, _bytes_on(Q.get_device(), "bsa_cross_workspace_bytes", Bt, H, K.shape[1], Lq,
                                   K.shape[2], d), stream)
    ptr, ws_bytes = _workspace_of(ws, Q.get_device())
    _cross(Q, qs, K, V, O, os_, key_len, key_mask, scale, lse, ptr, ws_bytes, status, stream)
    return (O if out is None else _given(O, stream)), lse


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)
