"""Refusals of the calls around the block attention (CPU): every call below is refused by
the host's checks before a pointer is read or anything is launched."""
import ctypes

import pytest
import torch

from piecewise_attention_diffusion_b200 import bsattn as b

P = ctypes.c_void_p(1 << 20)          # 16-byte aligned; never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 4)


def _dims(*v):
    return (ctypes.c_int32 * max(len(v), 1))(*v)


def _rotary(x=P, y=P, xs=None, ys=None, type=0, Bt=2, H=4, L=8, d=64, pos=P, per=0, axes=(16, 24),
            n=None, base=1e4, pairing=0, inverse=0):
    return b.lib().bsa_rotary(x, xs, y, ys, type, Bt, H, L, d, pos, per,
                              len(axes) if n is None else n, _dims(*axes), base, pairing, inverse,
                              None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), b.ERR_INVALID_ARG), (dict(y=None), b.ERR_INVALID_ARG),
    (dict(pos=None), b.ERR_INVALID_ARG), (dict(x=ODD), b.ERR_INVALID_ARG),
    (dict(pos=ctypes.c_void_p((1 << 20) + 2)), b.ERR_INVALID_ARG),
    (dict(Bt=0), b.ERR_INVALID_ARG), (dict(H=0), b.ERR_INVALID_ARG),
    (dict(L=0), b.ERR_INVALID_ARG), (dict(L=-1), b.ERR_INVALID_ARG),
    (dict(type=3), b.ERR_INVALID_ARG), (dict(pairing=2), b.ERR_INVALID_ARG),
    (dict(n=0), b.ERR_INVALID_ARG), (dict(axes=(8,) * 5), b.ERR_INVALID_ARG),
    (dict(axes=(15, 24)), b.ERR_INVALID_ARG), (dict(axes=(0, 24)), b.ERR_INVALID_ARG),
    (dict(axes=(48, 24)), b.ERR_INVALID_ARG),
    (dict(axes=(2 ** 30, 2 ** 30, 2 ** 30, 2 ** 30)), b.ERR_INVALID_ARG),
    (dict(base=1.0), b.ERR_INVALID_ARG), (dict(base=float("nan")), b.ERR_INVALID_ARG),
    (dict(base=float("inf")), b.ERR_INVALID_ARG),
    (dict(d=60), b.ERR_UNSUPPORTED), (dict(d=264), b.ERR_UNSUPPORTED),
    (dict(H=65536), b.ERR_UNSUPPORTED), (dict(Bt=2 ** 20, L=2 ** 20), b.ERR_UNSUPPORTED),
    (dict(xs=b.Strides(-64, 64, 64)), b.ERR_INVALID_ARG),
    (dict(xs=b.Strides(2048, 512, 68)), b.ERR_UNSUPPORTED),
    (dict(ys=b.Strides(2048, 512, 60), type=1), b.ERR_UNSUPPORTED),
    (dict(ys=b.Strides(0, 512, 64)), b.ERR_INVALID_ARG),
    (dict(ys=b.Strides(2048, 0, 64)), b.ERR_INVALID_ARG),
    (dict(ys=b.Strides(2048, 512, 0)), b.ERR_INVALID_ARG)])
def test_rotary_refuses(kw, want):
    assert _rotary(**kw) == want


def test_bindings_refuse_host_tensors():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        b.rotary(x, torch.zeros(8, 1), (64,))


def _linear(x=P, xs=None, xh=1, w=P, w_row=0, bias=None, act=0, gate=None, r=None, rs=None, y=P,
            ys=None, yh=1, type=0, Bt=2, L=8, K=128, N=192, ws=P, ws_bytes=1 << 40, status=None):
    return b.lib().bsa_linear(x, xs, xh, w, w_row, bias, act, gate, r, rs, y, ys, yh, type, Bt, L,
                              K, N, ws, ws_bytes, status, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), b.ERR_INVALID_ARG), (dict(w=None), b.ERR_INVALID_ARG),
    (dict(y=None), b.ERR_INVALID_ARG), (dict(x=ODD), b.ERR_INVALID_ARG),
    (dict(w=ODD), b.ERR_INVALID_ARG),
    (dict(y=ctypes.c_void_p((1 << 20) + 1)), b.ERR_INVALID_ARG),
    (dict(bias=ctypes.c_void_p((1 << 20) + 1)), b.ERR_INVALID_ARG),
    (dict(Bt=0), b.ERR_INVALID_ARG), (dict(L=0), b.ERR_INVALID_ARG),
    (dict(K=0), b.ERR_INVALID_ARG), (dict(N=0), b.ERR_INVALID_ARG),
    (dict(xh=0), b.ERR_INVALID_ARG), (dict(yh=-1), b.ERR_INVALID_ARG),
    (dict(xh=3), b.ERR_INVALID_ARG), (dict(yh=5), b.ERR_INVALID_ARG),
    (dict(xh=4), b.ERR_UNSUPPORTED), (dict(yh=2), b.ERR_UNSUPPORTED),
    (dict(act=-1), b.ERR_INVALID_ARG), (dict(act=4), b.ERR_INVALID_ARG),
    (dict(type=2), b.ERR_UNSUPPORTED), (dict(type=3), b.ERR_INVALID_ARG),
    (dict(w_row=64), b.ERR_INVALID_ARG), (dict(w_row=-128), b.ERR_INVALID_ARG),
    (dict(w_row=132), b.ERR_UNSUPPORTED), (dict(K=124), b.ERR_UNSUPPORTED),
    (dict(xs=b.Strides(1024, 0, 0)), b.ERR_INVALID_ARG),
    (dict(xs=b.Strides(1024, 0, 132)), b.ERR_UNSUPPORTED),
    (dict(xs=b.Strides(-1024, 0, 128)), b.ERR_INVALID_ARG),
    (dict(ys=b.Strides(0, 0, 192)), b.ERR_INVALID_ARG),
    (dict(ys=b.Strides(1536, 0, 0)), b.ERR_INVALID_ARG),
    (dict(r=P, rs=b.Strides(1536, 0, -192)), b.ERR_INVALID_ARG),
    (dict(Bt=2 ** 15, L=2 ** 15), b.ERR_UNSUPPORTED),
    (dict(Bt=2 ** 14, L=2 ** 15, N=2 ** 20), b.ERR_UNSUPPORTED)])
def test_linear_refuses(kw, want):
    assert _linear(**kw) == want


def _cross(q=P, qs=None, k=P, ks=None, v=P, vs=None, type=0, Bt=2, H=4, Hkv=2, Lq=8, Lk=16, d=64,
           n=None, m=None, scale=0.0, o=P, os=None, lse=None, ws=P, ws_bytes=1 << 40):
    return b.lib().bsa_cross_forward(q, qs, k, ks, v, vs, type, Bt, H, Hkv, Lq, Lk, d, n, m, scale,
                                     o, os, lse, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), b.ERR_INVALID_ARG), (dict(k=None), b.ERR_INVALID_ARG),
    (dict(v=None), b.ERR_INVALID_ARG), (dict(o=None), b.ERR_INVALID_ARG),
    (dict(q=ODD), b.ERR_INVALID_ARG), (dict(k=ODD), b.ERR_INVALID_ARG),
    (dict(o=ODD), b.ERR_INVALID_ARG), (dict(n=ctypes.c_void_p((1 << 20) + 2)), b.ERR_INVALID_ARG),
    (dict(lse=ctypes.c_void_p((1 << 20) + 2)), b.ERR_INVALID_ARG),
    (dict(Bt=0), b.ERR_INVALID_ARG), (dict(Lq=0), b.ERR_INVALID_ARG),
    (dict(Lk=-1), b.ERR_INVALID_ARG), (dict(H=3), b.ERR_INVALID_ARG),
    (dict(Hkv=0), b.ERR_INVALID_ARG), (dict(d=96), b.ERR_UNSUPPORTED),
    (dict(type=2), b.ERR_UNSUPPORTED), (dict(type=-1), b.ERR_INVALID_ARG),
    (dict(scale=-1.0), b.ERR_INVALID_ARG), (dict(scale=float("nan")), b.ERR_INVALID_ARG),
    (dict(scale=float("inf")), b.ERR_INVALID_ARG),
    (dict(qs=b.Strides(2048, 512, 68)), b.ERR_UNSUPPORTED),
    (dict(qs=b.Strides(2048, 512, 0)), b.ERR_INVALID_ARG),
    (dict(ks=b.Strides(2048, 1024, 0)), b.ERR_INVALID_ARG),
    (dict(vs=b.Strides(2048, -64, 64)), b.ERR_INVALID_ARG),
    (dict(os=b.Strides(0, 512, 64)), b.ERR_INVALID_ARG),
    (dict(os=b.Strides(2048, 0, 64)), b.ERR_INVALID_ARG),
    (dict(os=b.Strides(2048, 512, 0)), b.ERR_INVALID_ARG),
    (dict(Lq=1 << 30), b.ERR_UNSUPPORTED), (dict(Bt=1 << 16, H=1 << 8), b.ERR_UNSUPPORTED),
    (dict(Lq=1, Lk=8192, ws=None), b.ERR_WORKSPACE),
    (dict(Lq=1, Lk=8192, ws_bytes=64), b.ERR_WORKSPACE)])
def test_cross_refuses(kw, want):
    assert _cross(**kw) == want


def test_cross_workspace_sizes():
    assert b.bsa_cross_workspace_bytes(1, 40, 40, 16384, 512, 128) == 0   # every SM has rows
    assert b.bsa_cross_workspace_bytes(1, 2, 2, 1, 0, 64) == 0            # no key to split
    assert b.bsa_cross_workspace_bytes(1, 2, 2, 1, 32768, 64) > 0
    assert b.bsa_cross_workspace_bytes(1, 3, 2, 1, 32768, 64) == 0        # refused shapes
    assert b.bsa_cross_workspace_bytes(1, 2, 2, 1, 32768, 96) == 0


def test_timeout_selftests_refuse():
    lin, cro = b.lib().bsa_selftest_linear_timeout, b.lib().bsa_selftest_cross_timeout
    for wait in (0, -1, 10 ** 10 + 1):
        assert lin(P, P, P, 0, 8, 64, 64, P, 1 << 40, wait, P, None) == b.ERR_INVALID_ARG
        assert cro(P, P, P, P, 0, 2, 8, 64, 64, None, P, 1 << 40, wait, P, None) == b.ERR_INVALID_ARG
    assert lin(P, P, P, 0, 8, 64, 64, P, 1 << 40, 100, None, None) == b.ERR_INVALID_ARG
    assert cro(P, P, P, P, 0, 2, 8, 64, 64, None, P, 1 << 40, 100, None, None) == b.ERR_INVALID_ARG
    assert lin(P, P, P, 2, 8, 64, 64, P, 1 << 40, 100, P, None) == b.ERR_UNSUPPORTED
    assert cro(P, P, P, P, 0, 2, 8, 64, 96, None, P, 1 << 40, 100, P, None) == b.ERR_UNSUPPORTED
