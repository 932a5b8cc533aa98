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
