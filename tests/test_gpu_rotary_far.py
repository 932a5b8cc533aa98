"""bsa_rotary at far positions against angles formed in 60 decimal digits, to the documented bound: an
angle is off by less than |pos| 2^-50 radians besides what test_gpu_rotary.py derives for fp32
(2^-21 of |x_lo| + |x_hi|, and half a step of the result). A turn by an angle that is off by e moves a
component by at most e (|x_lo| + |x_hi|)."""
import decimal as dec
import math

import numpy as np
import pytest
import torch

from piecewise_attention_diffusion_b200 import bsattn as b

DEV = "cuda"


def _pi():
    """60 digits of pi, by Machin's formula."""
    def arctan_inverse(n, one):
        total = term = one // n
        i = 1
        while term:
            term //= -n * n
            i += 2
            total += term // i
        return total
    one = 10 ** 70
    return dec.Decimal(4 * (4 * arctan_inverse(5, one) - arctan_inverse(239, one))) / one


def _angles(pos, dim, base):
    """pos * base^(-2 i / dim) modulo 2 pi, for every i, exact to far below 2^-53."""
    with dec.localcontext() as ctx:
        ctx.prec = 60
        turn, log = 2 * _pi(), dec.Decimal(base).ln()
        out = []
        for i in range(dim // 2):
            phi = dec.Decimal(pos) * (-2 * i * log / dim).exp()
            out.append(float(phi - (phi / turn).to_integral_value() * turn))
        return np.array(out)


def test_the_angles_of_the_oracle():
    assert float(_pi()) == math.pi
    a = _angles(3.0, 8, 16.0)
    assert np.allclose(a, [3.0, 1.5, 0.75, 0.375], rtol=0, atol=0)
    for far in (1e15, 2.0 ** 44 + 2 ** 23, -4e9):    # the host's cosine reduces exactly
        assert abs(math.cos(_angles(far, 2, 16.0)[0]) - math.cos(far)) <= 2.0 ** -51


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("base", [10000.0, 1.5, 1e30])
def test_far_positions_to_the_documented_bound(cuda_ok, dtype, halves, base):
    pos = [2.0 ** 24 - 1, 2.0 ** 26, -(2.0 ** 26) + 4, 123456792.0, 1e9, -4e9, 2.0 ** 36 + 2 ** 14,
           2.0 ** 40, -(2.0 ** 40) - 2 ** 18, 2.0 ** 44 + 2 ** 23]
    d, L = 128, len(pos)
    g = torch.Generator().manual_seed(11)
    x = torch.randn(1, 2, L, d, generator=g).to(dtype)
    p = torch.tensor(pos, dtype=torch.float32)
    assert p.double().tolist() == pos    # a float holds each exactly
    got = b.rotary(x.to(DEV), p[:, None].contiguous().to(DEV), (d,), base=base,
                   pairing=b.PAIR_HALVES if halves else b.PAIR_ADJACENT)
    xs = x.double().numpy()
    lo, hi = (xs[..., :d // 2], xs[..., d // 2:]) if halves else (xs[..., ::2], xs[..., 1::2])
    phi = np.stack([_angles(v, d, base) for v in pos])
    c, s = np.cos(phi), np.sin(phi)
    want = [lo * c - hi * s, lo * s + hi * c]
    y = got.cpu().double().numpy()
    have = [y[..., :d // 2], y[..., d // 2:]] if halves else [y[..., ::2], y[..., 1::2]]
    size = np.abs(lo) + np.abs(hi)
    fi = torch.finfo(dtype)
    e = (2.0 ** -21 + np.abs(np.array(pos))[:, None] * 2.0 ** -50) * size
    for w, h in zip(want, have):
        tol = fi.eps / 2 * (np.abs(w) + e) + e + fi.smallest_normal * fi.eps / 2
        assert (np.abs(h - w) <= tol).all(), f"worst {np.max(np.abs(h - w) - tol):.3e}"
