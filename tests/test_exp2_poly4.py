"""The FMA-pipe 2^x of the cross attention (csrc/cross.cu, ex2_poly4) against its error bound. The
constants are read from the kernel source and its float32 steps (clamp, 1.5 * 2^23 shift, Horner,
exponent add) are replayed bit for bit in numpy."""
import os
import re

import numpy as np

from piecewise_attention_diffusion_b200 import exp2_poly_fit

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "piecewise_attention_diffusion_b200", "csrc", "cross.cu")
# The fit's error with its coefficients rounded, and the rounding of Horner's steps: half a step of
# a result in [0.7, 1.42] (2^-24 of at least 0.7), and of the steps before it, times f <= 1/2 each.
BOUND = 2.7e-6 + 2 * 2.0 ** -24 / 0.7


def _constants():
    src = open(SRC).read()
    vals = {k: float(v) for k, v in re.findall(r"kE([0-4]) = ([0-9.eE+-]+)f", src)}
    assert sorted(vals) == ["0", "1", "2", "3", "4"]
    body = src[src.index("float2 ex2_poly4(float2 x)"):]
    body = body[:body.index("\n}\n")]
    order = [body.index(f"kE{k}") for k in (4, 3, 2, 1, 0)]
    assert order == sorted(order)    # Horner, from the highest
    assert "12582912.0f" in body and "fmaxf(x.x, -126.0f)" in body and "<< 23" in body
    return [np.float32(vals[str(k)]) for k in range(5)]


def _ex2(x):
    f32 = np.float32
    c = _constants()
    x = np.maximum(x.astype(f32), f32(-126.0))
    t = (x + f32(12582912.0)).astype(f32)
    f = (x - (t - f32(12582912.0)).astype(f32)).astype(f32)
    q = np.full_like(f, c[4])
    for k in (3, 2, 1, 0):
        q = (q.astype(np.float64) * f + c[k]).astype(f32)    # one rounding
    return (q.view(np.uint32) + (t.view(np.uint32) << np.uint32(23))).view(f32)


def test_constants_are_the_fits():
    c, err = exp2_poly_fit.remez_exp2(4)
    assert err < 2.7e-6
    np.testing.assert_array_equal(np.asarray(_constants()), c.astype(np.float32))


def test_relative_error_over_the_used_range():
    """Exponents of weights: at most 8 above the row's reference, 15 in fp16; those below -126 and
    -inf are a positive number too small to count."""
    x = np.concatenate([np.linspace(-126.0, 15.0, 2_000_001),
                        np.random.default_rng(1).uniform(-30, 15, 1_000_000)]).astype(np.float32)
    got, want = _ex2(x).astype(np.float64), np.exp2(x.astype(np.float64))
    normal = want >= 2.0 ** -125
    assert (np.abs(got - want)[normal] <= BOUND * want[normal]).all()
    tiny = _ex2(np.asarray([-np.inf, -1e30, -200.0, -126.7], dtype=np.float32))
    assert (tiny >= 0).all() and (tiny <= 2.0 ** -125).all()
