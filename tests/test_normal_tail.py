"""The normal tail of bsa_linear's GELU (csrc/linear_common.cuh, normal_tail) against erfc. The
constants are read from the kernel source and its float32 steps are replayed in numpy."""
import math
import os
import re

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "piecewise_attention_diffusion_b200", "csrc", "linear_common.cuh")


def _constants():
    src = open(SRC).read()
    p = float(re.search(r"kTailP = ([0-9.e-]+)f", src).group(1))
    q = [float(v) for v in re.findall(r"(-?[0-9.]+)f", re.search(r"kTail\[7\] = \{(.*?)\}", src, re.S).group(1))]
    assert len(q) == 7
    return np.float32(p), np.array(q, dtype=np.float32)


def test_gelu_by_the_normal_tail():
    f32 = np.float32
    p, c = _constants()
    z = np.concatenate([np.linspace(-13, 13, 20001), np.linspace(-0.01, 0.01, 201)]).astype(f32)
    a = np.abs(z)
    t = f32(1) / (f32(1) + p * a)
    q = np.full_like(t, c[6])
    for k in range(5, -1, -1):
        q = q * t + c[k]
    h = q * t * np.exp2(a * a * f32(-0.72134752)).astype(f32)
    y = z * np.where(z < 0, h, f32(1) - h)
    want = np.array([0.5 * v * math.erfc(-v / math.sqrt(2)) for v in z.astype(float)])
    # the fit's 6.3e-7 of the tail (at most a half), and eight roundings of 2^-24
    bound = 0.5 * 6.3e-7 + 8 * 2.0 ** -24
    assert (np.abs(y - want) <= bound * np.abs(z)).all()
    # and of a tail's own size: an exponent of up to 2^7 rounded three times in 2^-24
    far = want != 0
    assert (np.abs(y - want)[far] <= (6.3e-7 + (8 + 3 * 2 ** 7 * math.log(2)) * 2.0 ** -24) * np.abs(want)[far]).all()
