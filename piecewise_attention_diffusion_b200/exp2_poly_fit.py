"""Fit of the polynomials that the attention kernels use for part of their exponentials.

The softmax of the forward kernels evaluates 2^x for x <= 8, that of the cross attention for
x <= 15 (its fp16 weights are held 2^7 times larger). Most values go through the
special-function unit (ex2); a fixed share is computed on the FMA pipe instead so that
both pipes work in parallel. That path uses a Cody-Waite style split x = n + f with
n = rint(x) and f in [-1/2, 1/2] (W. J. Cody and W. Waite, "Software Manual for the
Elementary Functions", 1980), evaluates 2^f with a polynomial and adds n to the exponent field: of degree 3 in the
forward kernels (7.5e-5 relative, far below the weights' bf16), of degree 4 in the cross
attention (2.7e-6, as its log-sum-exp is fp32). The polynomial minimises the maximum RELATIVE error of p(f) against 2^f
on [-1/2, 1/2]; its coefficients come from the Remez exchange below (float64), rounded to
float32. Run this file to reproduce them:

    python -m piecewise_attention_diffusion_b200.exp2_poly_fit
"""
import numpy as np


def remez_exp2(degree: int = 3, iters: int = 30, grid: int = 200001):
    a, b = -0.5, 0.5
    x = 0.5 * (a + b) + 0.5 * (b - a) * np.cos(np.pi * np.arange(degree + 2)[::-1] / (degree + 1))
    g = np.linspace(a, b, grid)
    for _ in range(iters):
        A = np.zeros((degree + 2, degree + 2))
        for i in range(degree + 2):
            A[i, :degree + 1] = x[i] ** np.arange(degree + 1)
            A[i, degree + 1] = -((-1) ** i) * 2.0 ** x[i]
        sol = np.linalg.solve(A, 2.0 ** x)
        c = sol[:degree + 1]
        err = (np.polyval(c[::-1], g) - 2.0 ** g) / 2.0 ** g
        ext, start, sign = [], 0, np.sign(err)
        for i in range(1, grid):
            if sign[i] != sign[start]:
                ext.append(start + int(np.argmax(np.abs(err[start:i]))))
                start = i
        ext.append(start + int(np.argmax(np.abs(err[start:]))))
        while len(ext) > degree + 2:
            ext.pop(0 if abs(err[ext[0]]) < abs(err[ext[-1]]) else -1)
        if len(ext) == degree + 2:
            x = g[ext]
    return c, float(np.abs(err).max())


if __name__ == "__main__":
    for degree in (3, 4):
        c, e = remez_exp2(degree)
        print(f"degree {degree}: max relative error {e:.3e}")
        for k, v in enumerate(c):
            print(f"c{k} = {np.float32(v)!r}  (0x{np.float32(v).view(np.uint32):08x})")
