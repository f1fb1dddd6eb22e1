"""Fits the polynomial the activation backward pass uses for GELU's derivative.

GELU'(x) = Phi(x) + x phi(x).  With a = |x| and T(a) = Phi(-a) - a phi(a) it is 1 - T(a)
for x >= 0 and T(a) below, and T(a) = exp(-a^2 / 2) P(a) with
P(a) = erfcx(a / sqrt 2) / 2 - a / sqrt(2 pi), a smooth function that a polynomial
approximates on [0, 6] (beyond, |T| < 4e-8).  The error in P is weighted by exp(-a^2 / 2),
what it costs in the derivative, and the fit made near-minimax by Lawson's iteratively
reweighted least squares; the reference is scipy.special.erfcx.  Run it to print the
coefficients (float32, lowest degree first) and the largest error of the derivative on
[-8, 8], evaluated in float32 the way the kernel does (Horner with fused multiply-adds,
exact exp2 in place of the hardware's).

    python fit_gelu_slope.py
"""

import numpy as np
from scipy.special import erfcx, ndtr

A_MAX = 6.0
DEGREE = 10


def fit(degree: int = DEGREE, a_max: float = A_MAX, iters: int = 300) -> np.ndarray:
    a = 0.5 * a_max * (1 - np.cos(np.linspace(0, np.pi, 6001)))
    p = 0.5 * erfcx(a / np.sqrt(2)) - a / np.sqrt(2 * np.pi)
    w = np.exp(-a * a / 2)
    V = np.vander(a / a_max, degree + 1, increasing=True)
    lw = np.ones_like(a)
    best = (np.inf, None)
    for _ in range(iters):
        sw = w * np.sqrt(lw)
        c, *_ = np.linalg.lstsq(V * sw[:, None], p * sw, rcond=None)
        e = np.abs(V @ c - p) * w
        if e.max() < best[0]:
            best = (e.max(), c)
        lw = lw * (e / e.max() + 1e-12)
        lw /= lw.sum()
    return (best[1] / a_max ** np.arange(degree + 1)).astype(np.float32)


def gelu_slope_f32(x: np.ndarray, coef: np.ndarray, a_max: float = A_MAX) -> np.ndarray:
    x = x.astype(np.float32)
    a = np.minimum(np.abs(x), np.float32(a_max))
    p = np.full_like(a, coef[-1])
    for c in coef[-2::-1]:
        p = (p.astype(np.float64) * a + np.float64(c)).astype(np.float32)
    u = (a * a * np.float32(-0.5 * np.log2(np.e))).astype(np.float32)
    t = (p * np.exp2(u.astype(np.float64)).astype(np.float32)).astype(np.float32)
    h = (np.float32(0.5) - t).astype(np.float32)
    return (np.float32(0.5) + np.copysign(h, h * np.where(np.signbit(x), -1, 1))).astype(np.float32)


def gelu_slope_exact(x: np.ndarray) -> np.ndarray:
    x = x.astype(np.float64)
    return ndtr(x) + x * np.exp(-x * x / 2) / np.sqrt(2 * np.pi)


if __name__ == "__main__":
    c = fit()
    print("coefficients:", ", ".join(f"{float(v):.9g}f" for v in c))
    x = np.linspace(-8, 8, 640001).astype(np.float32)
    print(f"  max |GELU' error| on [-8, 8]: {np.abs(gelu_slope_f32(x, c) - gelu_slope_exact(x)).max():.3g}")
