"""Fits the polynomial the activation backward pass uses for GELU's derivative.

GELU'(x) = Phi(x) + x phi(x).  With a = |x| and T(a) = Phi(-a) - a phi(a) it is 1 - T(a)
for x >= 0 and T(a) below, and T(a) = exp(-a^2 / 2) (E(a) - a / sqrt(2 pi)) with
E(a) = erfcx(a / sqrt 2) / 2.  E falls like 1 / a, and so does t = 1 / (1 + R a): a polynomial
in t follows E over the whole range (a is held to 14, from where on fp32's exp2 gives 0).  The
error in E is weighted by exp(-a^2 / 2), what it costs in the derivative, but at least by 1e-3,
so that it stays small beside E - a / sqrt(2 pi) and the derivative keeps its relative accuracy
where it is small.  The fit is made near-minimax by Lawson's iteratively reweighted least
squares; the reference is scipy.special.erfcx.  R is where such fits of this degree have the
smallest error.  Run it to print the coefficients (float32, lowest degree first), the largest
error of the derivative on [-12, 12] and the largest relative one on [-12, -2], evaluated in
float32 the way the kernel does (Horner with fused multiply-adds, exact exp2 and reciprocal in
place of the hardware's).

    python fit_gelu_slope.py
"""

import numpy as np
from numpy.polynomial import chebyshev
from scipy.special import erfcx, ndtr

A_MAX = 14.0
DEGREE = 6
R = 0.38
LEAST_WEIGHT = 1e-3


def fit(degree: int = DEGREE, a_max: float = A_MAX, iters: int = 300) -> np.ndarray:
    a = 0.5 * a_max * (1 - np.cos(np.linspace(0, np.pi, 6001)))
    e = 0.5 * erfcx(a / np.sqrt(2))
    w = np.maximum(np.exp(-a * a / 2), LEAST_WEIGHT)
    V = chebyshev.chebvander(2 / (1 + R * a) - 1, degree)
    lw = np.ones_like(a)
    best = (np.inf, None)
    for _ in range(iters):
        sw = w * np.sqrt(lw)
        c, *_ = np.linalg.lstsq(V * sw[:, None], e * sw, rcond=None)
        err = np.abs(V @ c - e) * w
        if err.max() < best[0]:
            best = (err.max(), c)
        lw = lw * (err / err.max() + 1e-12)
        lw /= lw.sum()
    poly = np.polynomial.Polynomial(chebyshev.cheb2poly(best[1]))
    return poly(np.polynomial.Polynomial([-1.0, 2.0])).coef.astype(np.float32)


def gelu_slope_f32(x: np.ndarray, coef: np.ndarray, a_max: float = A_MAX) -> np.ndarray:
    x = x.astype(np.float32)

    def fma(p, q, r):
        return (p.astype(np.float64) * np.float64(np.float32(q)) + np.float64(np.float32(r))).astype(np.float32)

    a = np.minimum(np.abs(x), np.float32(a_max))
    t = np.float32(1) / fma(a, R, 1)
    p = np.full_like(a, coef[-1])
    for c in coef[-2::-1]:
        p = (p.astype(np.float64) * t + np.float64(c)).astype(np.float32)
    p = (a.astype(np.float64) * np.float64(np.float32(-1 / np.sqrt(2 * np.pi))) + p).astype(np.float32)
    u = (a * np.float32(-0.5 * np.log2(np.e))).astype(np.float32) * a
    s = (p * np.exp2(u.astype(np.float64)).astype(np.float32)).astype(np.float32)
    return np.where(x < 0, s, np.float32(1) - s)


def gelu_slope_exact(x: np.ndarray) -> np.ndarray:
    x = x.astype(np.float64)
    return ndtr(x) + x * np.exp(-x * x / 2) / np.sqrt(2 * np.pi)


if __name__ == "__main__":
    c = fit()
    print("coefficients:", ", ".join(f"{float(v):.9g}f" for v in c))
    x = np.linspace(-12, 12, 960001).astype(np.float32)
    print(f"  max |GELU' error| on [-12, 12]: {np.abs(gelu_slope_f32(x, c) - gelu_slope_exact(x)).max():.3g}")
    x = x[x <= -2]
    print(f"  max relative error on [-12, -2]: {np.abs(gelu_slope_f32(x, c) / gelu_slope_exact(x) - 1).max():.3g}")
