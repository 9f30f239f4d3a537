"""Fits of the two polynomials of masked_attention.cu: 2^x on [-1/2, 1/2] (the
fraction behind Cody and Waite's reduction) and tanh(z) / z in z^2 on [0, 1]
(the score cap).  Weighted least squares on Chebyshev nodes whose weights are
raised where the relative residual is large (Lawson's iteration, which drives
the error toward equal ripple).  Running this file prints the coefficients and
their relative errors."""
import numpy as np


def fit(f, terms, lo, hi, nodes=4001, iters=400):
    """(coefficients, largest relative error) of a polynomial of ``terms``
    coefficients for f on [lo, hi]."""
    x = np.cos(np.linspace(0, np.pi, nodes)) * (hi - lo) / 2 + (lo + hi) / 2
    basis, y = np.vander(x, terms, increasing=True), f(x)
    w = np.ones_like(x)
    for _ in range(iters):
        r = np.sqrt(w) / y
        c, *_ = np.linalg.lstsq(basis * r[:, None], y * r, rcond=None)
        e = np.abs((basis @ c - y) / y)
        w = w * e + 1e-300
        w /= w.sum()
    return c, e.max()


def tanh_ratio(t):
    z = np.sqrt(np.maximum(t, 1e-300))
    return np.where(t > 1e-12, np.tanh(z) / z, 1.0)


if __name__ == "__main__":
    for terms in (4, 5):
        print("2^x", terms, *fit(np.exp2, terms, -0.5, 0.5))
    for terms in (5, 6):
        print("tanh(z) / z", terms, *fit(tanh_ratio, terms, 0.0, 1.0))
