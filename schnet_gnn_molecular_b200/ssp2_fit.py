"""Coefficients of the shifted softplus of small arguments, used by ``ssp2_small`` in
``csrc/readout.cu`` (readout energies and gradients, where the MUFU logarithm's absolute error,
2^-22 around 1, would be most of a small activation).

In base 2, ssp2(t) = log2((1 + 2^t) / 2) = t / 2 + log2(cosh(t ln2 / 2)): an odd linear part, which
is exact, and an even part, written t^2 q(t^2) and fitted on |t| <= RANGE.

Method: reweighted least squares (Lawson's iteration) on Chebyshev nodes for the error relative
to |ssp2(t)| (the larger of the two signs'), which converges towards the minimax polynomial of the
given degree; the result is rounded to float32 and checked in float32 on a dense grid.

    python -m schnet_gnn_molecular_b200.ssp2_fit      # prints the coefficients and the bound
"""
from __future__ import annotations

import numpy as np

DEGREE, RANGE = 5, 3.0


def ssp2(t: np.ndarray) -> np.ndarray:
    """log2((1 + 2^t) / 2) in float64, without cancellation around 0."""
    t = np.asarray(t, dtype=np.float64)
    return np.log1p(np.expm1(t * np.log(2.0)) / 2.0) / np.log(2.0)


def fit(degree: int = DEGREE, nodes: int = 4000, iterations: int = 200) -> np.ndarray:
    """float32 coefficients c_0 .. c_degree of (ssp2(t) - t / 2) / t^2 ~ sum_j c_j t^(2 j) on |t| <= RANGE."""
    k = np.arange(nodes)
    t = RANGE * np.sqrt((1.0 + np.cos(np.pi * (k + 0.5) / nodes)) / 2.0)
    scale = t * t / np.abs(ssp2(-t))                          # |ssp2| is smaller on the negative side
    # the even part, as the mean of the two signs: their odd parts cancel exactly
    q = (ssp2(t) + ssp2(-t)) / 2.0 / (t * t)
    small = t < 1e-2                                          # (where that mean has lost digits: the series)
    y = t * np.log(2.0)
    q[small] = ((y * y / 8.0 - y ** 4 / 192.0) / np.log(2.0) / (t * t))[small]
    A = np.vander(t * t, degree + 1, increasing=True) * scale[:, None]
    b = q * scale
    w = np.ones(nodes)
    c = np.zeros(degree + 1)
    for _ in range(iterations):
        c = np.linalg.lstsq(A * w[:, None], b * w, rcond=None)[0]
        err = np.abs(A @ c - b)
        w = w * (err / err.max()) ** 0.3 + 1e-12
        w /= w.max()
    return c.astype(np.float32)


def horner_f32(c: np.ndarray, t: np.ndarray) -> np.ndarray:
    """t (1/2 + t q(t^2)) evaluated as the device does: float32 fused multiply-adds."""
    t = t.astype(np.float32)
    s = t * t
    acc = np.full_like(t, c[-1])
    for cj in c[-2::-1]:
        acc = (acc.astype(np.float64) * s + np.float64(cj)).astype(np.float32)
    return t * (acc.astype(np.float64) * t + 0.5).astype(np.float32)


def max_rel_error(c: np.ndarray, samples: int = 2_000_000) -> float:
    """Largest relative error on |t| <= RANGE (an even number of samples: 0 is not among them)."""
    t = np.linspace(-RANGE, RANGE, samples).astype(np.float32)
    return float(np.max(np.abs(horner_f32(c, t).astype(np.float64) / ssp2(t) - 1.0)))


if __name__ == "__main__":
    c = fit()
    print(f"coefficients c0..c{DEGREE}:", ", ".join(repr(float(x)) for x in c))
    print(f"max relative error (float32 Horner): {max_rel_error(c):.3e}")
