"""Problems and error bounds shared by the tight GPU tests of the readout-tuning kernels and the CPU tests that show
what those bounds would notice.  u = 2^-24.

Tensor-core sums: the products of one K = 16 step and the accumulator are aligned to the largest of them and cut
off, at most 2u of it each, so a step errs by at most 17 * 2u * M, M the largest accumulator or product on the way."""
from __future__ import annotations

import numpy as np

from oracle import tuning

U = 2.0 ** -24
STEP = 17 * 2 * U


def stored(x):
    """(values, scales) that the 8-bit store keeps of the rows of x, in float64."""
    x = np.asarray(x, dtype=np.float64)
    m, k = np.frexp(np.abs(x).max(1))                        # a = m 2^k, m in [1/2, 1); 448 = 0.875 * 2^9
    scale = np.ldexp(1.0, np.maximum(np.where(m > 0.875, k - 8, k - 9), -100))[:, None]
    return tuning.round_e4m3(x / scale) * scale, scale[:, 0]


def weights(F, rng, scale=1.0):
    H = F // 2
    return {"R1": (rng.normal(size=(F, H)) * scale / np.sqrt(F)).astype(np.float32),
            "c1": (0.3 * scale * rng.normal(size=H)).astype(np.float32),
            "R2": rng.normal(size=H).astype(np.float32), "c2": rng.normal(size=1).astype(np.float32)}


def preactivation(x, w):
    """(p, bound on its error): F / 16 steps on R1's leading fp16 terms; as many on the rests, 2^-11 of them; R1 itself
    to 2^-22; the row's factor, c1 log2 e and their sum to 4u."""
    R1, c1 = w["R1"].astype(np.float64), w["c1"].astype(np.float64)
    n, F = x.shape
    p = np.zeros((n, R1.shape[1]))
    top = np.abs(x).max(1)[:, None] * np.abs(R1).max(0)       # no product is larger
    for f in range(0, F, 16):
        p += x[:, f:f + 16] @ R1[f:f + 16]
        np.maximum(top, np.abs(p), out=top)
    steps = (F + 15) // 16
    size = np.abs(x) @ np.abs(R1)
    b = steps * STEP * top + (steps * STEP * 2.0 ** -11 + 2.0 ** -22) * size + 4 * U * (np.abs(p) + np.abs(c1))
    return p + c1, b


def unit_energy(x, w, h):
    """(eps, bound) with R2 the unit vector h and c2 = 0: one hidden unit, so that no error hides in the sum."""
    one = {"R1": w["R1"][:, h:h + 1], "c1": w["c1"][h:h + 1]}
    p, b = preactivation(x, one)
    p, b = p[:, 0], b[:, 0]
    return tuning.ssp(p), b + 2.0 ** -20 * (1 + np.abs(p)) + 4 * U * np.abs(tuning.ssp(p))


def once_rounded(R1):
    """R1 as the leading fp16 term alone, scaled as the kernels scale it (a planted mistake)."""
    s = 14 - (int(np.floor(np.log2(np.abs(R1).max()))))
    return np.ldexp(np.ldexp(R1.astype(np.float64), s).astype(np.float16).astype(np.float64), -s)
