"""Float64 restatement of the readout-tuning operators (NumPy, from the definitions in include/schnet.h):
the 8-bit feature store, readout energies and weight gradients, the preference loss.  Shares no code with
the CUDA library; used only by the tests."""
from __future__ import annotations

import numpy as np


def round_e4m3(v):
    """The e4m3 value nearest to each v (ties to the even significand; |v| <= 448): four significant bits,
    and multiples of 2^-9 below 2^-6."""
    v = np.asarray(v, dtype=np.float64)
    _, k = np.frexp(np.maximum(np.abs(v), 2.0 ** -6))       # v = m 2^k, m in [1/2, 1)
    unit = np.ldexp(1.0, k - 4)
    return np.round(v / unit) * unit


def store(x):
    """(values [n, F] = what the codes stand for, over the row's scale; exponents e [n], None where the scale is NaN)."""
    x = np.asarray(x, dtype=np.float64)
    q = np.zeros_like(x)
    e = []
    for i, row in enumerate(x):
        a = np.max(np.abs(row))
        if not a < 2.0 ** 127:                              # NaN, infinity, or too large
            e.append(None)
            continue
        k = -100
        while a > 448.0 * 2.0 ** k:
            k += 1
        e.append(k)
        q[i] = round_e4m3(row / 2.0 ** k)
    return q, e


def ssp(p):
    return np.maximum(p, 0.0) + np.log1p(np.exp(-np.abs(p))) - np.log(2.0)


def sigma(p):
    t = np.exp(-np.abs(p))
    return np.where(p >= 0, 1.0, t) / (1.0 + t)


def hidden(x, w):
    return np.asarray(x, np.float64) @ np.asarray(w["R1"], np.float64) + np.asarray(w["c1"], np.float64)


def energy(x, off, w):
    """(E [R], eps [n])."""
    eps = ssp(hidden(x, w)) @ np.asarray(w["R2"], np.float64) + float(np.asarray(w["c2"]).reshape(-1)[0])
    return np.array([eps[off[r]:off[r + 1]].sum() for r in range(len(off) - 1)]), eps


def atom_grad(n, off, g):
    """dL/d eps_i: g of the atom's replica, 0 outside all replicas."""
    out = np.zeros(n)
    for r in range(len(off) - 1):
        out[off[r]:off[r + 1]] = g[r]
    return out


def gradients(x, off, w, g):
    x = np.asarray(x, np.float64)
    gi = atom_grad(len(x), off, np.asarray(g, np.float64))
    keep = gi != 0
    x, gi = x[keep], gi[keep]
    p = hidden(x, w)
    dp = gi[:, None] * np.asarray(w["R2"], np.float64) * sigma(p)
    return {"R1": x.T @ dp, "c1": dp.sum(0), "R2": (gi[:, None] * ssp(p)).sum(0), "c2": np.array([gi.sum()])}


def preference(E, pairs, kT, ref=None, smoothing=0.0):
    """(loss, margins [P], dL/dE [R], how many pairs count)."""
    d = np.asarray(E, np.float64) - (0.0 if ref is None else np.asarray(ref, np.float64))
    m, g, total = np.zeros(len(pairs)), np.zeros(len(d)), 0.0
    ok = [p for p, (a, b) in enumerate(pairs) if 0 <= a < len(d) and 0 <= b < len(d)]
    for p in ok:
        a, b = pairs[p]
        m[p] = -(d[a] - d[b]) / kT
        up, down = np.logaddexp(0.0, -m[p]), np.logaddexp(0.0, m[p])
        total += ((1 - smoothing) * up if smoothing < 1 else 0.0) + (smoothing * down if smoothing > 0 else 0.0)
        c = (smoothing - sigma(-m[p])) / (kT * len(ok))     # sigma(m) - (1 - s)
        g[a] -= c
        g[b] += c
    return total / max(1, len(ok)), m, g, len(ok)
