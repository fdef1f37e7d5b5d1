"""Problems and error bounds shared by the tight GPU tests of the readout-tuning kernels and the CPU tests that show
what those bounds would notice.  u = 2^-24.

Tensor-core sums: the products of one K = 16 step and the accumulator are aligned to the largest of them and cut
off, at most 2u of it each, so a step errs by at most 17 * 2u * M, M the largest accumulator or product on the way."""
from __future__ import annotations

import numpy as np

import oracle
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


class GradientProblem:
    """Many tiles of 128 atoms with seeds of one size (+-1 a replica of 131 atoms): whatever a single tile adds is
    larger than the bound on the sum's error."""

    def __init__(self, F, n=300_007, seed=0):
        rng = np.random.default_rng(seed + F)
        self.F, self.n = F, n
        self.x32 = rng.normal(size=(n, F)).astype(np.float32)
        self.x, self.scale = stored(self.x32)
        self.w = weights(F, rng, scale=0.25)
        self.off = np.array([0, *range(11, n, 131), n], dtype=np.int32)
        self.g = rng.choice([-1.0, 1.0], size=len(self.off) - 1).astype(np.float32)
        gi = tuning.atom_grad(n, self.off, self.g.astype(np.float64))
        r2 = self.w["R2"].astype(np.float64)
        tiles = (n + 127) // 128
        H = F // 2
        bR1, bsig, bssp = np.zeros((F, H)), np.zeros(H), np.zeros(H)      # sums over the atoms: errors of sigma and ssp,
        asig, assp = np.zeros(H), np.zeros(H)                             # and their magnitudes
        self.tR1 = np.zeros((tiles, F, H))                    # what each tile adds
        self.tc1, self.tR2 = np.zeros((tiles, H)), np.zeros((tiles, H))
        aR1 = np.zeros((F, H))                                # largest sum of magnitudes over a tile
        for a in range(0, tiles, 128):
            t = slice(a, min(a + 128, tiles))
            i = slice(a * 128, min((a + 128) * 128, n))
            x, s = self.x[i], gi[i][:, None]
            p, b = preactivation(x, self.w)
            sig, ssp = tuning.sigma(p), tuning.ssp(p)
            e = b / 4 + 2.0 ** -20
            bR1 += np.abs(x).T @ (e + 2.0 ** -22 * sig)
            bsig += e.sum(0)
            bssp += (b + 2.0 ** -20 * (1 + np.abs(p))).sum(0)
            asig += sig.sum(0)
            assp += np.abs(ssp).sum(0)
            rows = (t.stop - t.start) * 128

            def by_tile(v):
                return np.concatenate([v, np.zeros((rows - len(v), v.shape[1]))]).reshape(-1, 128, v.shape[1])

            X, S, P = by_tile(x), by_tile(s * sig), by_tile(s * ssp)
            self.tR1[t] = X.transpose(0, 2, 1) @ S
            aR1 = np.maximum(aR1, (np.abs(X).transpose(0, 2, 1) @ np.abs(S)).max(0))
            self.tc1[t], self.tR2[t] = S.sum(1), P.sum(1)
        # an accumulator takes at most 8 tiles: the largest it gets, and what a step cuts off
        c = np.concatenate([np.zeros((1, F, H)), np.cumsum(self.tR1, 0)])
        top = aR1.copy()
        for k in range(1, 9):
            top = np.maximum(top, np.abs(c[k:] - c[:-k]).max(0) + aR1)
        floor = 2.0 ** -34 * self.scale.max() * (np.abs(self.x) / self.scale[:, None]).sum(0)[:, None]
        # then float32 sums of a CTA's accumulators (at most one in 8 tiles and two a CTA of 148)
        adds = (tiles / 8 + 2 * 148) * 2 * U * 4 * top
        self.want = {"R1": self.tR1.sum(0) * r2, "c1": self.tc1.sum(0) * r2, "R2": self.tR2.sum(0),
                     "c2": np.array([gi.sum()])}
        last = {k: 2 * U * np.abs(v) for k, v in self.want.items()}
        # the column sums: at most 32 tiles and 5 shuffles in float32, then float64
        self.tol = {"R1": np.abs(r2) * (bR1 + tiles * 8 * STEP * (1 + 2.0 ** -10) * top + adds + floor) + last["R1"],
                    "c1": np.abs(r2) * (bsig + 38 * U * asig) + last["c1"],
                    "R2": bssp + 38 * U * assp + last["R2"], "c2": last["c2"]}
        self.r2 = r2

    def noticed(self):
        """Per tile: whether leaving it out would exceed the bound of dR1, and of dc1 or dR2."""
        R1 = (np.abs(self.tR1 * self.r2) > 2 * self.tol["R1"]).any((1, 2))
        sums = (np.abs(self.tc1 * self.r2) > 2 * self.tol["c1"]).any(1) | (np.abs(self.tR2) > 2 * self.tol["R2"]).any(1)
        return R1, sums


def trunk(model: oracle.Model, pos, types, replica_offsets):
    """The interaction blocks' output x^L in float64: x += ssp(m Wo1 + bo1) Wo2 + bo2 with m the oracle's aggregation."""
    w = {k: np.asarray(v, dtype=np.float64) for k, v in model.weights.items()}
    x = w["emb"][types].copy()
    for l in range(model.L):
        m = oracle.cfconv(model, l, pos, x @ w["W_in"][l], replica_offsets)
        x += tuning.ssp(m @ w["Wo1"][l] + w["bo1"][l]) @ w["Wo2"][l] + w["bo2"][l]
    return x


def row_bound(x, scale):
    """How far stored features may be from the trunk's x: half a step of e4m3 (2^-4 of the value, or 2^-10 of the row's
    scale) beside 1e-4 of the row's largest for the trunk's own single precision."""
    d = 1e-4 * np.abs(x).max(1)[:, None]
    return np.maximum(2.0 ** -4 * (np.abs(x) + d), 2.0 ** -10 * scale[:, None]) + d
