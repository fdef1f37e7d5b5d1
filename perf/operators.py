"""Cases of the readout-tuning operators: the 8-bit feature store, readout energies and weight
gradients from stored features, and the preference loss over pairs of conformations.

Sizes are this library's own: 64-bead chains (F = 64), 269-bead chains (F = 128) alone, in batches of
64 and as sets of sampled frames, the 10^6-bead box.
"""
import math
import random

import numpy as np
import torch

own = False

FLOATS = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16, "fp64": torch.float64}
MAX_ATOMS = 15_600 * 269
MAX_PAIRS = 4_000_000


def listed():
    return [
        # one tiny chain's features: the launch is all
        {"name": "store chain 64", "op": "store", "n": 64, "F": 64, "stride": 64, "dtype": "fp32"},
        # one evaluation of the 64-replica batch, 16-bit features out of a wider array
        {"name": "store batch bf16", "op": "store", "n": 17_216, "F": 100, "stride": 128, "dtype": "bf16"},
        # the large box
        {"name": "store box 1M", "op": "store", "n": 1_000_000, "F": 128, "stride": 128, "dtype": "fp32"},
        # one protein-sized chain, between two sampling steps
        {"name": "energy 1 chain", "op": "energy", "R": 1, "atoms": 269, "ragged": False, "F": 128},
        # chains of uneven length, some empty, an odd hidden width
        {"name": "energy ragged F=98", "op": "energy", "R": 900, "atoms": 131, "ragged": True, "F": 98},
        # a tuning epoch over all sampled frames
        {"name": "energy 15600 frames", "op": "energy", "R": 15_600, "atoms": 269, "ragged": False, "F": 128},
        # one minibatch of the bench's 64 chains
        {"name": "gradients 64 chains", "op": "gradients", "R": 64, "atoms": 269, "ragged": False, "F": 128},
        {"name": "gradients ragged F=64", "op": "gradients", "R": 3_001, "atoms": 64, "ragged": True, "F": 64},
        {"name": "gradients 15600 frames", "op": "gradients", "R": 15_600, "atoms": 269, "ragged": False, "F": 128},
        # a minibatch of pairs among one batch's replicas, energies as the evaluation returns them
        {"name": "preference 64", "op": "preference", "R": 64, "P": 32, "dtype": "fp64", "reference": True,
         "smoothing": 0.0},
        {"name": "preference 100k", "op": "preference", "R": 15_600, "P": 100_003, "dtype": "fp32",
         "reference": True, "smoothing": 0.1},
        # every native-decoy pair of a large decoy set
        {"name": "preference 4M", "op": "preference", "R": 1_000_000, "P": 4_000_000, "dtype": "fp64",
         "reference": True, "smoothing": 0.05},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "energy", "gradients", "preference"])
    if op == "preference":
        return {"op": op, "R": _log(rng, 2, 1_000_000), "P": _log(rng, 1, MAX_PAIRS),
                "dtype": rng.choice(["fp32", "fp64"]), "reference": rng.random() < 0.7,
                "smoothing": rng.choice([0.0, 0.05, 0.1, 0.2])}
    F = rng.choice([128, 64, 2 * rng.randint(8, 64)])
    if op == "store":
        return {"op": op, "n": _log(rng, 1, 1_000_000), "F": F, "stride": F + rng.choice([0, 0, 1, 8, 28]),
                "dtype": rng.choice(["fp32", "fp16", "bf16"])}
    atoms = _log(rng, 8, 8192)
    ragged = rng.random() < 0.5
    R = _log(rng, 1, max(2, MAX_ATOMS // (3 * atoms if ragged else atoms)))
    return {"op": op, "R": R, "atoms": atoms, "ragged": ragged, "F": F}


def _offsets(case):
    """Replica offsets of a case: even chains, or lengths from empty to twice the mean."""
    if not case["ragged"]:
        return np.arange(case["R"] + 1, dtype=np.int64) * case["atoms"]
    lengths = np.random.RandomState(case["R"] * 7919 + case["atoms"]).randint(0, 2 * case["atoms"] + 1, case["R"])
    lengths[0] = max(1, lengths[0])
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def _width(F):
    return (F + 15) // 16 * 16


def _readout(case, g):
    """Readout weights as a trained model has them: Xavier range, small biases."""
    F, H = case["F"], case["F"] // 2
    u = lambda *s: torch.rand(*s, device="cuda", generator=g) * 2 - 1  # noqa: E731
    return {"R1": u(F, H) * math.sqrt(6.0 / (F + H)), "c1": u(H) * 0.1, "R2": u(H) * math.sqrt(6.0 / (H + 1)),
            "c2": u(1) * 0.1}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    if op == "store":
        x = torch.randn(case["n"], case["stride"], device="cuda", generator=g)
        x *= torch.exp(0.7 * torch.randn(case["n"], 1, device="cuda", generator=g))
        return {"case": case, "x": x.to(FLOATS[case["dtype"]])[:, :case["F"]]}
    if op == "preference":
        t = FLOATS[case["dtype"]]
        e = torch.randn(case["R"], device="cuda", generator=g, dtype=torch.float64) * 1.5 - 40.0
        ref = e + 0.5 * torch.randn(case["R"], device="cuda", generator=g, dtype=torch.float64)
        pairs = torch.randint(0, case["R"], (case["P"], 2), device="cuda", generator=g, dtype=torch.int32)
        if case["P"] > 16:
            pairs[torch.rand(case["P"], device="cuda", generator=g) < 0.02, 1] = -1  # padding
        return {"case": case, "energy": e.to(t), "reference": ref.to(t) if case["reference"] else None,
                "pairs": pairs, "kT": 0.5962}
    off = _offsets(case)
    n, F = int(off[-1]), case["F"]
    x = torch.randn(n, F, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(n, 1, device="cuda", generator=g))
    codes, scales = _store(x)
    del x
    s = {"case": case, "codes": codes, "scales": scales, **_readout(case, g),
         "offsets": torch.tensor(off, dtype=torch.int32, device="cuda")}
    if op == "gradients":
        s["grad"] = torch.randn(case["R"], device="cuda", generator=g) * (1.7 / case["R"])
    return s


def _store(x):
    """e4m3 codes [n][width] and power-of-two scales [n] of the rows of x."""
    x = x.float()
    top = x.abs().amax(1)
    m, k = torch.frexp(top)                                  # top = m 2^k, m in [1/2, 1)
    e = torch.where(m > 0.875, k - 8, k - 9).clamp(min=-100)  # the smallest with top <= 448 * 2^e
    e = torch.where(top > 0, e, -100).int()
    codes = torch.zeros(x.shape[0], _width(x.shape[1]), dtype=torch.float8_e4m3fn, device=x.device)
    codes[:, :x.shape[1]] = (x * ((127 - e) << 23).int().view(torch.float32)[:, None]).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _hidden(s):
    """Pre-activations of the readout's hidden layer, and the features."""
    x = s["codes"].float()[:, :s["R1"].shape[0]] * s["scales"].float()[:, None]
    return x, x @ s["R1"] + s["c1"]


def _ssp(p):
    return p.clamp(min=0) + torch.log1p(torch.exp(-p.abs())) - math.log(2.0)


def _replica_of(off, n):
    return torch.repeat_interleave(torch.arange(off.numel() - 1, device=off.device), (off[1:] - off[:-1]).long(),
                                   output_size=n)


def _plain(s):
    op = s["case"]["op"]
    if op == "store":
        codes, scales = _store(s["x"])
        return {"codes": codes, "scales": scales}
    if op == "preference":
        e = s["energy"].double()
        d = e - s["reference"].double() if s["reference"] is not None else e
        w, l = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
        ok = (w >= 0) & (l >= 0)
        w, l = w.clamp(min=0), l.clamp(min=0)
        m = torch.where(ok, -(d[w] - d[l]) / s["kT"], 0.0)
        t, sm = torch.log1p(torch.exp(-m.abs())), s["case"]["smoothing"]
        count = ok.sum().clamp(min=1)
        loss = torch.where(ok, (1 - sm) * ((-m).clamp(min=0) + t) + sm * (m.clamp(min=0) + t), 0.0).sum() / count
        c = torch.where(ok, 1 / (1 + torch.exp(-m)) - (1 - sm), 0.0) / (s["kT"] * count)
        grad = torch.zeros_like(d).index_add_(0, w, -c).index_add_(0, l, c)
        return {"loss": loss, "margins": m.float(), "grad": grad.float()}
    n = s["codes"].shape[0]
    x, p = _hidden(s)
    rep = _replica_of(s["offsets"], n)
    if op == "energy":
        eps = _ssp(p) @ s["R2"] + s["c2"]
        energy = torch.zeros(s["case"]["R"], dtype=torch.float64, device=x.device).index_add_(0, rep, eps.double())
        return {"energy": energy.float(), "eps": eps}
    g = s["grad"][rep]
    dp = g[:, None] * s["R2"] / (1 + torch.exp(-p))
    return {"R1": x.T @ dp, "c1": dp.double().sum(0).float(),
            "R2": (g[:, None] * _ssp(p)).double().sum(0).float(), "c2": g.double().sum().float().view(1)}


def run(state):
    if not own:
        return _plain(state)
    from schnet_gnn_molecular_b200 import api
    op = state["case"]["op"]
    if op == "store":
        codes, scales = api.store_features(state["x"])
        return {"codes": codes, "scales": scales}
    if op == "preference":
        loss, margins, grad = api.preference_loss(state["energy"], state["pairs"], kT=state["kT"],
                                                  reference=state["reference"],
                                                  smoothing=state["case"]["smoothing"])
        return {"loss": loss, "margins": margins, "grad": grad}
    readout = {k: state[k] for k in ("R1", "c1", "R2", "c2")}
    if op == "energy":
        energy, eps = api.readout_energy(state["codes"], state["scales"], state["offsets"], readout)
        return {"energy": energy, "eps": eps}
    return api.readout_gradients(state["codes"], state["scales"], state["offsets"], readout, state["grad"])


def work(case):
    op = case["op"]
    if op == "store":
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": case["n"] * (case["F"] * size + _width(case["F"]) + 1), "flops": 2 * case["n"] * case["F"]}
    if op == "preference":
        size = FLOATS[case["dtype"]].itemsize
        return {"bytes": case["P"] * 12 + case["R"] * (size * (2 if case["reference"] else 1) + 4) + 8,
                "flops": 30 * case["P"]}
    n, F, H, R = int(_offsets(case)[-1]), case["F"], case["F"] // 2, case["R"]
    weights = 4 * (F * H + 2 * H + 1)
    if op == "energy":
        return {"bytes": n * (_width(F) + 5) + 8 * R + 4 + weights, "flops": n * H * (2 * F + 8)}
    return {"bytes": n * (_width(F) + 1) + 8 * R + 4 + 2 * weights, "flops": n * H * (4 * F + 14)}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _two_to(e):
    """2^e in 64 bits, by its exponent field (a power function may round)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_store(x):
    """The stored value nearest to each x / 2^e (ties to an even significand), and 2^e, in 64 bits."""
    a = x.double().abs().max(dim=1).values
    e = torch.ceil(torch.log2(a / 448.0)).clamp(min=-100.0)
    e = torch.where(a > 448.0 * _two_to(e), e + 1, e)         # the logarithm's own rounding
    e = torch.where(a <= 448.0 * _two_to(e - 1), e - 1, e).clamp(min=-100.0)
    scale = _two_to(e)
    v = x.double() / scale[:, None]
    size = v.abs().clamp(min=2.0 ** -6)
    binade = torch.floor(torch.log2(size))
    binade = torch.where(_two_to(binade) > size, binade - 1, binade)
    binade = torch.where(_two_to(binade + 1) <= size, binade + 1, binade)
    unit = _two_to(binade - 3)
    q = torch.round(v / unit) * unit                          # rounds half to even
    out = torch.zeros(x.shape[0], _width(x.shape[1]), dtype=torch.float64, device=x.device)
    out[:, :x.shape[1]] = q
    return out, scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "store":
        codes, scales = _exact_store(s["x"])
        return {"codes": codes, "scales": scales}
    if op == "preference":
        gap = s["energy"].double()
        if s["reference"] is not None:
            gap = gap - s["reference"].double()
        keep = torch.nonzero((s["pairs"] >= 0).all(dim=1)).view(-1)
        first, second = s["pairs"][keep].long().unbind(1)
        margin = (gap[second] - gap[first]) / s["kT"]
        sm, count = case["smoothing"], max(1, keep.numel())
        loss = -((1 - sm) * torch.nn.functional.logsigmoid(margin)
                 + sm * torch.nn.functional.logsigmoid(-margin)).sum() / count
        slope = (sm - torch.sigmoid(-margin)) / count         # dL / d margin
        grad = torch.zeros_like(gap)
        grad.scatter_add_(0, second, slope / s["kT"])
        grad.scatter_add_(0, first, -slope / s["kT"])
        margins = torch.zeros(case["P"], dtype=torch.float64, device=gap.device)
        margins[keep] = margin
        return {"loss": loss, "margins": margins, "grad": grad}
    F, R = case["F"], case["R"]
    x = s["codes"].double()[:, :F] * _two_to(s["scales"].view(torch.uint8).long() - 127)[:, None]
    w = {k: s[k].double() for k in ("R1", "c1", "R2", "c2")}
    p = torch.addmm(w["c1"], x, w["R1"])
    a = torch.logaddexp(p, torch.zeros((), dtype=p.dtype, device=p.device)) - math.log(2.0)
    if op == "energy":
        eps = torch.mv(a, w["R2"]) + w["c2"]
        total = torch.cat([eps.new_zeros(1), eps.cumsum(0)])
        o = s["offsets"].long()
        return {"energy": total[o[1:]] - total[o[:-1]], "eps": eps}
    counts = torch.diff(s["offsets"].long())
    g = torch.repeat_interleave(s["grad"].double(), counts)
    dp = torch.sigmoid(p) * w["R2"] * g[:, None]
    return {"R1": torch.mm(x.T, dp), "c1": torch.mv(dp.T, torch.ones_like(g)), "R2": torch.mv(a.T, g),
            "c2": torch.dot(s["grad"].double(), counts.double()).view(1)}


if __name__ == "__main__":
    for c in listed():
        print(c["name"], work(c))
    print(draw(random.Random(0)))
