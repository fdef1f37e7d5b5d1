"""Readout tuning on the GPU against the float64 oracle: the 8-bit feature store, readout energies and weight
gradients, the preference loss, and a run of them together with a context.

Tolerances (u = 2^-24).  The stored features are exact inputs of the readout.  A hidden pre-activation is a sum of F
products of them with R1, carried to 2^-22 or better and accumulated in fp32, on the tensor cores without rounding to
nearest (up to 2u a step, at most 2 F / 16 + F steps): |dp| <= (2 F + 16) 2u (|x| |R1| + |c1|) =: b.  ssp and sigma
have slopes of at most 1 and 1/4 and are formed from a base-2 exponential and logarithm good to 2^-22, so to
2^-20 (1 + |p|).  Sums over atoms are chains of at most 512 roundings (longer ones are cut into partial sums)."""
import ctypes as C
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import tuning
from schnet_gnn_molecular_b200 import _native as nat
from schnet_gnn_molecular_b200 import api, workloads

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype).cuda()


# ---------------------------------------------------------------- store
def _check_store(x, codes, scales):
    """x: the values given, float64 numpy [n, F]."""
    n, F = x.shape
    q, e = tuning.store(x)
    c = codes.float().cpu().numpy().astype(np.float64)
    b = scales.view(torch.uint8).cpu().numpy()
    assert c.shape == (n, (F + 15) // 16 * 16) and not c[:, F:].any()
    assert np.array_equal(c[:, :F], q)
    assert b.tolist() == [255 if k is None else k + 127 for k in e]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("F,n", [(2, 1), (6, 5), (16, 33), (50, 129), (64, 64), (98, 1000), (126, 7), (128, 4099)])
def test_store_is_the_rounding(dtype, F, n):
    g = torch.Generator().manual_seed(F * 1000 + n)
    x = torch.randn(n, F, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g))
    x[n // 2] = 0
    x = x.to(dtype)
    codes, scales = api.store_features(x.cuda())
    _check_store(x.double().numpy(), codes, scales)


@pytest.mark.parametrize("shift,wide", [(0, 0), (1, 0), (0, 4), (3, 7), (4, 28)])
def test_store_strides(shift, wide):
    F, n = 60, 300
    base = torch.randn(n, F + shift + wide, generator=torch.Generator().manual_seed(5))
    x = base.cuda()[:, shift:shift + F]
    codes, scales = api.store_features(x)
    _check_store(base[:, shift:shift + F].double().numpy(), codes, scales)


def test_store_odd_rows():
    x = torch.randn(12, 32, generator=torch.Generator().manual_seed(6))
    x[0] = 0.0
    x[1, 3] = float("nan")
    x[2, 31] = float("inf")
    x[3, 0] = -float("inf")
    x[4] = 448.0
    x[5, 1] = 2.0 ** 127
    x[6, 1] = -(2.0 ** 126)
    x[7] *= 2.0 ** -120
    x[8] = torch.finfo(torch.float32).tiny / 4      # subnormal
    x[9] *= 2.0 ** 100
    codes, scales = api.store_features(x.cuda())
    _check_store(x.double().numpy(), codes, scales)


def test_store_of_no_rows():
    codes, scales = api.store_features(torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 64) and scales.shape == (0,)
    with pytest.raises(ValueError):
        api.store_features(torch.randn(64, 64, device="cuda").t())
    with pytest.raises(ValueError):
        api.store_features(torch.randn(4, 64, device="cuda").double())
    with pytest.raises(api.SchNetError):
        api.store_features(torch.randn(4, 63, device="cuda"))


# ---------------------------------------------------------------- readout
LAYOUTS = {
    "one atom": (1, [0, 1]),
    "one replica": (269, [0, 269]),
    "empty ones": (300, [0, 0, 100, 100, 100, 299, 300, 300]),
    "outside": (400, [37, 130, 130, 260]),
    "none": (70, [5, 5]),
    "ragged": (1013, [0, 1, 3, 130, 258, 259, 640, 641, 1000, 1013]),
    "long": (40_003, [0, 20_000, 20_001, 40_003]),
    "many": (9_000, list(range(0, 9_001, 3))),
}


def _weights(F, rng, scale=1.0):
    H = F // 2
    return {"R1": (rng.normal(size=(F, H)) * scale / np.sqrt(F)).astype(np.float32),
            "c1": (0.3 * rng.normal(size=H)).astype(np.float32), "R2": rng.normal(size=H).astype(np.float32),
            "c2": rng.normal(size=1).astype(np.float32)}


def _stored(n, F, rng):
    """Stored features and the values that they stand for (float64)."""
    x = (rng.normal(size=(n, F)) * np.exp(0.7 * rng.normal(size=(n, 1)))).astype(np.float32)
    codes, scales = api.store_features(_dev(x))
    v = codes.double().cpu().numpy()[:, :F] * scales.double().cpu().numpy()[:, None]
    return codes, scales, v


def _dw(w):
    return {k: _dev(v) for k, v in w.items()}


def _bounds(x, w):
    F = x.shape[1]
    p = tuning.hidden(x, w)
    b = (2 * F + 16) * 2 * U * (np.abs(x) @ np.abs(w["R1"].astype(np.float64)) + np.abs(w["c1"]))
    fn = 2.0 ** -20 * (1 + np.abs(p))
    r2 = np.abs(w["R2"].astype(np.float64))
    eps = (b + fn) @ r2 + 2 * (F // 2 + 2) * U * (np.abs(tuning.ssp(p)) @ r2 + abs(float(w["c2"][0])))
    return p, b, fn, eps


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("F", [2, 18, 64, 98, 128])
def test_readout_energy(layout, F):
    n, off = LAYOUTS[layout]
    rng = np.random.default_rng(n + F)
    codes, scales, x = _stored(n, F, rng)
    w = _weights(F, rng)
    E, eps = api.readout_energy(codes, scales, _dev(off, torch.int32), _dw(w))
    want_E, want = tuning.energy(x, off, w)
    tol = _bounds(x, w)[3]
    assert np.all(np.abs(eps.cpu().numpy() - want) <= tol)
    for r in range(len(off) - 1):
        assert abs(float(E[r]) - want_E[r]) <= tol[off[r]:off[r + 1]].sum() + U * abs(want_E[r])


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("F", [2, 18, 64, 98, 128])
def test_readout_gradients(layout, F):
    n, off = LAYOUTS[layout]
    rng = np.random.default_rng(n + F + 1)
    codes, scales, x = _stored(n, F, rng)
    w = _weights(F, rng)
    g = (rng.normal(size=len(off) - 1) * np.exp(3 * rng.normal(size=len(off) - 1))).astype(np.float32)
    if len(g) > 4:
        g[3] = 0
    got = api.readout_gradients(codes, scales, _dev(off, torch.int32), _dw(w), _dev(g))
    want = tuning.gradients(x, off, w, g)
    p, b, fn, _ = _bounds(x, w)
    gi = np.abs(tuning.atom_grad(n, off, g))
    r2 = np.abs(w["R2"].astype(np.float64))
    chain = 512 * 2 * U
    ddp = gi[:, None] * r2 * (b / 4 + fn)
    adp = gi[:, None] * r2 * tuning.sigma(p)
    aga = gi[:, None] * np.abs(tuning.ssp(p))
    tol = {"R1": np.abs(x).T @ (ddp + chain * adp), "c1": (ddp + chain * adp).sum(0),
           "R2": (gi[:, None] * (b + fn) + chain * aga).sum(0), "c2": np.array([chain * gi.sum()])}
    for k in want:
        # what the running scale of dp keeps: 2^-34 of the largest term
        floor = 2.0 ** -30 * (adp.max() if adp.size else 0) * max(1.0, np.abs(x).max()) * max(1, (gi != 0).sum())
        assert np.all(np.abs(got[k].cpu().numpy() - want[k]) <= tol[k] + floor), (k, layout)


@pytest.mark.parametrize("scale", [1e-12, 1e-4, 1e6])
def test_gradients_keep_their_precision_at_any_scale(scale):
    rng = np.random.default_rng(8)
    codes, scales, x = _stored(700, 64, rng)
    off = [0, 300, 700]
    w = _weights(64, rng)
    g = (np.array([1.0, -0.3]) * scale).astype(np.float32)
    got = api.readout_gradients(codes, scales, _dev(off, torch.int32), _dw(w), _dev(g))
    want = tuning.gradients(x, off, w, g)
    for k in want:
        assert np.linalg.norm(got[k].cpu().numpy() - want[k]) <= 2e-5 * np.linalg.norm(want[k]), k


def test_large_and_saturated_hidden_layers():
    rng = np.random.default_rng(9)
    codes, scales, x = _stored(500, 128, rng)
    w = _weights(128, rng, scale=200.0)                       # pre-activations in the hundreds, both signs
    off = [0, 500]
    E, eps = api.readout_energy(codes, scales, _dev(off, torch.int32), _dw(w))
    assert np.all(np.abs(eps.cpu().numpy() - tuning.energy(x, off, w)[1]) <= _bounds(x, w)[3])
    got = api.readout_gradients(codes, scales, _dev(off, torch.int32), _dw(w), _dev(np.ones(1, np.float32)))
    want = tuning.gradients(x, off, w, [1.0])
    for k in want:
        assert np.linalg.norm(got[k].cpu().numpy() - want[k]) <= 1e-4 * np.linalg.norm(want[k]), k


def test_no_atoms():
    w = _dw(_weights(64, np.random.default_rng(0)))
    codes = torch.empty(0, 64, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(0, dtype=torch.float8_e8m0fnu, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    E, eps = api.readout_energy(codes, scales, off, w)
    assert E.tolist() == [0.0] * 3 and eps.numel() == 0
    got = api.readout_gradients(codes, scales, off, w, torch.ones(3, device="cuda"))
    assert all(not v.any() for v in got.values())


def test_offsets_out_of_range_are_read_as_the_ends():
    rng = np.random.default_rng(10)
    codes, scales, x = _stored(200, 64, rng)
    w = _weights(64, rng)
    a = api.readout_energy(codes, scales, _dev([-7, 90, 10_000], torch.int32), _dw(w))
    b = api.readout_energy(codes, scales, _dev([0, 90, 200], torch.int32), _dw(w))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    g = _dev(np.array([1.0, 2.0], np.float32))
    a = api.readout_gradients(codes, scales, _dev([-7, 90, 10_000], torch.int32), _dw(w), g)
    b = api.readout_gradients(codes, scales, _dev([0, 90, 200], torch.int32), _dw(w), g)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_nan_rows_stay_in_their_replica():
    rng = np.random.default_rng(11)
    x = rng.normal(size=(400, 64)).astype(np.float32)
    x[130, 7] = np.nan
    codes, scales = api.store_features(_dev(x))
    w, off = _dw(_weights(64, rng)), _dev([0, 120, 260, 400], torch.int32)
    E, eps = api.readout_energy(codes, scales, off, w)
    assert torch.isnan(E).tolist() == [False, True, False] and torch.isnan(eps).nonzero().view(-1).tolist() == [130]
    clean = api.readout_gradients(codes, scales, off, w, _dev(np.array([1, 0, -1], np.float32)))
    assert all(torch.isfinite(v).all() for v in clean.values())
    bad = api.readout_gradients(codes, scales, off, w, _dev(np.array([1, 1, -1], np.float32)))
    assert torch.isnan(bad["R1"]).all() and torch.isnan(bad["c1"]).all() and torch.isnan(bad["R2"]).all()


@pytest.mark.parametrize("name,value", [("R1", np.nan), ("R1", np.inf), ("c1", np.nan), ("c1", -np.inf)])
def test_nonfinite_weights_make_everything_nan(name, value):
    rng = np.random.default_rng(15)
    codes, scales, _ = _stored(300, 64, rng)
    w = _weights(64, rng)
    w[name].reshape(-1)[5] = value
    off, g = _dev([0, 100, 300], torch.int32), _dev(np.array([1.0, -1.0], np.float32))
    E, eps = api.readout_energy(codes, scales, off, _dw(w))
    assert torch.isnan(E).all() and torch.isnan(eps).all()
    got = api.readout_gradients(codes, scales, off, _dw(w), g)
    assert torch.isnan(got["R1"]).all() and torch.isnan(got["c1"]).all() and torch.isnan(got["R2"]).all()


def test_tiny_and_huge_weights():
    rng = np.random.default_rng(16)
    codes, scales, x = _stored(300, 64, rng)
    off = [0, 100, 300]
    for scale in (1e-20, 1e-6, 1e6):
        w = _weights(64, rng, scale=scale)
        E, eps = api.readout_energy(codes, scales, _dev(off, torch.int32), _dw(w))
        assert np.all(np.abs(eps.cpu().numpy() - tuning.energy(x, off, w)[1]) <= _bounds(x, w)[3])
    zero = {k: np.zeros_like(v) for k, v in w.items()}
    E, eps = api.readout_energy(codes, scales, _dev(off, torch.int32), _dw(zero))
    assert not eps.any() and not E.any()
    got = api.readout_gradients(codes, scales, _dev(off, torch.int32), _dw(zero), _dev(np.ones(2, np.float32)))
    assert not got["R1"].any() and not got["c1"].any() and float(got["c2"]) == 300 and not got["R2"].any()


@pytest.mark.parametrize("F", [18, 64, 128])
@pytest.mark.parametrize("zero", ["weights", "features"])
def test_hidden_layers_of_zero_add_nothing_to_dR2(F, zero):
    """ssp(0) = 0: whatever the seeds, no term of dR2 is left."""
    rng = np.random.default_rng(F)
    codes, scales, _ = _stored(30_000, F, rng)
    w = _weights(F, rng)
    w["c1"][:] = 0
    if zero == "weights":
        w["R1"][:] = 0
    else:
        codes, scales = api.store_features(torch.zeros(30_000, F, device="cuda"))
    off = list(range(0, 30_001, 30))
    g = (rng.normal(size=1000) * np.exp(2 * rng.normal(size=1000))).astype(np.float32)
    got = api.readout_gradients(codes, scales, _dev(off, torch.int32), _dw(w), _dev(g))
    assert not got["R2"].any()


@pytest.mark.parametrize("n", [1000, 500_009])                  # up to 9 tiles a group: looked at twice
@pytest.mark.parametrize("F", [18, 64, 128])
def test_energies_of_small_activations(F, n):
    """p = c1 from 1e-6 to 2 in size, one hidden unit at a time: eps to 2e-7 (the activation) and 4u (c1 log2 e and its
    product, R2 ln2 and its), E to u more."""
    rng = np.random.default_rng(F)
    H = F // 2
    codes, scales, _ = _stored(n, F, rng)
    w = _weights(F, rng)
    w["R1"][:] = 0
    w["c1"] = (np.geomspace(1e-6, 2.0, H) * np.where(np.arange(H) % 2, 1, -1)).astype(np.float32)
    w["c2"][:] = 0
    p = w["c1"].astype(np.float64)
    want = np.log1p(np.expm1(p) / 2.0)                                   # ssp(p) without cancellation
    for h in range(H) if n == 1000 else (0, H // 2, H - 1):
        w["R2"] = np.eye(H, dtype=np.float32)[h]
        E, eps = api.readout_energy(codes, scales, _dev([0, n], torch.int32), _dw(w))
        assert np.all(np.abs(eps.cpu().numpy() - want[h]) <= (2e-7 + 4 * U) * abs(want[h])), h
        assert abs(float(E[0]) - n * want[h]) <= (2e-7 + 5 * U) * n * abs(want[h]), h


@pytest.mark.parametrize("F", [18, 64, 128])
def test_dR2_of_small_activations(F):
    """p = c1 from 1e-6 to 2 in size: each term of dR2 to 2e-7 (the activation) and 3u (c1 log2 e and its product),
    their sum to the u of at most 32 + 5 float32 additions before float64 takes over, and u at the end."""
    rng = np.random.default_rng(F)
    n, H = 50_000, F // 2
    codes, scales, _ = _stored(n, F, rng)
    w = _weights(F, rng)
    w["R1"][:] = 0
    w["c1"] = (np.geomspace(1e-6, 2.0, H) * np.where(np.arange(H) % 2, 1, -1)).astype(np.float32)
    off = [0, 20_000, n]
    g = np.array([1.0, 0.75], np.float32)
    got = api.readout_gradients(codes, scales, _dev(off, torch.int32), _dw(w), _dev(g))["R2"].cpu().numpy()
    p = w["c1"].astype(np.float64)
    want = (20_000 + 0.75 * 30_000) * np.log1p(np.expm1(p) / 2.0)        # ssp(p) without cancellation
    assert np.all(np.abs(got - want) <= (2e-7 + 41 * U) * np.abs(want))


@pytest.mark.parametrize("F", [64, 128])
@pytest.mark.parametrize("ex", [125, 126, 127])
def test_weights_near_the_largest_finite(F, ex):
    """|R1| in [2^ex, 2^(ex+1)), features of a few 2^-109: pre-activations of +-2^17 to 2^27, one sign a unit."""
    rng = np.random.default_rng(ex)
    n, H, off = 300, F // 2, [0, 100, 300]
    x = np.ldexp(rng.integers(0, 8, size=(n, F)).astype(np.float64), -109)
    codes, scales = api.store_features(_dev(x.astype(np.float32)))
    w = _weights(F, rng)
    sign = np.where(np.arange(H) % 3 == 0, -1.0, 1.0)
    w["R1"] = (np.ldexp(rng.uniform(1.0, 1.99, size=(F, H)), ex) * sign).astype(np.float32)
    E, eps = api.readout_energy(codes, scales, _dev(off, torch.int32), _dw(w))
    want_E, want = tuning.energy(x, off, w)
    tol = _bounds(x, w)[3]
    assert np.all(np.abs(eps.cpu().numpy() - want) <= tol)
    for r in range(2):
        assert abs(float(E[r]) - want_E[r]) <= tol[off[r]:off[r + 1]].sum() + U * abs(want_E[r])
    # one seed and one sign a unit: nothing cancels.  n / 16 steps of 17 terms, each cut off by 2u of the sum at most,
    # beside the pre-activation's (2 F + 16) 2u and the functions' 2^-20
    got = api.readout_gradients(codes, scales, _dev(off, torch.int32), _dw(w), _dev(np.ones(2, np.float32)))
    want = tuning.gradients(x, off, w, np.ones(2))
    rel = (n / 16 + 1) * 17 * 2 * U + (2 * F + 16) * 2 * U + 2.0 ** -20
    for k in want:
        # where a unit's pre-activations are negative: ssp's 2^-20 (1 + |p|); sigma is not below 2^-126
        floor = n * 2.0 ** -20 * (1 + np.abs(tuning.hidden(x, w)).max(0)) if k == "R2" else n * 2.0 ** -125 * 4
        assert np.all(np.abs(got[k].cpu().numpy() - want[k]) <= rel * np.abs(want[k]) + floor), k


# A group of the energies' kernel takes 9 tiles, a CTA of the gradients' 27: the kernels' rings of stages, operands and
# accumulators go round, and layers with fewer units than the upper warps hold run beside full ones.
LAYOUTS["tiles"] = (500_009, [0, *range(11, 500_000, 131), 500_009])


@pytest.mark.parametrize("F", [2, 32, 62, 64, 66, 94, 128])
def test_many_tiles(F):
    test_readout_energy("tiles", F)
    test_readout_gradients("tiles", F)


@pytest.mark.parametrize("n,R", [(1, 1), (5000, 3), (100_000, 3), (300, 900)])
def test_a_wait_that_gives_up_makes_every_result_nan(n, R):
    lib = nat.load()
    need = C.c_size_t(0)
    assert lib.schnet_readout_workspace_bytes(n, 128, C.byref(need)) == 0
    off = _dev(np.linspace(0, n, R + 1).astype(np.int32))
    ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    p = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    for given_up in (0, 1):
        E, eps = torch.ones(R, device="cuda"), torch.ones(n, device="cuda")
        assert lib.schnet_test_readout_timeout(n, R, p(off), given_up, p(E), p(eps), p(ws), need.value, stream) == 0
        assert torch.isnan(E).all() == bool(given_up) and torch.isnan(eps).all() == bool(given_up)
        if not given_up:
            assert torch.isfinite(E).all() and torch.equal(eps, torch.ones_like(eps))


def test_same_inputs_same_bits():
    rng = np.random.default_rng(12)
    codes, scales, _ = _stored(30_000, 128, rng)
    w, off = _dw(_weights(128, rng)), _dev(list(range(0, 30_001, 250)), torch.int32)
    g = _dev(rng.normal(size=120).astype(np.float32))
    first = api.readout_energy(codes, scales, off, w), api.readout_gradients(codes, scales, off, w, g)
    for _ in range(3):
        again = api.readout_energy(codes, scales, off, w), api.readout_gradients(codes, scales, off, w, g)
        assert torch.equal(first[0][0], again[0][0]) and torch.equal(first[0][1], again[0][1])
        assert all(torch.equal(first[1][k], again[1][k]) for k in first[1])


def test_binding_refusals():
    rng = np.random.default_rng(13)
    codes, scales, _ = _stored(40, 64, rng)
    w, off = _dw(_weights(64, rng)), _dev([0, 40], torch.int32)
    for bad in (dict(w, R1=w["R1"].double()), dict(w, R1=w["R1"].t()), dict(w, c1=w["c1"][:-1]),
                dict(w, c2=w["c1"]), dict(w, R2=w["R2"].cpu())):
        with pytest.raises(ValueError):
            api.readout_energy(codes, scales, off, bad)
    with pytest.raises(ValueError):
        api.readout_energy(codes, scales, off.long(), w)
    with pytest.raises(ValueError):
        api.readout_energy(codes[:, :32], scales, off, w)
    with pytest.raises(ValueError):
        api.readout_energy(codes, scales[:-1], off, w)
    with pytest.raises(ValueError):
        api.readout_gradients(codes, scales, off, w, torch.ones(2, device="cuda"))


# ---------------------------------------------------------------- preference loss
def _check_preference(E, pairs, kT, ref, s, got):
    loss, m, g = got
    wl, wm, wg, count = tuning.preference(E, pairs, kT, ref, s)
    assert abs(float(loss) - wl) <= 1e-12 * max(1.0, abs(wl))
    assert np.all(np.abs(m.cpu().numpy() - wm) <= 2 * U * np.abs(wm))
    # the sums are exact to 2^-25 of their terms; one rounding to fp32
    part = np.zeros(len(wg))
    for a, b in pairs:
        if 0 <= a < len(wg) and 0 <= b < len(wg):
            part[a] += 1
            part[b] += 1
    assert np.all(np.abs(g.cpu().numpy() - wg) <= U * np.abs(wg) + part * 2.0 ** -25 / (kT * max(count, 1)))


@pytest.mark.parametrize("dtype", [np.float32, np.float64])
@pytest.mark.parametrize("R,P,with_ref,s", [(1, 1, False, 0.0), (2, 1, True, 0.0), (64, 32, True, 0.1),
                                            (300, 5000, True, 0.0), (5000, 300, False, 0.3), (7, 4000, True, 1.0),
                                            (70_000, 20_001, True, 0.05)])
def test_preference(dtype, R, P, with_ref, s):
    rng = np.random.default_rng(R + P)
    E = (rng.normal(size=R) * 2 - 30).astype(dtype)
    ref = (E + rng.normal(size=R)).astype(dtype) if with_ref else None
    pairs = rng.integers(0, R, size=(P, 2)).astype(np.int32)
    if P > 20:
        pairs[3] = (-1, 0)
        pairs[5] = (0, -1)
        pairs[6] = (-1, -1)
        pairs[8] = pairs[7]
        pairs[9] = (1 % R, 1 % R)
    flags = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    got = api.preference_loss(_dev(E), _dev(pairs), kT=0.6, reference=None if ref is None else _dev(ref), smoothing=s,
                              flags=flags)
    _check_preference(E, pairs.tolist(), 0.6, ref, s, got)
    assert int(flags) == 0
    again = api.preference_loss(_dev(E), _dev(pairs), kT=0.6, reference=None if ref is None else _dev(ref),
                                smoothing=s)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_preference_without_pairs():
    E = torch.randn(5, device="cuda")
    for pairs in (torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.full((9, 2), -1, dtype=torch.int32).cuda()):
        loss, m, g = api.preference_loss(E, pairs, kT=1.0)
        assert float(loss) == 0 and not m.any() and not g.any()


def test_preference_extremes():
    E = np.array([0.0, 800.0, 1e6, -1e6, 30.0, 60.0])
    pairs = [(0, 1), (1, 0), (2, 3), (3, 2), (4, 5), (5, 4)]
    got = api.preference_loss(_dev(E), _dev(pairs, torch.int32), kT=1.0)
    _check_preference(E, pairs, 1.0, None, 0.0, got)
    # one pair far on the right side: its slope, e^-40, is kept to the gradient's own precision
    loss, _, g = api.preference_loss(_dev(np.array([0.0, 40.0])), _dev([(0, 1)], torch.int32), kT=1.0)
    assert abs(float(g[0]) - np.exp(-40.0)) <= 2.0 ** -23 * np.exp(-40.0) and float(loss) > 0
    E = _dev(np.array([0.0, np.inf, 1.0]))
    loss, m, g = api.preference_loss(E, _dev([(0, 1)], torch.int32), kT=1.0)
    assert float(loss) == 0 and float(m[0]) == np.inf and not g.any()
    loss, m, g = api.preference_loss(E, _dev([(1, 0)], torch.int32), kT=2.0)
    assert float(loss) == np.inf and g.tolist() == [-0.5, 0.5, 0.0]


def test_preference_flags():
    E = _dev(np.array([0.0, 1.0, np.nan, 2.0]))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, m, g = api.preference_loss(E, _dev([(0, 1), (4, 0), (0, -2), (3, 2_000_000)], torch.int32), kT=1.0, flags=flags)
    assert int(flags) == nat.FLAG_BADINDEX
    one = api.preference_loss(E, _dev([(0, 1)], torch.int32), kT=1.0, flags=flags)
    assert int(flags) == 0 and float(one[0]) == float(loss) and torch.equal(one[2], g) and not m[1:].any()
    loss, m, g = api.preference_loss(E, _dev([(0, 1), (2, 3)], torch.int32), kT=1.0, flags=flags)
    assert int(flags) == nat.FLAG_NONFINITE and np.isnan(float(loss))
    assert torch.isnan(g).tolist() == [False, False, True, True] and torch.isnan(m).tolist() == [False, True]


def test_preference_binding_refusals():
    E, pairs = torch.randn(5, device="cuda"), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    for kw in (dict(reference=E.double()), dict(reference=E[:4]), dict(flags=torch.zeros(2, dtype=torch.int32).cuda())):
        with pytest.raises(ValueError):
            api.preference_loss(E, pairs, kT=1.0, **kw)
    for e, p in ((E.half(), pairs), (E, pairs.long()), (E, pairs.t()[:1]), (E.cpu(), pairs), (E[::2], pairs)):
        with pytest.raises(ValueError):
            api.preference_loss(e, p, kT=1.0)
    for kw in (dict(kT=0.0), dict(kT=1.0, smoothing=2.0)):
        with pytest.raises(api.SchNetError):
            api.preference_loss(E, pairs, **kw)


# ---------------------------------------------------------------- streams and graphs
def test_side_stream_and_captured_graph():
    rng = np.random.default_rng(14)
    x = rng.normal(size=(1076, 128)).astype(np.float32)
    off, w = _dev([0, 269, 538, 807, 1076], torch.int32), _dw(_weights(128, rng))
    pairs = _dev([(0, 1), (2, 3), (3, 0)], torch.int32)

    def step(x):
        codes, scales = api.store_features(x)
        E, eps = api.readout_energy(codes, scales, off, w)
        loss, _, g = api.preference_loss(E, pairs, kT=0.6)
        return loss, E, api.readout_gradients(codes, scales, off, w, g)

    def same(a, b):
        return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(a[2][k], b[2][k]) for k in a[2])

    xd = _dev(x)
    want = step(xd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step(xd)
    side.synchronize()
    assert same(want, got)
    # a tensor freed on the way is not reused by what the call itself allocates
    free = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    del free
    first = api.preference_loss(_dev(np.arange(300.0)), _dev([[k, 299 - k] for k in range(300)], torch.int32), kT=9.0,
                                reference=_dev(np.arange(300.0)[::-1].copy()))
    for _ in range(3):
        again = api.preference_loss(_dev(np.arange(300.0)), _dev([[k, 299 - k] for k in range(300)], torch.int32),
                                    kT=9.0, reference=_dev(np.arange(300.0)[::-1].copy()))
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    # two graphs of the same calls, replayed on two streams at once, on other inputs
    inputs = [xd.clone(), _dev((x * 1.5).astype(np.float32))]
    wants = [step(t) for t in inputs]
    graphs, outs = [], []
    for t in inputs:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(step(t))
        graphs.append((graph, s))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(wants, outs))


# ---------------------------------------------------------------- together, with a context
W4 = workloads.PROTEIN64.with_(name="cg_protein_4x269", n_replicas=4)


def _readout_of(weights):
    return {"R1": weights["R1"], "c1": weights["c1"], "R2": weights["R2"],
            "c2": np.array([weights["c2"]], dtype=np.float32)}


@pytest.mark.parametrize("w", [workloads.TINY, W4], ids=lambda w: w.name)
def test_tuning_with_a_context(w):
    weights = workloads.weights(w, bias_scale=0.1)
    model = api.from_workload(w, weights)
    pos, types = _dev(workloads.positions(w)), _dev(workloads.types(w), torch.int32)
    model.build_neighbors(pos)
    with pytest.raises(api.SchNetError) as e:
        model.features()                          # no evaluation yet
    assert e.value.status == 7
    E0, F0 = model.energy_forces(pos, types)
    eps0 = model.atom_energies()
    codes, scales = model.features()
    off = _dev(w.replica_offsets(), torch.int32)
    readout = _dw(_readout_of(weights))
    E, eps = api.readout_energy(codes, scales, off, readout)
    # the stored features are within 2^-4 of the trunk's (2^(e-10) for small ones): through the readout's slopes
    x = codes.double().cpu().numpy()[:, :w.F] * scales.double().cpu().numpy()[:, None]
    dx = np.maximum(np.abs(x) / 15, scales.double().cpu().numpy()[:, None] * 2.0 ** -10)
    tol = (dx @ np.abs(weights["R1"].astype(np.float64))) @ np.abs(weights["R2"]) + 1e-5
    assert np.all(np.abs((eps - eps0).cpu().numpy()) <= tol)
    # a step of tuning: loss over pairs of replicas, its gradient through the energies to the weights
    R = w.n_replicas
    pairs = [(r, (r + 1) % R) for r in range(R)]
    ref = (E0 + torch.arange(R, device="cuda")).float()
    loss, _, g = api.preference_loss(E, _dev(pairs, torch.int32), kT=0.6, reference=ref, smoothing=0.1)
    grads = api.readout_gradients(codes, scales, off, readout, g)
    host = _readout_of(weights)
    offs = w.replica_offsets()

    def oracle_loss(v):
        return tuning.preference(tuning.energy(x, offs, v)[0], pairs, 0.6, ref.cpu().numpy(), 0.1)[0]

    assert abs(float(loss) - oracle_loss(host)) <= 1e-4
    if R > 1:
        rng = np.random.default_rng(2)
        for k in host:                            # along a direction of each weight, against differences
            d = rng.normal(size=host[k].shape)
            h = 1e-5
            up, dn = ({**host, k: host[k].astype(np.float64) + s * h * d} for s in (1, -1))
            diff = (oracle_loss(up) - oracle_loss(dn)) / (2 * h)
            got = float((grads[k].double().cpu().numpy() * d).sum())
            size = float((np.abs(grads[k].double().cpu().numpy() * d)).sum())
            # dL/dE sums to zero over the replicas, which are equally long: c2's gradient is what the fp32 rounding
            # of each g_r leaves, at most u |g_r| for every atom of replica r
            left = U * float(g.abs().sum()) * w.beads * float(np.abs(d).max())
            assert abs(diff - got) <= 1e-3 * size + left + 1e-7, k
    # the tuned readout in the context: the same results as a context made with it
    tuned = {k: (readout[k] - 0.05 * grads[k]) for k in readout}
    tuned["c2"] = tuned["c2"] + 0.25
    model.set_readout(tuned)
    E1, F1 = model.energy_forces(pos, types)
    assert not torch.equal(E1, E0)
    fresh_w = dict(weights, R1=tuned["R1"].cpu().numpy(), c1=tuned["c1"].cpu().numpy(), R2=tuned["R2"].cpu().numpy(),
                   c2=float(tuned["c2"]))
    fresh = api.from_workload(w, fresh_w)
    fresh.build_neighbors(pos)
    E2, F2 = fresh.energy_forces(pos, types)
    assert torch.equal(E1, E2) and torch.equal(F1, F2)
    # and in MD: a step after the change, resumed, is the fresh context's
    mass = _dev(workloads.masses(w))
    out = []
    for m in (model, fresh):
        p, v = pos.clone(), torch.zeros_like(pos)
        m.step(p, v, types, mass, 3, dt=2.0, gamma=0.0)
        out.append(p)
    assert torch.equal(*out)
    c1 = model.features()
    c2 = fresh.features()
    assert torch.equal(c1[0].view(torch.uint8), c2[0].view(torch.uint8))
    assert torch.equal(c1[1].view(torch.uint8), c2[1].view(torch.uint8))


def test_resume_after_set_readout_uses_the_new_forces():
    w = workloads.TINY
    weights = workloads.weights(w)
    pos, types = _dev(workloads.positions(w)), _dev(workloads.types(w), torch.int32)
    mass = _dev(workloads.masses(w))
    new = _dw({k: v * 1.5 for k, v in _readout_of(weights).items()})
    runs = []
    for resume in (True, False):
        m = api.from_workload(w, weights)
        p, v = pos.clone(), torch.zeros_like(pos)
        m.step(p, v, types, mass, 20, dt=2.0, gamma=0.0)
        m.set_readout(new)
        m.step(p, v, types, mass, 5, dt=2.0, gamma=0.0, step0=20, resume=resume)
        runs.append((p, v))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


def test_first_call_of_a_process_inside_a_capture():
    code = """
import torch
from schnet_gnn_molecular_b200 import api
x = torch.arange(300 * 64, device="cuda").reshape(300, 64).float().cos()
off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
w = {"R1": x[:64, :32].contiguous(), "c1": x[0, :32].clone(), "R2": x[1, :32].clone(), "c2": x[2, :1].clone()}
pairs = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
def step():
    codes, scales = api.store_features(x)
    E, _ = api.readout_energy(codes, scales, off, w)
    loss, _, g = api.preference_loss(E, pairs, kT=1.0)
    return loss, api.readout_gradients(codes, scales, off, w, g)["R1"]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
want = step()
assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=240)


def test_a_call_that_fails_leaves_no_error_behind():
    """Calls into a capture that has already failed report it, and the next call on a sound stream works."""
    code = """
import ctypes as C
import torch
from schnet_gnn_molecular_b200 import _native as nat
from schnet_gnn_molecular_b200 import api
lib = nat.load()
x = torch.arange(300 * 64, device="cuda").reshape(300, 64).float().cos()
off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
w = {"R1": x[:64, :32].contiguous(), "c1": x[0, :32].clone(), "R2": x[1, :32].clone(), "c2": x[2, :1].clone()}
g = torch.ones(2, device="cuda")
E5, pairs = torch.arange(5000, device="cuda").float(), torch.randint(0, 5000, (3000, 2), device="cuda").int()
codes, scales = api.store_features(x)
want = [api.readout_energy(codes, scales, off, w)[0], api.readout_gradients(codes, scales, off, w, g)["R1"],
        api.preference_loss(E5, pairs, kT=1.0)[2]]
E, eps, dR1, dc1, dR2, dc2 = (torch.zeros(n, device="cuda") for n in (2, 300, 64 * 32, 32, 32, 1))
loss, dE = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(5000, device="cuda")
ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
p = lambda t: C.c_void_p(t.data_ptr())
def calls(stream):
    s, n = C.c_void_p(stream.cuda_stream), ws.numel()
    head = (p(codes), p(scales), 300, 64, 2, p(off), p(w["R1"]), p(w["c1"]), p(w["R2"]), p(w["c2"]))
    return (lib.schnet_readout_energy(*head, p(E), p(eps), p(ws), n, s),
            lib.schnet_readout_gradients(*head, p(g), p(dR1), p(dc1), p(dR2), p(dc2), p(ws), n, s),
            lib.schnet_preference_loss(p(E5), None, 0, 5000, p(pairs), 3000, 1.0, 0.0, p(loss), None, p(dE), None,
                                       p(ws), n, s))
main = torch.cuda.current_stream()
torch.cuda.synchronize()
for first in range(3):
    try:
        side = torch.cuda.Stream()
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            try:
                torch.cuda.synchronize()          # not allowed here: the capture is lost
            except RuntimeError:
                pass
            status = calls(side)[first]
    except RuntimeError:
        pass
    assert status == 2, status
    torch.cuda.set_stream(main)
    assert calls(main) == (0, 0, 0), first
    torch.cuda.synchronize()
    assert torch.equal(E, want[0]) and torch.equal(dR1.view(64, 32), want[1]) and torch.equal(dE, want[2])
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=240)


def test_a_tuning_loop_over_frames():
    w = W4
    weights = workloads.weights(w)
    model = api.from_workload(w, weights)
    pos, types = _dev(workloads.positions(w)), _dev(workloads.types(w), torch.int32)
    frames = []
    for k in range(3):                            # frames of three evaluations, concatenated
        p = (pos * (1.0 + 0.01 * k)).contiguous()
        model.build_neighbors(p)
        model.energy_forces(p, types, forces=False)
        frames.append(model.features())
    codes, scales = torch.cat([c for c, _ in frames]), torch.cat([s for _, s in frames])
    off = np.concatenate([[0]] + [w.replica_offsets()[1:] + k * w.n_atoms for k in range(3)]).astype(np.int32)
    offsets, readout = _dev(off), _dw(_readout_of(weights))
    pairs = _dev([[r, r + 4] for r in range(8)], torch.int32)
    reference, _ = api.readout_energy(codes, scales, offsets, readout)
    for _ in range(3):
        E, _ = api.readout_energy(codes, scales, offsets, readout)
        loss, margins, dE = api.preference_loss(E, pairs, kT=0.5962, reference=reference, smoothing=0.05)
        grads = api.readout_gradients(codes, scales, offsets, readout, dE)
        for k in readout:
            readout[k] -= 1e-3 * grads[k]
    x = codes.double().cpu().numpy()[:, :w.F] * scales.double().cpu().numpy()[:, None]
    host = {k: v.cpu().numpy() for k, v in readout.items()}
    E, _ = api.readout_energy(codes, scales, offsets, readout)
    want, eps = tuning.energy(x, off, host)
    scale = np.array([np.abs(eps[off[r]:off[r + 1]]).sum() for r in range(len(off) - 1)])
    assert np.all(np.abs(E.cpu().numpy() - want) <= 1e-5 * scale)
    model.set_readout(readout)


def test_features_are_ready_on_the_current_stream():
    """The model lives on one stream, which is busy; the features are read on another at once."""
    w = W4
    own, reader = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(own):
        model = api.from_workload(w, workloads.weights(w), device="cuda")
        pos, types = _dev(workloads.positions(w)), _dev(workloads.types(w), torch.int32)
        model.build_neighbors(pos)
        model.energy_forces(pos, types, forces=False)
        want = [t.view(torch.uint8).clone() for t in model.features()]
        # the memory that the next features will be given holds something else
        for t in [torch.full_like(t, 0x55) for t in want]:
            del t
        own.synchronize()
        torch.cuda._sleep(100_000_000)            # some 50 ms
    with torch.cuda.stream(reader):
        codes, scales = model.features()
        got = [codes.view(torch.uint8).clone(), scales.view(torch.uint8).clone()]
        del codes, scales                         # (their memory stays theirs until the copies are made)
    with torch.cuda.stream(own):
        for t in [torch.full_like(t, 0x55) for t in want]:
            del t
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_set_readout_refusals():
    w = workloads.TINY
    m = api.from_workload(w, workloads.weights(w))
    good = _readout_of(workloads.weights(w))
    with pytest.raises(ValueError):
        m.set_readout(dict(good, R1=good["R1"].T))
    with pytest.raises(ValueError):
        m.set_readout(dict(good, c1=good["c1"][:-1]))
