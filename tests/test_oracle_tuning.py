"""What pins the oracle of the readout-tuning operators (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import tuning


def test_e4m3_rounding_is_the_formats():
    # every pair of neighbouring values: themselves, the tie between them, and a little to each side
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    v = codes.float().numpy().astype(np.float64)
    mid = (v[:-1] + v[1:]) / 2
    x = np.concatenate([v, mid, mid * (1 + 1e-6), mid * (1 - 1e-6)])
    x = np.concatenate([x, -x])
    want = torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(tuning.round_e4m3(x), want)
    assert tuning.round_e4m3(17.0) == 16.0 and tuning.round_e4m3(19.0) == 20.0       # ties to even


def test_store_scales():
    x = np.array([[448.0, 1.0], [448.1, 1.0], [0.0, 0.0], [2.0 ** -130, 0.0], [np.inf, 0.0], [2.0 ** 127, 1.0]])
    q, e = tuning.store(x)
    assert e == [0, 1, -100, -100, None, None]
    assert q[0, 0] == 448.0 and q[1, 0] == 224.0 and not q[2:].any()
    rng = np.random.default_rng(0)
    x = rng.normal(size=(200, 12)) * np.exp(rng.normal(size=(200, 1)))
    q, e = tuning.store(x)
    back = q * 2.0 ** np.array(e)[:, None]
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (np.array(e)[:, None] - 10.0)))


def _case(F=6, n=9, seed=1):
    rng = np.random.default_rng(seed)
    w = {"R1": rng.normal(size=(F, F // 2)), "c1": rng.normal(size=F // 2), "R2": rng.normal(size=F // 2),
         "c2": rng.normal(size=1)}
    return rng.normal(size=(n, F)), [1, 1, 4, 8], w, rng.normal(size=3)


def test_energy_by_hand():
    w = {"R1": np.array([[1.0], [2.0]]), "c1": np.array([0.0]), "R2": np.array([3.0]), "c2": np.array([0.5])}
    E, eps = tuning.energy(np.array([[np.log(3.0), 0.0], [0.0, 0.0]]), [0, 2], w)
    assert np.allclose(eps, [3 * np.log(2.0) + 0.5, 0.5], atol=1e-15) and np.allclose(E, eps.sum(), atol=1e-15)


@pytest.mark.parametrize("name", ["R1", "c1", "R2", "c2"])
def test_gradients_are_differences_of_the_energy(name):
    x, off, w, g = _case()
    got = tuning.gradients(x, off, w, g)[name]
    h = 1e-6
    for idx in np.ndindex(w[name].shape):
        both = []
        for sgn in (1, -1):
            v = {k: a.copy() for k, a in w.items()}
            v[name][idx] += sgn * h
            both.append(float(np.dot(g, tuning.energy(x, off, v)[0])))
        assert abs((both[0] - both[1]) / (2 * h) - got[idx]) < 1e-7


@pytest.mark.parametrize("s", [0.0, 0.2, 1.0])
def test_preference_gradient_is_the_difference_of_the_loss(s):
    rng = np.random.default_rng(3)
    E, ref = rng.normal(size=7), rng.normal(size=7)
    pairs = [(0, 1), (1, 0), (2, 2), (3, -1), (5, 1), (0, 1), (9, 0)]
    _, m, g, count = tuning.preference(E, pairs, 0.6, ref, s)
    assert count == 5 and m[2] == 0 and m[3] == 0 and m[6] == 0 and g[4] == 0 and g[6] == 0
    for r in range(7):
        e1, e2 = E.copy(), E.copy()
        e1[r] += 1e-6
        e2[r] -= 1e-6
        d = (tuning.preference(e1, pairs, 0.6, ref, s)[0] - tuning.preference(e2, pairs, 0.6, ref, s)[0]) / 2e-6
        assert abs(d - g[r]) < 1e-8
    assert tuning.preference(E, [(0, 1)], 1.0)[0] == pytest.approx(np.log1p(np.exp(E[0] - E[1])), abs=1e-15)
