"""CPU: what the bounds of tests/test_gpu_readout_tight.py would notice, with the mistake planted in the float64
formulas, and that those formulas agree with the oracle's own."""
import numpy as np
import pytest

import oracle
from _helpers import oracle_model
from _readout_bounds import GradientProblem, once_rounded, preactivation, row_bound, stored, trunk, unit_energy, weights
from oracle import tuning
from schnet_gnn_molecular_b200 import workloads


def test_stored_is_the_oracles_store():
    x = np.random.default_rng(0).normal(size=(200, 30)) * np.exp(np.random.default_rng(1).normal(size=(200, 1)))
    q, e = tuning.store(x)
    v, scale = stored(x)
    assert np.array_equal(scale, 2.0 ** np.array(e)) and np.array_equal(v, q * scale[:, None])


@pytest.mark.parametrize("F", [18, 64, 98, 128])
def test_preactivations_are_the_oracles(F):
    rng = np.random.default_rng(F)
    x, _ = stored(rng.normal(size=(50, F)))
    w = weights(F, rng)
    p, b = preactivation(x, w)
    assert np.allclose(p, tuning.hidden(x, w), rtol=0, atol=1e-12) and (b > 0).all()


@pytest.mark.parametrize("F", [98, 128])
def test_energies_with_R1_rounded_once_would_be_noticed(F):
    rng = np.random.default_rng(F)
    x, _ = stored(rng.normal(size=(1013, F)) * np.exp(0.7 * rng.normal(size=(1013, 1))))
    w = weights(F, rng)
    wrong = dict(w, R1=once_rounded(w["R1"]))
    for h in (0, F // 4 - 1, F // 4, F // 2 - 1):
        eps, bound = unit_energy(x, w, h)
        assert (np.abs(tuning.ssp(tuning.hidden(x, wrong)[:, h]) - eps) > 2 * bound).mean() > 0.1


@pytest.mark.parametrize("F", [64, 94, 128])
def test_a_tile_left_out_of_the_gradients_would_be_noticed(F):
    g = GradientProblem(F)
    R1, sums = g.noticed()
    assert len(R1) > 15 * 148                     # tiles: rings of 2 and 3 and runs of 8 go round on 148 SMs
    assert R1.all() and sums.mean() > 0.99       # (where the seed's sign changes inside a tile its halves may cancel)
    want = tuning.gradients(g.x[:4096], np.minimum(g.off, 4096), g.w, g.g)
    assert np.allclose(g.tR1[:32].sum(0) * g.r2, want["R1"]) and np.allclose(g.tR2[:32].sum(0), want["R2"])


@pytest.mark.parametrize("w", [workloads.TINY, workloads.PROTEIN64.with_(name="cg_protein_4x269", n_replicas=4)],
                         ids=lambda w: w.name)
def test_features_of_another_atom_would_be_noticed(w):
    """The trunk's formula is the oracle's (its energies follow from it), and no atom's features pass for another's."""
    W = workloads.weights(w, bias_scale=0.1)
    model = oracle_model(w, W)
    pos, types, off = workloads.positions(w).astype(np.float64), workloads.types(w), w.replica_offsets()
    x = trunk(model, pos, types, off)
    _, eps, _ = oracle.energy_forces(model, pos, types, off, forces=False)
    mine = tuning.ssp(tuning.hidden(x, W)) @ W["R2"].astype(np.float64) + W["c2"]
    assert np.allclose(mine, eps, rtol=0, atol=1e-10)
    v, scale = stored(x)
    bound = row_bound(x, scale)
    assert (np.abs(v - x) <= bound).all()
    for i in range(len(x)):
        same = (np.abs(v - x[i]) <= row_bound(x[i:i + 1], scale[i:i + 1])).all(1)
        assert same.sum() == 1 and same[i]
