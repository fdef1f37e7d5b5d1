"""The readout-tuning kernels against bounds tight enough for what tests/test_readout_bounds.py plants: a hidden layer
formed from R1 rounded once to 16 bits, a tile of atoms left out of the gradients, features in another order."""
import numpy as np
import pytest
import torch

from _helpers import oracle_model
from _readout_bounds import GradientProblem, row_bound, stored, trunk, unit_energy, weights
from schnet_gnn_molecular_b200 import api, workloads

pytestmark = pytest.mark.gpu


def _dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype).cuda()


def _dw(w):
    return {k: _dev(v) for k, v in w.items()}


def _values(codes, scales, F):
    return codes.double().cpu().numpy()[:, :F] * scales.double().cpu().numpy()[:, None]


@pytest.mark.parametrize("F", [64, 98, 128])
@pytest.mark.parametrize("n", [1, 269, 1013])
def test_energies_hold_both_terms_of_R1(F, n):
    rng = np.random.default_rng(F + n)
    x32 = (rng.normal(size=(n, F)) * np.exp(0.7 * rng.normal(size=(n, 1)))).astype(np.float32)
    codes, scales = api.store_features(_dev(x32))
    x, _ = stored(x32)
    assert np.array_equal(_values(codes, scales, F), x)
    w = weights(F, rng)
    for h in (0, F // 4 - 1, F // 4, F // 2 - 1):
        one = dict(w, R2=np.eye(F // 2, dtype=np.float32)[h], c2=np.zeros(1, np.float32))
        E, eps = api.readout_energy(codes, scales, _dev([0, n], torch.int32), _dw(one))
        want, bound = unit_energy(x, w, h)
        assert np.all(np.abs(eps.cpu().numpy() - want) <= bound), h
        assert abs(float(E[0]) - want.sum()) <= bound.sum() + 2.0 ** -24 * abs(want.sum())


@pytest.mark.parametrize("F", [64, 94, 128])
def test_gradients_hold_every_tile(F):
    p = GradientProblem(F)
    codes, scales = api.store_features(_dev(p.x32))
    assert np.array_equal(_values(codes, scales, F), p.x)
    got = api.readout_gradients(codes, scales, _dev(p.off), _dw(p.w), _dev(p.g))
    for k, want in p.want.items():
        error = np.abs(got[k].cpu().numpy() - want)
        assert np.all(error <= p.tol[k]), (k, float((error / p.tol[k]).max()))


def test_rows_past_32_bits():
    """17 million rows of 128: the codes' bytes and the features' elements pass 2^31.  The last rows' results are those
    of the last rows alone."""
    n, tail, F = 17_000_000, 1280, 128
    rng = np.random.default_rng(4)
    x = torch.zeros(n, F, device="cuda")
    last = rng.normal(size=(tail, F)).astype(np.float32)
    x[-tail:] = _dev(last)
    codes, scales = api.store_features(x)
    del x
    want = api.store_features(_dev(last))
    assert all(torch.equal(a[-tail:].view(torch.uint8), b.view(torch.uint8)) for a, b in zip((codes, scales), want))
    assert not codes[:-tail].view(torch.uint8).any()
    w = _dw(weights(F, rng))
    E, eps = api.readout_energy(codes, scales, _dev([0, n - 700, n], torch.int32), w)
    E1, eps1 = api.readout_energy(*want, _dev([0, tail - 700, tail], torch.int32), w)
    assert n % 128 == 64 and tail % 128 == 0       # (the same rows at other places of a tile)
    assert torch.equal(eps[-tail:], eps1)
    assert abs(float(E[1] - E1[1])) <= 2.0 ** -24 * abs(float(E1[1]))
    g = _dev([0.0, 1.0], torch.float32)
    got = api.readout_gradients(codes, scales, _dev([0, n - 700, n], torch.int32), w, g)
    alone = api.readout_gradients(*want, _dev([0, tail - 700, tail], torch.int32), w, g)
    assert float(got["c2"]) == 700.0
    for k in got:                                  # the same terms, summed in other tiles: 700 roundings of them
        size = {"R1": np.abs(last[-700:]).sum(0)[:, None] * w["R2"].abs().cpu().numpy(),
                "c1": 700 * w["R2"].abs().cpu().numpy(), "R2": np.full(F // 2, 700 * 4.0), "c2": 0.0}[k]
        assert np.all(np.abs((got[k] - alone[k]).cpu().numpy()) <= 700 * 2.0 ** -23 * size), k


@pytest.mark.parametrize("w", [workloads.TINY, workloads.TINY.with_(name="tiny_chain64_f50", F=50),
                               workloads.PROTEIN64.with_(name="cg_protein_4x269", n_replicas=4)],
                         ids=lambda w: w.name)
@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("evaluate", ["energies", "forces", "steps"])
def test_features_are_the_trunks_in_the_callers_order(w, shuffled, evaluate):
    W = workloads.weights(w, bias_scale=0.1)
    off = w.replica_offsets()
    pos, types = workloads.positions(w).astype(np.float32), workloads.types(w)
    if shuffled:                                  # beads listed in any order: no list order is the cells'
        rng = np.random.default_rng(3)
        order = np.concatenate([a + rng.permutation(b - a) for a, b in zip(off[:-1], off[1:])])
        pos, types = pos[order], types[order]
    model = api.from_workload(w, W)
    p, t = _dev(pos), _dev(types, torch.int32)
    if evaluate == "steps":
        model.step(p, torch.zeros_like(p), t, _dev(np.full(w.n_atoms, w.mass, np.float32)), 5, dt=2.0, gamma=0.0,
                   n_rebuild=2)
    else:
        model.build_neighbors(p)
        model.energy_forces(p, t, forces=evaluate == "forces")
    codes, scales = model.features()
    want = trunk(oracle_model(w, W), p.double().cpu().numpy(), types, off)
    got = _values(codes, scales, w.F)
    assert np.all(np.abs(got - want) <= row_bound(want, scales.double().cpu().numpy()))
