"""The readout-tuning kernels against bounds tight enough for what tests/test_readout_bounds.py plants: a hidden layer
formed from R1 rounded once to 16 bits, a tile of atoms left out of the gradients."""
import numpy as np
import pytest
import torch

from _readout_bounds import GradientProblem, stored, unit_energy, weights
from schnet_gnn_molecular_b200 import api

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
