"""CPU: the polynomial of the small shifted softplus in csrc/readout.cu is the one the committed fit produces, and
its float32 Horner form stays within the bound stated beside it (relative error <= 2e-7 on |t| <= 3)."""
import os
import re

import numpy as np

from schnet_gnn_molecular_b200 import ssp2_fit

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _source():
    return open(os.path.join(ROOT, "schnet_gnn_molecular_b200", "csrc", "readout.cu")).read()


def test_device_coefficients_are_the_fit():
    src = _source()
    body = src[src.index("float2 ssp2_small(float2 t)"):]
    body = body[:body.index("return")]
    lits = [float(x) for x in re.findall(r"dup2\((-?[0-9.]+(?:e-?[0-9]+)?)f\)", body)]      # c5 .. c0
    assert np.array_equal(np.array(lits[::-1], dtype=np.float32), ssp2_fit.fit())
    assert float(re.search(r"SSP2_SMALL = ([0-9.]+)f", src)[1]) == ssp2_fit.RANGE


def test_fit_error_bound():
    c = ssp2_fit.fit()
    assert ssp2_fit.max_rel_error(c) <= 2e-7
    tiny = np.array([1e-30, -1e-30, 1e-6, -1e-6], dtype=np.float32)
    assert np.allclose(ssp2_fit.horner_f32(c, tiny), ssp2_fit.ssp2(tiny), rtol=2e-7, atol=0)
