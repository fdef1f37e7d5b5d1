"""Refused calls of the readout-tuning entry points: argument errors come back before any CUDA call, so they
are checked without a GPU."""
import ctypes as C

import numpy as np
import pytest
import torch

from schnet_gnn_molecular_b200 import _native as nat
from schnet_gnn_molecular_b200 import api, build

P = C.c_void_p(4096)          # a pointer that no refused call follows


@pytest.fixture(scope="module")
def lib():
    build.build()
    return nat.load()


def test_store_refusals(lib):
    ok = dict(x=P, dtype=0, n=4, F=64, stride=64, codes=P, scales=P)
    def call(**kw):
        a = {**ok, **kw}
        return lib.schnet_store_features(a["x"], a["dtype"], a["n"], a["F"], a["stride"], a["codes"], a["scales"], None)
    assert call(F=0) == 9 and call(F=3) == 9 and call(F=130) == 9
    for bad in (dict(x=None), dict(codes=None), dict(scales=None), dict(dtype=3), dict(dtype=-1), dict(n=-1),
                dict(stride=63), dict(codes=C.c_void_p(4104)), dict(x=C.c_void_p(4098))):
        assert call(**bad) == 1, bad


def test_readout_refusals(lib):
    big = 1 << 40
    def energy(codes=P, scales=P, n=8, F=64, R=2, off=P, R1=P, c1=P, R2=P, c2=P, e=P, eps=P, ws=P, size=big):
        return lib.schnet_readout_energy(codes, scales, n, F, R, off, R1, c1, R2, c2, e, eps, ws, size, None)
    def grad(codes=P, scales=P, n=8, F=64, R=2, off=P, R1=P, c1=P, R2=P, c2=P, g=P, d=P, ws=P, size=big):
        return lib.schnet_readout_gradients(codes, scales, n, F, R, off, R1, c1, R2, c2, g, P, P, P, d, ws, size, None)
    for f in (energy, grad):
        assert f(F=3) == 9 and f(F=0) == 9 and f(F=256) == 9
        for bad in (dict(codes=None), dict(scales=None), dict(n=-1), dict(n=2 ** 31 - 1), dict(R=0), dict(off=None),
                    dict(R1=None),
                    dict(c1=None), dict(R2=None), dict(c2=None), dict(ws=None), dict(ws=C.c_void_p(4100)),
                    dict(size=64), dict(codes=C.c_void_p(4097))):
            assert f(**bad) == 1, (f, bad)
    assert energy(e=None) == 1 and energy(eps=None) == 1 and grad(g=None) == 1 and grad(d=None) == 1
    n = C.c_size_t(0)
    assert lib.schnet_readout_workspace_bytes(100, 64, C.byref(n)) == 0 and n.value > 0
    assert lib.schnet_readout_workspace_bytes(100, 63, C.byref(n)) == 9
    assert lib.schnet_readout_workspace_bytes(-1, 64, C.byref(n)) == 1
    assert lib.schnet_readout_workspace_bytes(1, 64, None) == 1


# the kernels step through the replicas in 32 bits: past this many an index could wrap
MAX_REPLICAS = 0x7ff00000


def test_too_many_replicas(lib):
    big = 1 << 62
    need = C.c_size_t(0)
    for R in (MAX_REPLICAS + 1, 2 ** 31 - 1):
        assert lib.schnet_preference_workspace_bytes(R, 9, C.byref(need)) == 1
        assert lib.schnet_preference_loss(P, None, 0, R, P, 9, 0.6, 0.0, P, None, P, None, P, big, None) == 1
        assert lib.schnet_readout_energy(P, P, 8, 64, R, P, P, P, P, P, P, P, P, big, None) == 1
        assert lib.schnet_readout_gradients(P, P, 8, 64, R, P, P, P, P, P, P, P, P, P, P, P, big, None) == 1
    assert lib.schnet_preference_workspace_bytes(MAX_REPLICAS, 9, C.byref(need)) == 0
    # the largest stride of a loop over replicas is 1184 CTAs of 256 threads
    assert MAX_REPLICAS - 1 + 1184 * 256 < 2 ** 31


def test_preference_refusals(lib):
    need = C.c_size_t(0)
    assert lib.schnet_preference_workspace_bytes(16, 9, C.byref(need)) == 0
    def call(e=P, ref=None, dtype=0, R=16, pairs=P, n=9, kT=0.6, s=0.0, loss=P, m=None, g=P, ws=P, size=need.value):
        return lib.schnet_preference_loss(e, ref, dtype, R, pairs, n, kT, s, loss, m, g, None, ws, size, None)
    for bad in (dict(e=None), dict(dtype=1), dict(dtype=2), dict(R=0), dict(pairs=None), dict(n=-1), dict(n=2 ** 31),
                dict(kT=0.0), dict(kT=-1.0), dict(kT=float("nan")), dict(kT=float("inf")), dict(s=-0.1), dict(s=1.1),
                dict(s=float("nan")), dict(loss=None), dict(g=None), dict(ws=None), dict(ws=C.c_void_p(4100)),
                dict(size=need.value - 1), dict(pairs=C.c_void_p(4100))):
        assert call(**bad) == 1, bad
    assert lib.schnet_preference_workspace_bytes(0, 1, C.byref(need)) == 1
    assert lib.schnet_preference_workspace_bytes(1, 1, None) == 1


def test_kT_whose_reciprocal_is_infinite(lib):
    """Margins of 0 would be 0 times infinity."""
    for kT in (5e-324, 5.5e-309):
        assert lib.schnet_preference_loss(P, None, 0, 16, P, 9, kT, 0.0, P, None, P, None, P, 1 << 40, None) == 1


def test_timeout_tap_refusals(lib):
    def call(n=8, R=2, off=P, e=P, eps=P, ws=P, size=1 << 40):
        return lib.schnet_test_readout_timeout(n, R, off, 1, e, eps, ws, size, None)
    for bad in (dict(n=0), dict(n=-1), dict(R=0), dict(R=MAX_REPLICAS + 1), dict(off=None), dict(e=None), dict(eps=None),
                dict(ws=None), dict(ws=C.c_void_p(4100)), dict(size=64)):
        assert call(**bad) == 1, bad


def test_context_calls_refuse_null(lib):
    assert lib.schnet_get_features(None, P, P) == 1
    assert lib.schnet_set_readout(None, P, P, P, 0.0) == 1


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        api.store_features(x)
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8)
    w = {"R1": torch.zeros(64, 32), "c1": torch.zeros(32), "R2": torch.zeros(32), "c2": torch.zeros(1)}
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        api.readout_energy(codes, scales, off, w)
    with pytest.raises(ValueError):
        api.preference_loss(torch.zeros(4), torch.zeros(1, 2, dtype=torch.int32), kT=1.0)


def test_binding_refuses_other_8_bit_types(lib):
    """Their bytes are not e4m3 codes and e8m0 scales; plain bytes are taken as such."""
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8)
    w = {"R1": torch.zeros(64, 32), "c1": torch.zeros(32), "R2": torch.zeros(32), "c2": torch.zeros(1)}
    off, g = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(1)
    calls = (lambda c, s: api.readout_energy(c, s, off, w), lambda c, s: api.readout_gradients(c, s, off, w, g))
    for call in calls:
        for t in (torch.int8, torch.bool, torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e8m0fnu):
            with pytest.raises(ValueError, match="codes must be Float8_e4m3fn or Byte"):
                call(codes.view(t), scales)
        for t in (torch.int8, torch.bool, torch.float8_e4m3fn):
            with pytest.raises(ValueError, match="scales must be Float8_e8m0fnu or Byte"):
                call(codes, scales.view(t))
        for c, s in ((codes, scales), (codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu))):
            with pytest.raises(ValueError, match="CUDA"):
                call(c, s)


def test_binding_refuses_what_autograd_would_lose(lib):
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8)
    w = {"R1": torch.zeros(64, 32), "c1": torch.zeros(32), "R2": torch.zeros(32), "c2": torch.zeros(1)}
    off, g = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(1)
    E, pairs = torch.zeros(4), torch.zeros(1, 2, dtype=torch.int32)
    calls = [("x", lambda t: api.store_features(t), torch.zeros(4, 64)),
             ("grad_energy", lambda t: api.readout_gradients(codes, scales, off, w, t), g),
             ("energy", lambda t: api.preference_loss(t, pairs, kT=1.0), E),
             ("reference", lambda t: api.preference_loss(E, pairs, kT=1.0, reference=t), E)]
    for k in w:
        calls.append((k, lambda t, k=k: api.readout_energy(codes, scales, off, dict(w, **{k: t})), w[k]))
        calls.append((k, lambda t, k=k: api.readout_gradients(codes, scales, off, dict(w, **{k: t}), g), w[k]))
    for name, call, t in calls:
        leaf = t.clone().requires_grad_()
        for value in (leaf, leaf * 2):
            with pytest.raises(ValueError, match=f"{name} requires grad"):
                call(value)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
                call(value)
            with pytest.raises(ValueError, match="CUDA"):
                call(value.detach())


def test_binding_refuses_flags_that_are_no_integer(lib):
    E, pairs = torch.zeros(4), torch.zeros(1, 2, dtype=torch.int32)
    for t in (torch.float32, torch.int64, torch.int16):
        with pytest.raises(ValueError, match="flags must be one 32-bit integer"):
            api.preference_loss(E, pairs, kT=1.0, flags=torch.zeros(1, dtype=t))
    for t in (torch.int32, torch.uint32):
        with pytest.raises(ValueError, match="CUDA"):
            api.preference_loss(E, pairs, kT=1.0, flags=torch.zeros(1, dtype=t))
