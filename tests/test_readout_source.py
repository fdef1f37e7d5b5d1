"""A rule of the tensor-core kernels that no run can show: after a wait for something that MMAs complete or that
other warps hand over to them, a tensor-memory operation follows only behind tcgen05.fence::after_thread_sync,
which is what orders it after the other thread's."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "schnet_gnn_molecular_b200", "csrc",
                   "readout.cu")

TOKENS = re.compile(r"(?P<wait>(?<![\w.])wait\((?:done|ready)[12]\b|mbar_wait_bounded\(full \+ FWD_STAGES\b)"
                    r"|(?P<fence>\btc_fence_after\(\))"
                    r"|(?P<op>\b(?:tmem_ld|tmem_st16|mma_ts|mma_ss|tmem_dealloc)\(|\bgemm[12]\(it\b)")


def _kernel(name):
    src = open(SRC).read()
    body = src[src.index(name + "(const __grid_constant__"):]
    return re.sub(r"//[^\n]*", "", body[:body.index("\n}\n")])


def unfenced(body):
    """Tensor-memory operations that follow a wait without a fence between."""
    out, pending = [], None
    for m in TOKENS.finditer(body):
        if m["wait"]:
            pending = m.group()
        elif m["fence"]:
            pending = None
        elif pending:
            out.append((pending, m.group(), body[:m.start()].count("\n")))
    return out


@pytest.mark.parametrize("name", ["k_readout_eps", "k_readout_grad"])
def test_tensor_memory_is_touched_behind_a_fence(name):
    body = _kernel(name)
    assert len(TOKENS.findall(body)) > 8
    assert unfenced(body) == []


def test_the_scan_sees_a_missing_fence():
    body = _kernel("k_readout_eps")
    at = body.index("tc_fence_after();", body.index("FWD_STAGES + 1, (uint32_t)it"))
    assert unfenced(body[:at] + body[at + len("tc_fence_after();"):])
