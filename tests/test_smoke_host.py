"""The smoke step's check of the shaped attention tells a call that leaves a rule out
from one that does not."""
import numpy as np
import pytest

import __graft_entry__ as entry
import workloads as W


@pytest.fixture(scope="module")
def step():
    w = W.make_workload("tree", seed=0, L=700, T=16, depth=4)
    pos = (w.seqlens[:, None] + np.stack([W.chain_depths(p) for p in w.parent])).astype(np.int32)[0]
    return w, pos, entry.shaped_reference(w, pos, 2.0, 300)


def test_the_definition_passes(step):
    w, pos, ref = step
    assert entry.check_shaped(ref[0] * (1 + 2.0 ** -9), ref[1] + 1e-4, ref) <= 2e-4


@pytest.mark.parametrize("softcap,window", [(1e6, 300), (2.0, 1 << 20), (1e6, 1 << 20), (2.0, 299)])
def test_a_lost_rule_fails(step, softcap, window):
    """No cap, no window, neither, and a window of one slot less."""
    w, pos, ref = step
    out, lse = entry.shaped_reference(w, pos, softcap, window)
    with pytest.raises(AssertionError):
        entry.check_shaped(out, lse, ref)


def test_the_unshaped_reference_is_the_oracle(step):
    import oracle

    w, pos, _ = step
    out, lse = entry.shaped_reference(w, pos, 1e9, 1 << 30)
    ref = oracle.verify(w)
    assert np.abs(out - ref["out"][0]).max() <= 1e-6 and np.abs(lse - ref["lse"][0]).max() <= 1e-6
