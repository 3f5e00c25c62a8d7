"""Waits of the attention over caches held in 8 or 4 bits that run out: every role of
the block goes on to its end, the call records VA_ERR_TIMEOUT, and the next call with a
fresh workspace gives what the first one gave.  (No GPU fault: the waits are bounded.)"""
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests.test_gpu_attn_quant import Case

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

WAIT_NS = 2_000_000
# (format, D, T, Hq, Hkv, page): every block size and way of loading
FORMS = {
    "16 rows": ("e2m1", 128, 4, 8, 2, 0),
    "32 rows, pages of 16": ("e4m3", 128, 8, 8, 2, 16),
    "32 rows, pages of 2": ("e2m1", 128, 8, 8, 2, 2),
    "64 rows": ("e4m3", 128, 16, 8, 2, 0),
    "64 rows, d64, pages of 4": ("e2m1", 64, 16, 8, 2, 4),
    "128 rows": ("e2m1", 128, 32, 8, 2, 0),
    "200 rows in blocks": ("e2m1", 128, 50, 8, 2, 64),
    "200 rows in blocks of 64": ("e4m3", 64, 50, 8, 2, 0),
}


def _gives_up(c, hook, undo):
    fresh = lambda: va.Workspace.for_shape(va.make_shape(len(c.L), c.T, c.Hq, c.Hkv, c.D, 0))  # noqa: E731
    ws = fresh()
    want = [x.clone() for x in c.run(ws)]
    va.verify_attn_check_status(ws)
    assert hook() == 0
    try:
        c.run(ws)
        with pytest.raises(va.VerifyAttnError) as e:
            va.verify_attn_check_status(ws)
        assert e.value.status == va.api.VA_ERR_TIMEOUT
    finally:
        assert undo() == 0
    ws = fresh()
    got = c.run(ws)
    va.verify_attn_check_status(ws)
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("form", FORMS)
def test_a_block_that_is_never_told_of_its_scores(form):
    fmt, D, T, Hq, Hkv, page = FORMS[form]
    c = Case(3, fmt, D, [100 + 37 * i for i in range(24)], T, Hq, Hkv, page, "tree")
    L = va.api.lib()
    _gives_up(c, lambda: L.verify_attn_test_stall(WAIT_NS, 5), lambda: L.verify_attn_test_stall(0, -1))


@pytest.mark.parametrize("form", FORMS)
def test_a_part_that_never_arrives(form):
    fmt, D, T, Hq, Hkv, page = FORMS[form]
    c = Case(3, fmt, D, [9000], T, Hq, Hkv, page, "tree")
    L = va.api.lib()
    _gives_up(c, lambda: L.verify_attn_test_inject(WAIT_NS, 0), lambda: L.verify_attn_test_inject(0, -1))


@pytest.mark.parametrize("form", ["16 rows", "32 rows, pages of 16", "32 rows, pages of 2", "64 rows", "128 rows"])
def test_a_block_with_many_tiles_left_when_it_gives_up(form):
    """Ten tiles to a block, more than its ring holds: it loads none over copies under way."""
    fmt, D, T, Hq, Hkv, page = FORMS[form]
    c = Case(3, fmt, D, [4000 + 37 * i for i in range(24)], T, Hq, Hkv, page, "chain")
    L = va.api.lib()
    _gives_up(c, lambda: L.verify_attn_test_stall(WAIT_NS, 5), lambda: L.verify_attn_test_stall(0, -1))
