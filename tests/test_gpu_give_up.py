"""A wait inside a block that runs out: every role of the block goes on to its end
without waiting, the call returns VA_ERR_TIMEOUT, and the next call with a fresh
workspace gives what the first one gave.  Blocks hold parts of several segments of
several tiles, so the roles pass every barrier between them more than once."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests import shaped

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

WAIT_NS = 2_000_000
RANGE, SCORE = dict(window=300), dict(softcap=20.0, slopes=True)
# (T, Hq, Hkv, D, page, rules): the kernels and their ways of loading tiles
ATTEND = {
    "16 rows": (4, 32, 8, 128, 0, SCORE),
    "32 rows": (8, 32, 8, 128, 0, SCORE),
    "64 rows, pages of 16": (16, 32, 8, 128, 16, RANGE),
    "64 rows, pages of 64": (16, 32, 8, 128, 64, SCORE),
    "32 rows, pages of 2": (8, 32, 8, 128, 2, RANGE),
    "d64, 20 rows": (5, 32, 8, 64, 0, SCORE),
    "d64, 64 rows, pages of 8": (16, 32, 8, 64, 8, SCORE),
    "d64, blocks of rows": (24, 32, 8, 64, 0, RANGE),
    "100 rows": (25, 32, 8, 128, 0, RANGE),
    "128 rows, pages of 4": (32, 32, 8, 128, 4, SCORE),
    "256 rows": (64, 32, 8, 128, 0, SCORE),
    "256 rows, pages of 64": (64, 32, 8, 128, 64, RANGE),
}
PLAIN = ["16 rows", "32 rows", "64 rows, pages of 16", "32 rows, pages of 2", "100 rows", "128 rows, pages of 4",
         "256 rows"]
WEIGH = {
    "32 rows": (8, 32, 8, 128, 0, {}),
    "32 rows, capped": (8, 32, 8, 128, 0, SCORE),
    "64 rows, pages of 16": (16, 32, 8, 128, 16, {}),
    "64 rows, pages of 2": (16, 32, 8, 128, 2, {}),
    "256 rows": (64, 32, 8, 128, 0, {}),
    "256 rows, pages of 8": (64, 32, 8, 128, 8, {}),
    "384 rows in two passes": (64, 48, 8, 128, 0, {}),
    "d64": (8, 32, 8, 64, 0, SCORE),
}


def _case(form, seed=3):
    T, Hq, Hkv, D, page, rules = form
    rng = np.random.default_rng(seed)
    return shaped.make(seed, rng.integers(100, 500, 40).tolist(), T, Hq, Hkv, D, "bf16", page, **rules)


def _gives_up(call, fresh):
    """call(workspace) -> outputs: right, then with block 5 stalled, then right again."""
    L = va.api.lib()
    ws = fresh()
    want = [x.clone() for x in call(ws)]
    va.verify_attn_check_status(ws)
    assert L.verify_attn_test_stall(WAIT_NS, 5) == 0
    try:
        call(ws)
        with pytest.raises(va.VerifyAttnError) as ei:
            va.verify_attn_check_status(ws)
        assert ei.value.status == va.api.VA_ERR_TIMEOUT
    finally:
        assert L.verify_attn_test_stall(0, -1) == 0
    ws = fresh()
    got = call(ws)
    va.verify_attn_check_status(ws)
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("form", ATTEND)
def test_shaped_attention(form):
    c = _case(ATTEND[form])
    shape = va.make_shape(c.B, c.T, c.Hq, c.Hkv, c.D, 0)
    _gives_up(lambda ws: shaped.run_attend(va, c, workspace=ws), lambda: va.Workspace.for_shape(shape))


@pytest.mark.parametrize("form,kernel", [(f, "default") for f in PLAIN] + [("256 rows", "tcp")])
def test_plain_attention(form, kernel, monkeypatch):
    if kernel == "tcp":  # the two-M-tile kernel of 128-key tiles
        monkeypatch.setenv("VA_MANY_ROWS_KERNEL", "tcp")
    c = _case(ATTEND[form])
    shape = va.make_shape(c.B, c.T, c.Hq, c.Hkv, c.D, 0)
    q, k, v, L = c.q.cuda(), c.k.cuda(), c.v.cuda(), shaped.dev(c.L)

    def call(ws):
        if c.table is not None:
            return va.verify_attn_paged(q, k, v, shaped.dev(c.table), L, workspace=ws)
        return va.verify_attn_dense(q, k, v, L, workspace=ws)

    _gives_up(call, lambda: va.Workspace.for_shape(shape))


@pytest.mark.parametrize("form", WEIGH)
def test_accumulated_weight(form):
    c = _case(WEIGH[form])
    lse = torch.full((c.B, c.Hq, c.T), 6.0, device="cuda")
    start = torch.rand(c.B, c.Hkv, c.cap, device="cuda")

    def call(ws):
        return [shaped.run_weight(va, c, lse, start.clone(), decay=0.9, workspace=ws)]

    _gives_up(call, lambda: va.Workspace(256))


def test_refusals():
    L = va.api.lib()
    assert L.verify_attn_test_stall(100_000_001, 0) == va.api.VA_ERR_INVALID_ARG
    assert L.verify_attn_test_stall(0, -1) == 0
