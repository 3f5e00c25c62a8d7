"""GPU parity of the accumulated attention weight against a plain fp64 statement.

Tolerance.  A term is exp(s - lse) with s and lse in fp32: the products of 128
bf16 values add up to within 1e-5 of a score of a few units, the cap and the
bias to within 2^-21 of |s| <= 100, and 2^x is good to 2^-22, so every term is
within a relative 2e-4 (the lse handed over is the fp64 one, rounded to fp32).
A total adds such terms to an fp32 running total: 2e-4 of it, plus 1e-7 for
terms below the flushed range.
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests import shaped

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

SENTINEL = 77.0


def _inputs(c, seed, accept):
    rng = np.random.default_rng(seed)
    path = np.full((c.B, c.T), -1, np.int32)
    for b, a in enumerate(accept):
        path[b, :a] = np.sort(rng.permutation(c.T)[:a])
    # what the verification of a chain of the accepted tokens returns, in fp64:
    # rows by accepted rank, put at their draft nodes
    lse = rng.standard_normal((c.B, c.Hq, c.T)).astype(np.float32)
    full = np.zeros((c.B, c.Hq, c.T))
    q = c.q.clone()
    for b, a in enumerate(accept):
        for i in range(a):
            q[b, i] = c.q[b, path[b, i]]
    import copy
    d = copy.copy(c)
    d.q, d.pos = q, c.L[:, None] + np.arange(c.T)[None]
    d.draft = np.tile(np.tril(np.ones((c.T, c.T), bool)), (c.B, 1, 1))
    _, full = shaped.attend(d)
    for b, a in enumerate(accept):
        for i in range(a):
            lse[b, :, path[b, i]] = full[b, :, i]
    weight = rng.random((c.B, c.Hkv, c.cap + 5)).astype(np.float32)
    return path, np.asarray(accept, np.int32), lse, weight


def _check(got, want, c, accept, before):
    for b in range(c.B):
        n = int(c.L[b]) + int(accept[b])
        err = np.abs(got[b, :, :n] - want[b, :, :n])
        bound = 2e-4 * np.abs(want[b, :, :n]) + 1e-7
        assert (err <= bound).all(), f"sequence {b}: worst excess {(err - bound).max():.3e}"
        assert np.array_equal(got[b, :, n:], before[b, :, n:]), "totals past the committed slots were written"


FORMS = {
    "bf16 d128": ("bf16", 128, 8, 8, 2, 0),
    "bf16 d128 one token": ("bf16", 128, 1, 4, 4, 0),
    "bf16 d128 pages of 16": ("bf16", 128, 16, 8, 2, 16),
    "bf16 d128 pages of 2": ("bf16", 128, 7, 3, 1, 2),
    "bf16 d128 256 rows": ("bf16", 128, 64, 4, 1, 0),
    "bf16 d128 520 rows pages of 64": ("bf16", 128, 65 - 13, 10, 1, 64),
    "bf16 d64": ("bf16", 64, 5, 8, 2, 0),
    "bf16 d64 320 rows pages of 8": ("bf16", 64, 40, 8, 1, 8),
    "fp32 d64": ("fp32", 64, 8, 4, 1, 0),
    "fp32 d64 pages of 1": ("fp32", 64, 9, 8, 1, 1),
}
RULES = {
    "plain": (dict(), 1.0),
    "cap and decay": (dict(softcap=20.0, gain=4.0), 0.75),
    "window and start": (dict(window=70, start=[0, 1, 40, 64, 70, 100, 128, 500, -3]), 1.0),
    "all, forgetting": (dict(softcap=20.0, slopes=True, window=90, start=[0, 0, 9, 64, 3, 100, 127, 128, 250]), 0.0),
}


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("form", FORMS)
def test_matches_the_definition(form, rule):
    dtype, D, T, Hq, Hkv, page = FORMS[form]
    kw, decay = RULES[rule]
    i = list(FORMS).index(form)
    L = [0, 1, 63, 64, 65, 127, 128, 129, 300]
    c = shaped.make(11 * i + len(rule), L, T, Hq, Hkv, D, dtype, page, **kw)
    accept = [(3 * b + i) % (T + 1) for b in range(len(L))]
    path, acc, lse, weight = _inputs(c, i, accept)
    ws = va.Workspace(256)
    w = shaped.dev(weight)
    shaped.run_weight(va, c, shaped.dev(lse), w, path=shaped.dev(path), n_accept=shaped.dev(acc), decay=decay,
                      workspace=ws)
    va.verify_attn_check_status(ws)
    _check(w.cpu().numpy(), shaped.accumulate(c, path, acc, lse, decay, weight), c, acc, weight)


def test_a_whole_block_without_path():
    """path and n_accept omitted: every token counts, a plain chain."""
    c = shaped.make(3, [200, 0], 8, 8, 2)
    path = np.tile(np.arange(8, dtype=np.int32), (2, 1))
    acc = np.full(2, 8, np.int32)
    _, lse = shaped.attend(c)
    lse = lse.astype(np.float32)
    weight = np.random.default_rng(0).random((2, 2, c.cap)).astype(np.float32)
    w = shaped.dev(weight)
    shaped.run_weight(va, c, shaped.dev(lse), w)
    _check(w.cpu().numpy(), shaped.accumulate(c, path, acc, lse, 1.0, weight), c, acc, weight)
    # each row's weights sum to 1: what a step adds is its rows
    added = w.cpu().numpy().astype(np.float64)
    added[0, :, :200] -= weight[0, :, :200]
    assert np.allclose(added[0, :, :208].sum(-1), 4 * 8, rtol=1e-4)


def test_new_slots_start_from_nothing_and_stale_totals_may_be_nan():
    c = shaped.make(3, [130], 4, 4, 1)
    path, acc, lse, weight = _inputs(c, 1, [3])
    want = shaped.accumulate(c, path, acc, lse, 1.0, weight)
    weight[0, :, 130:] = np.nan
    w = shaped.dev(weight)
    shaped.run_weight(va, c, shaped.dev(lse), w, path=shaped.dev(path), n_accept=shaped.dev(acc))
    got = w.cpu().numpy()
    assert np.allclose(got[0, :, :133], want[0, :, :133], rtol=2e-4, atol=1e-7)
    assert np.isnan(got[0, :, 133:]).all()


@pytest.mark.parametrize("form", ["bf16 d128", "bf16 d64", "fp32 d64"])
@pytest.mark.parametrize("kw", [dict(), dict(window=30)], ids=["plain", "window"])
def test_decay_zero_does_not_read_the_old_totals(form, kw):
    """Totals that were never written (NaN) are replaced, where rows see the key
    and where none does, and in a step that accepts nothing."""
    dtype, D, T, Hq, Hkv, page = FORMS[form]
    c = shaped.make(5, [400, 60], T, Hq, Hkv, D, dtype, page, **kw)
    path, acc, lse, weight = _inputs(c, 1, [4, 0])
    weight[:] = 0.0
    want = shaped.accumulate(c, path, acc, lse, 0.0, weight)
    w = shaped.dev(weight)
    for b, n in enumerate([400, 60]):
        w[b, :, :n] = float("nan")
    shaped.run_weight(va, c, shaped.dev(lse), w, path=shaped.dev(path), n_accept=shaped.dev(acc), decay=0.0)
    _check(w.cpu().numpy(), want, c, acc, weight)


@pytest.mark.parametrize("page", [0, 16, 2])
def test_hidden_keys_and_rows_without_keys(page):
    """NaN keys below the window, -1 page entries there, and rows whose lse is
    -inf: they add nothing."""
    c = shaped.make(5, [400, 60], 4, 4, 2, page=page, window=30)
    path, acc, lse, weight = _inputs(c, 1, [4, 2])
    lse[0, 1, path[0, 2]] = -np.inf
    want = shaped.accumulate(c, path, acc, lse, 0.5, weight)
    for b, n in enumerate([400, 60]):
        for j in range(n - 30 + 1):
            if page:
                c.k[c.table[b][j // page], j % page] = float("nan")
            else:
                c.k[b, j] = float("nan")
        if page:
            c.table[b, : (n - 30 + 1) // page] = -1
    ws = va.Workspace(256)
    w = shaped.dev(weight)
    shaped.run_weight(va, c, shaped.dev(lse), w, path=shaped.dev(path), n_accept=shaped.dev(acc), decay=0.5,
                      workspace=ws)
    va.verify_attn_check_status(ws)
    _check(w.cpu().numpy(), want, c, acc, weight)


def test_long_prefix_and_determinism():
    c = shaped.make(8, [20000], 8, 8, 2, softcap=30.0, gain=2.0)
    path, acc, lse, weight = _inputs(c, 2, [5])
    runs = []
    for _ in range(2):
        w = shaped.dev(weight)
        shaped.run_weight(va, c, shaped.dev(lse), w, path=shaped.dev(path), n_accept=shaped.dev(acc))
        runs.append(w.cpu().numpy())
    assert np.array_equal(runs[0], runs[1])
    _check(runs[0], shaped.accumulate(c, path, acc, lse, 1.0, weight), c, acc, weight)


def test_bad_lengths_counts_and_paths_are_recorded():
    """A sequence that does not fit is left alone, a bad path entry adds nothing."""
    c = shaped.make(3, [100, 100, 100], 4, 4, 1)
    path, acc, lse, weight = _inputs(c, 1, [3, 3, 3])
    want = shaped.accumulate(c, path, acc, lse, 1.0, weight)
    gone = lse.copy()
    gone[2, :, path[2, 1]] = -np.inf
    want2 = shaped.accumulate(c, path, acc, gone, 1.0, weight)
    L = c.L.copy()
    L[0] = c.cap
    acc[1], path[2, 1] = 5, 99
    c.L = L
    ws = va.Workspace(256)
    w = shaped.dev(weight)
    shaped.run_weight(va, c, shaped.dev(lse), w, path=shaped.dev(path), n_accept=shaped.dev(acc), workspace=ws)
    with pytest.raises(va.VerifyAttnError) as ei:
        va.verify_attn_check_status(ws)
    assert ei.value.status == va.api.VA_ERR_DEVICE_BOUNDS
    got = w.cpu().numpy()
    assert np.array_equal(got[:2], weight[:2])
    assert np.allclose(got[2, :, :103], want2[2, :, :103], rtol=2e-4, atol=1e-7)
    assert not np.allclose(want2[2], want[2], rtol=2e-4, atol=1e-7)


def test_captured_graph():
    c = shaped.make(8, [700], 8, 8, 2)
    path, acc, lse, weight = _inputs(c, 2, [5])
    mod, L = shaped.mod_of(va, c), shaped.dev(c.L)
    q, k, l, pa, na, w = c.q.cuda(), c.k.cuda(), shaped.dev(lse), shaped.dev(path), shaped.dev(acc), shaped.dev(weight)
    va.verify_accumulate_weight_dense(q, k, L, l, w, mod=mod, path=pa, n_accept=na)
    once = w.cpu().numpy()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        va.verify_accumulate_weight_dense(q, k, L, l, w, mod=mod, path=pa, n_accept=na)
    w.copy_(torch.from_numpy(weight))
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(w.cpu().numpy(), once)
