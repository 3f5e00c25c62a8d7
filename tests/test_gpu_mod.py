"""GPU parity of attention with score shaping against a plain fp64 statement.

Tolerances.  bf16 outputs: each weight keeps about 16 bits where it is more
than 1/16 of its row and 8 bits below that, so an output of values |v| <= 6 is
off by less than 6 * 2^-9 / 16 plus what the scores' fp32 rounding moves, well
below 2e-3, and then rounds to bf16 (half a step of the value): the bar is 2e-3
plus that half step.  lse: the fp32 scores (|s| <= 100, some 2^-22 relative
from 128 products, the cap and the bias) move it by less than 1e-4; the bar is
1e-3.  fp32 (d 64): outputs within 1e-4 by the same score error.
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests import shaped
from tests.gpu_util import compare

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

EDGE = [0, 1, 63, 64, 65, 127, 128, 129, 300]
RULES = {
    "cap": dict(softcap=5.0, gain=3.0),
    "slopes": dict(slopes=True),
    "window": dict(window=70),
    "window of one": dict(window=1),
    "start": dict(start=[0, 1, 40, 64, 70, 100, 128, 500, -3]),
    "all": dict(softcap=20.0, slopes=True, window=90, start=[0, 0, 9, 64, 3, 100, 127, 128, 250], gain=4.0),
    "none": dict(),
}
# (dtype, D, T, Hq, Hkv, page): rows of one kv-head 1 to 512, every kernel and layout
FORMS = {
    "bf16 d128 1 row": ("bf16", 128, 1, 2, 2, 0),
    "bf16 d128 20 rows": ("bf16", 128, 5, 8, 2, 0),
    "bf16 d128 64 rows": ("bf16", 128, 16, 8, 2, 0),
    "bf16 d128 64 rows pages of 16": ("bf16", 128, 16, 8, 2, 16),
    "bf16 d128 21 rows pages of 2": ("bf16", 128, 7, 3, 1, 2),
    "bf16 d128 100 rows": ("bf16", 128, 25, 4, 1, 0),
    "bf16 d128 256 rows": ("bf16", 128, 64, 4, 1, 0),
    "bf16 d128 320 rows pages of 64": ("bf16", 128, 40, 8, 1, 64),
    "bf16 d128 132 rows pages of 1": ("bf16", 128, 33, 4, 1, 1),
    "bf16 d64 12 rows": ("bf16", 64, 3, 8, 2, 0),
    "bf16 d64 20 rows pages of 2": ("bf16", 64, 5, 4, 1, 2),
    "bf16 d64 64 rows pages of 16": ("bf16", 64, 16, 4, 1, 16),
    "bf16 d64 33 rows pages of 1": ("bf16", 64, 11, 3, 1, 1),
    "bf16 d64 80 rows pages of 8": ("bf16", 64, 20, 4, 1, 8),
    "fp32 d64 32 rows": ("fp32", 64, 8, 4, 1, 0),
    "fp32 d64 72 rows pages of 256": ("fp32", 64, 9, 8, 1, 256),
}


def _check(c, out, lse):
    ro, rl = shaped.attend(c)
    tol = dict(tol_out=1e-4, tol_lse=1e-4) if c.q.dtype == torch.float32 else {}
    compare(out, lse, {"out": ro, "lse": rl}, **tol)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("form", FORMS)
def test_matches_the_definition(form, rule):
    dtype, D, T, Hq, Hkv, page = FORMS[form]
    i = list(FORMS).index(form)
    draft = ["chain", "tree", "block", "empty"][(i + list(RULES).index(rule)) % 4]
    c = shaped.make(7 * i + len(rule), EDGE, T, Hq, Hkv, D, dtype, page, draft, **RULES[rule])
    shape = va.make_shape(c.B, T, Hq, Hkv, D, 0 if dtype == "bf16" else 2)
    ws = va.Workspace.for_shape(shape)
    out, lse = shaped.run_attend(va, c, workspace=ws)
    va.verify_attn_check_status(ws)
    _check(c, out, lse)


def test_no_rule_is_the_unshaped_call():
    """Without any rule the scores are scale * q.k: the plain call's result to
    the bars of both."""
    c = shaped.make(1, [2000, 77], 8, 8, 2)
    out, lse = shaped.run_attend(va, c, mod=va.ScoreMod())
    ref, ref_lse = va.verify_attn_dense(c.q.cuda(), c.k.cuda(), c.v.cuda(), shaped.dev(c.L), scale=c.scale)
    assert (out.float() - ref.float()).abs().max() <= 2 ** -8 * ref.float().abs().max()
    assert (lse - ref_lse).abs().max() <= 1e-5


@pytest.mark.parametrize("T,Hq,Hkv,D", [(8, 8, 2, 128), (64, 4, 1, 128), (3, 8, 2, 64), (5, 8, 2, 64), (16, 8, 2, 64)])
def test_split_over_many_ctas(T, Hq, Hkv, D):
    """A prefix long enough that one segment is cut over every CTA: partial
    results at very different biases are merged."""
    c = shaped.make(5, [9000], T, Hq, Hkv, D, draft="tree", softcap=30.0, slopes=True, gain=2.0)
    out, lse = shaped.run_attend(va, c)
    _check(c, out, lse)


@pytest.mark.parametrize("rule", ["all", "cap", "window", "none"])
@pytest.mark.parametrize("T,Hq,Hkv,page", [(1, 1, 1, 0), (4, 4, 1, 1), (8, 4, 2, 16), (6, 10, 2, 0), (8, 8, 1, 4),
                                           (16, 9, 1, 0)])
def test_fp32_rows_and_key_groups(rule, T, Hq, Hkv, page):
    """fp32 with 1 to 144 rows of a kv-head: 16, 32 and 64 rows a segment, whose keys
    eight, four and two threads of a row share; NaN in the K and V rows that nobody sees."""
    kw = dict(RULES[rule])
    L = [0, 1, 63, 64, 65, 200, 1500]
    if "start" in kw:
        kw["start"] = [0, 1, 40, 64, 0, 100, 1400]
    c = shaped.make(5 * T + Hq, L, T, Hq, Hkv, 64, "fp32", page, ["tree", "block", "empty", "chain"][T % 4], **kw)
    ro, rl = shaped.attend(c)
    if not page:
        for b, n in enumerate(L):
            c.k[b, n + T:], c.v[b, n + T:] = float("nan"), float("inf")
            lo = max(int(c.start[b]), int(c.pos[b].min()) - c.window + 1 if c.window else 0, 0)
            c.k[b, :min(lo, n)], c.v[b, :min(lo, n)] = float("nan"), float("nan")
    ws = va.Workspace.for_shape(va.make_shape(c.B, T, Hq, Hkv, 64, 2))
    out, lse = shaped.run_attend(va, c, workspace=ws)
    va.verify_attn_check_status(ws)
    compare(out, lse, {"out": ro, "lse": rl}, tol_out=1e-4, tol_lse=1e-4)


@pytest.mark.parametrize("rule", ["all", "cap", "window", "none"])
@pytest.mark.parametrize("T,Hq,Hkv,page,L", [(17, 8, 2, 0, [9000]), (40, 3, 1, 16, [300, 0, 77]), (64, 8, 1, 2, [130, 65]),
                                             (1, 96, 1, 0, [2000, 1]), (3, 70, 1, 64, [129, 4000]),
                                             (64, 10, 2, 0, [0, 600])])
def test_d64_blocks_of_rows(rule, T, Hq, Hkv, page, L):
    """d 64 above 64 rows: blocks of 64, which may begin and end inside a token's heads."""
    kw = dict(RULES[rule])
    if "start" in kw:
        kw["start"] = [0, 64, 3][:len(L)]
    c = shaped.make(3 * T + Hq, L, T, Hq, Hkv, 64, "bf16", page, ["tree", "block", "empty"][T % 3], **kw)
    ws = va.Workspace.for_shape(va.make_shape(c.B, T, Hq, Hkv, 64, 0))
    out, lse = shaped.run_attend(va, c, workspace=ws)
    va.verify_attn_check_status(ws)
    _check(c, out, lse)


@pytest.mark.parametrize("T,Hq,Hkv,D,page", [(8, 8, 2, 128, 0), (8, 8, 2, 128, 16), (6, 8, 2, 128, 2),
                                              (64, 4, 1, 128, 0), (5, 4, 1, 64, 8), (9, 6, 1, 64, 0), (24, 4, 1, 64, 0)])
def test_hidden_keys_may_hold_anything(T, Hq, Hkv, D, page):
    """NaN and infinities in every K and V row that no row sees, and -1 in the
    page entries below the lowest visible slot."""
    L = [700, 130, 0, 64]
    c = shaped.make(9, L, T, Hq, Hkv, D, "bf16", page, "chain", window=40, start=[0, 128, 0, 64], softcap=30.0)
    ro, rl = shaped.attend(c)
    k, v = c.k.clone(), c.v.clone()
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")])
    for b, n in enumerate(L):
        lo = min(n, max(int(c.start[b]), n - c.window + 1, 0))
        hidden = list(range(lo)) + list(range(n + T, c.cap))
        for j in hidden:
            if page:
                e = int(c.table[b][j // page]) if j // page < c.table.shape[1] else -1
                if e < 0:
                    continue
                k[e, j % page], v[e, j % page] = bad[j % 3], bad[(j + 1) % 3]
            else:
                k[b, j], v[b, j] = bad[j % 3], bad[(j + 1) % 3]
        if page:
            c.table[b, : lo // page] = -1
    c.k, c.v = k, v
    ws = va.Workspace.for_shape(va.make_shape(c.B, T, Hq, Hkv, D, 0))
    out, lse = shaped.run_attend(va, c, workspace=ws)
    va.verify_attn_check_status(ws)
    compare(out, lse, {"out": ro, "lse": rl})


def test_draft_keys_that_nobody_sees_may_hold_anything():
    c = shaped.make(3, [100], 8, 8, 2, draft="block")
    c.draft[:, :, 5] = False
    import workloads as W
    c.words = W.pack_bits(c.draft)
    ro, rl = shaped.attend(c)
    c.k[0, 105], c.v[0, 105] = float("nan"), float("inf")
    out, lse = shaped.run_attend(va, c)
    compare(out, lse, {"out": ro, "lse": rl})


@pytest.mark.parametrize("reach", [1e-4, 0.1, 0.44, 0.74, 1.5, 30.0])
@pytest.mark.parametrize("cap", [0.5, 50.0, 1e6])
@pytest.mark.parametrize("dtype,D,T,Hq,Hkv", [("bf16", 128, 1, 2, 2), ("bf16", 128, 5, 8, 2), ("bf16", 128, 16, 8, 2),
                                              ("bf16", 128, 25, 4, 1), ("bf16", 128, 64, 4, 1), ("bf16", 64, 8, 8, 2),
                                              ("bf16", 64, 24, 4, 1), ("fp32", 64, 8, 4, 1)])
def test_every_part_of_the_cap(dtype, D, T, Hq, Hkv, cap, reach):
    """Scores |s| / cap up to `reach`, each alone in its row (a window of one) and
    an exact product (one element of q is not zero), so that lse is the capped
    score.  The cap is good to 3.3e-7 of it, and y, its units and the way back
    round five times: 1e-6 of it, and 1e-6 for the row's sum (2^0 and log2 of it).
    The weight of such a key, exp(s - lse), is 1 to the same error and lse's
    rounding."""
    g = torch.Generator().manual_seed(T)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    B = 3
    L = torch.tensor([0, 70, 200], dtype=torch.int32)
    q = torch.zeros(B, T, Hq, D)
    col = torch.randint(D, (B, T, Hq), generator=g)
    q.scatter_(3, col[..., None], 2.0)
    k = ((torch.rand(B, 200 + T, Hkv, D, generator=g) * 2 - 1) * (reach * cap / 2)).to(dt)
    v = torch.randn(B, 200 + T, Hkv, D, generator=g).to(dt)
    pos = L[:, None] + torch.arange(T, dtype=torch.int32)
    own = k.double()[torch.arange(B)[:, None], pos.long()]  # [B][T][Hkv][D]: each token's own key
    raw = 2.0 * own.repeat_interleave(Hq // Hkv, 2).gather(3, col[..., None])[..., 0]
    s = (cap * torch.tanh(raw / cap)).transpose(1, 2)  # [B][Hq][T]
    mod = va.ScoreMod(softcap=cap, window=1, token_pos=pos.cuda())
    out, lse = va.verify_attn_dense_mod(q.to(dt).cuda(), k.cuda(), v.cuda(), L.cuda(), mod, scale=1.0)
    err = (lse.cpu().double() - s).abs()
    assert (err <= 1e-6 * s.abs() + 1e-6).all(), float((err / (s.abs() + 1)).max())
    vals = v[torch.arange(B)[:, None], pos.long()].repeat_interleave(Hq // Hkv, 2)
    assert (out.cpu().float() - vals.float()).abs().max() <= 2 ** -8 * 6
    if cap > 100.0:  # (lse's own rounding is too much of exp's argument)
        return
    w = torch.zeros(B, Hkv, 200 + T, device="cuda")
    va.verify_accumulate_weight_dense(q.to(dt).cuda(), k.cuda(), L.cuda(), s.float().contiguous().cuda(), w, mod=mod,
                                      scale=1.0)
    got = w.cpu()[torch.arange(B)[:, None], :, pos.long()] / (Hq // Hkv)  # [B][T][Hkv]
    assert (got - 1).abs().max() <= 2e-6 * cap + 2e-6


def test_large_scores_stay_at_the_cap():
    """Products far past the cap, both signs, and the largest finite ones: all
    weights of a row are then 0 or equal."""
    c = shaped.make(2, [257], 4, 4, 1, softcap=10.0, gain=2000.0)
    out, lse = shaped.run_attend(va, c)
    _check(c, out, lse)
    assert torch.isfinite(lse).all() and float(lse.max()) <= 10 + np.log(261) + 1e-3


def test_positions_out_of_range_are_recorded():
    c = shaped.make(2, [200], 2, 2, 1, window=10)
    c.pos = c.pos + np.int32(1 << 24)
    ws = va.Workspace.for_shape(va.make_shape(1, 2, 2, 1, 128, 0))
    shaped.run_attend(va, c, workspace=ws)
    with pytest.raises(va.VerifyAttnError) as ei:
        va.verify_attn_check_status(ws)
    assert ei.value.status == va.api.VA_ERR_DEVICE_BOUNDS


def test_bad_visible_page_is_recorded():
    c = shaped.make(2, [200], 2, 2, 1, page=16, window=50)
    c.table[0, 200 // 16] = 10 ** 6
    ws = va.Workspace.for_shape(va.make_shape(1, 2, 2, 1, 128, 0))
    shaped.run_attend(va, c, workspace=ws)
    with pytest.raises(va.VerifyAttnError) as ei:
        va.verify_attn_check_status(ws)
    assert ei.value.status == va.api.VA_ERR_DEVICE_BOUNDS


def test_captured_graph_and_side_stream():
    """A captured call replays on new contents of its inputs; a call on another
    stream with its own workspace gives the same."""
    c = shaped.make(4, [600, 33], 8, 8, 2, draft="tree", softcap=30.0, slopes=True, window=200)
    d = shaped.make(6, [600, 33], 8, 8, 2, draft="tree", softcap=30.0, slopes=True, window=200)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    L, parent, mod = shaped.dev(c.L), shaped.dev(c.parent), shaped.mod_of(va, c)
    shape = va.make_shape(2, 8, 8, 2, 128, 0)
    ws = va.Workspace.for_shape(shape)
    out, lse = torch.empty_like(q), torch.empty(2, 8, 8, device="cuda")
    args = dict(tree_parent=parent, out=out, lse=lse, scale=c.scale)
    va.verify_attn_dense_mod(q, k, v, L, mod, workspace=ws, **args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        va.verify_attn_dense_mod(q, k, v, L, mod, workspace=ws, **args)
    q.copy_(d.q), k.copy_(d.k), v.copy_(d.v), parent.copy_(torch.from_numpy(d.parent))
    mod.token_pos.copy_(torch.from_numpy(d.pos))
    g.replay()
    torch.cuda.synchronize()
    _check(d, out, lse)
    first = out.clone(), lse.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    va.verify_attn_dense_mod(q, k, v, L, mod, stream=s, **args)
    s.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_workspace_shared_with_the_unshaped_calls():
    c = shaped.make(4, [900], 8, 8, 2, softcap=30.0)
    ws = va.Workspace.for_shape(va.make_shape(1, 64, 8, 2, 128, 0))
    for _ in range(3):
        out, lse = shaped.run_attend(va, c, workspace=ws)
        va.verify_attn_dense(c.q.cuda(), c.k.cuda(), c.v.cuda(), shaped.dev(c.L), workspace=ws)
    va.verify_attn_check_status(ws)
    _check(c, out, lse)


@pytest.mark.parametrize("T,Hq,Hkv,D", [(8, 8, 2, 128), (16, 8, 2, 128), (64, 4, 1, 128), (8, 8, 2, 64)])
def test_timeout_then_recovery(T, Hq, Hkv, D):
    """A lost part of a split segment ends in the documented error within the
    wait limit, and a fresh workspace gives the right result again."""
    c = shaped.make(5, [5000], T, Hq, Hkv, D, draft="tree", softcap=30.0, slopes=True)
    shape = va.make_shape(1, T, Hq, Hkv, D, 0)
    ws = va.Workspace.for_shape(shape)
    L = va.api.lib()
    assert L.verify_attn_test_inject(2_000_000, 0) == 0
    try:
        shaped.run_attend(va, c, workspace=ws)
        with pytest.raises(va.VerifyAttnError) as ei:
            va.verify_attn_check_status(ws)
        assert ei.value.status == va.api.VA_ERR_TIMEOUT
    finally:
        assert L.verify_attn_test_inject(0, -1) == 0
    ws = va.Workspace.for_shape(shape)
    out, lse = shaped.run_attend(va, c, workspace=ws)
    va.verify_attn_check_status(ws)
    _check(c, out, lse)


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its own workspace."""
    cs = [shaped.make(s, [3000, 40], 8, 8, 2, softcap=30.0, window=500) for s in (1, 2)]
    args, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c in cs:
        ws = va.Workspace.for_shape(va.make_shape(2, 8, 8, 2, 128, 0))
        args.append((c.q.cuda(), c.k.cuda(), c.v.cuda(), shaped.dev(c.L), shaped.mod_of(va, c), ws,
                     torch.empty(2, 8, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 8, 8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for (q, k, v, L, m, ws, out, lse), s in zip(args, streams):
            va.verify_attn_dense_mod(q, k, v, L, m, out=out, lse=lse, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c, a in zip(cs, args):
        _check(c, a[6], a[7])


def test_python_refusals():
    """Tensors of another type, shape or order are refused before the call."""
    c = shaped.make(1, [64], 4, 4, 2)
    q, k, v, L, mod = c.q.cuda(), c.k.cuda(), c.v.cuda(), shaped.dev(c.L), shaped.mod_of(va, c)
    call = va.verify_attn_dense_mod
    with pytest.raises(TypeError):
        call(q, k.float(), v, L, mod)
    with pytest.raises(TypeError):
        call(q, k, v, L.long(), mod)
    with pytest.raises(TypeError):
        call(q, k, v, L, None)
    with pytest.raises(TypeError):
        call(q, k, None, L, mod)
    with pytest.raises(ValueError):
        call(q, k[:, :-1], v, L, mod)
    with pytest.raises(ValueError):
        call(q, k, v, L, va.ScoreMod(slopes=torch.ones(3, device="cuda")))
    with pytest.raises(ValueError):
        call(q, k, v, L, va.ScoreMod(token_pos=L))
    with pytest.raises(ValueError):
        call(q.transpose(1, 2), k, v, L, mod)
    with pytest.raises(ValueError):
        call(torch.cat([q, q]), k, v, torch.cat([L, L]), mod)
    with pytest.raises(ValueError):
        call(q, k, v, L, mod, lse=torch.empty(1, 4, 5, device="cuda"))
