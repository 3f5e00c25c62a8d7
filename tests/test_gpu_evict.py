"""Eviction: the kept rows move exactly (bit for bit), everything behind the new
length stays as it was."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests.shaped import dev

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)


def _keep(rng, L, Hkv, n, kind):
    out = []
    for _ in range(Hkv):
        if kind == "front":      # nothing moves
            s = np.arange(n)
        elif kind == "back":     # every row moves as far as it can
            s = np.arange(L - n, L)
        elif kind == "one":      # every row moves by one slot: the tightest overlap
            s = np.arange(n) + (L > n)
        else:
            s = np.sort(rng.permutation(L)[:n])
        out.append(s)
    return np.stack(out) if n else np.zeros((Hkv, 0), int)


def _make(seed, L, keep, Hkv, D, dtype, page, kind, max_indices=None, weight=True):
    rng = np.random.default_rng(seed)
    B = len(L)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    m = max_indices or max(max(keep), 1)
    idx = np.full((B, Hkv, m), -1, np.int32)
    n = np.zeros((B, Hkv), np.int32)
    for b in range(B):
        idx[b, :, : keep[b]] = _keep(rng, L[b], Hkv, keep[b], kind)
        n[b] = keep[b]
    table = None
    if page:
        need = [max(1, -(-x // page)) for x in L]
        perm = rng.permutation(sum(need) + 1).astype(np.int32)
        table = np.full((B, max(need)), -1, np.int32)
        for b, x in enumerate(need):
            table[b, :x], perm = perm[:x], perm[x:]
        shape = (sum(need) + 1, page, Hkv, D)
        cap = max(need) * page
    else:
        cap = max(L) + 2
        shape = (B, cap, Hkv, D)
    k, v = (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dt) for _ in range(2))
    w = rng.random((B, Hkv, cap + 1)).astype(np.float32) if weight else None
    return idx, n, table, k, v, w


def _expect(L, idx, n, table, page, k, v, w):
    k2, v2 = k.clone(), v.clone()
    w2 = w.copy() if w is not None else None
    for b in range(len(L)):
        for h in range(k.shape[2]):
            src = idx[b, h, : n[b, h]].astype(np.int64)
            to = np.arange(n[b, h])
            if table is None:
                k2[b, to, h], v2[b, to, h] = k[b, src, h], v[b, src, h]
            else:
                t = table[b].astype(np.int64)
                k2[t[to // page], to % page, h] = k[t[src // page], src % page, h]
                v2[t[to // page], to % page, h] = v[t[src // page], src % page, h]
            if w is not None:
                w2[b, h, to] = w[b, h, src]
    return k2, v2, w2


def _run(L, idx, n, table, k, v, w, **kw):
    kd, vd, wd = k.cuda(), v.cuda(), dev(w) if w is not None else None
    args = (dev(np.asarray(L, np.int32)), dev(idx), dev(n))
    if table is None:
        new = va.verify_evict_kv_dense(kd, vd, *args, weight=wd, **kw)
    else:
        new = va.verify_evict_kv_paged(kd, vd, dev(table), *args, weight=wd, **kw)
    return kd.cpu(), vd.cpu(), wd.cpu().numpy() if wd is not None else None, new.cpu().numpy()


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("kind", ["random", "front", "back", "one"])
@pytest.mark.parametrize("dtype,D,Hkv,page", [("bf16", 128, 2, 0), ("bf16", 64, 3, 16), ("fp32", 64, 1, 0),
                                              ("bf16", 8, 2, 0), ("fp32", 256, 2, 8), ("bf16", 128, 2, 1),
                                              ("bf16", 72, 1, 64)])
def test_kept_rows_move(dtype, D, Hkv, page, kind):
    L = [0, 1, 2, 130, 300, 1000, 257]
    keep = [0, 1, 1, 129, 64, 700, 257]
    case = _make(D + page, L, keep, Hkv, D, dtype, page, kind)
    idx, n, table, k, v, w = case
    ws = va.Workspace(256)
    got = _run(L, *case, workspace=ws)
    va.verify_attn_check_status(ws)
    k2, v2, w2 = _expect(L, idx, n, table, page, k, v, w)
    assert _same(got[0], k2) and _same(got[1], v2) and np.array_equal(got[2], w2)
    assert got[3].tolist() == keep


def test_long_sequences_share_the_gpu():
    """Enough rows that one kv-head's moves spread over many blocks, whose reads
    and writes overlap; several calls on one scratch."""
    L, keep = [20000, 9000], [15000, 8999]
    sc = va.EvictScratch(2, 4, 15000)
    for seed, kind in enumerate(["random", "one", "back", "random"]):
        case = _make(seed, L, keep, 4, 128, "bf16", 16 if seed % 2 else 0, kind)
        idx, n, table, k, v, w = case
        got = _run(L, *case, scratch=sc)
        k2, v2, w2 = _expect(L, idx, n, table, 16, k, v, w)
        assert _same(got[0], k2) and _same(got[1], v2) and np.array_equal(got[2], w2)
    assert int(sc.buffer[sc.offset:sc.offset + sc.nbytes].sum()) == 0


def test_without_weights():
    case = _make(0, [100], [40], 2, 128, "bf16", 0, "random", weight=False)
    got = _run([100], *case)
    k2, v2, _ = _expect([100], *case[:3], 0, *case[3:])
    assert _same(got[0], k2) and _same(got[1], v2)


def test_bad_counts_and_lengths_leave_the_sequence_alone():
    L = [100, 100, 100, 100]
    case = _make(0, L, [40] * 4, 2, 128, "bf16", 0, "random")
    idx, n, table, k, v, w = case
    n[0, 1] = 39           # kv-heads keep different numbers
    n[1] = 41              # more than max_indices
    n[2] = -1
    ws = va.Workspace(256)
    got = _run([100, 100, 100, 100], idx, n, table, k, v, w, workspace=ws)
    with pytest.raises(va.VerifyAttnError) as ei:
        va.verify_attn_check_status(ws)
    assert ei.value.status == va.api.VA_ERR_DEVICE_BOUNDS
    k2, v2, w2 = _expect(L, idx, np.array([[0, 0], [0, 0], [0, 0], [40, 40]]), None, 0, k, v, w)
    assert _same(got[0], k2) and _same(got[1], v2) and np.array_equal(got[2], w2)
    assert got[3].tolist() == [100, 100, 100, 40]


def test_bad_indices_and_pages_are_recorded():
    for what in ("index", "order", "page"):
        case = _make(0, [100], [40], 1, 128, "bf16", 16, "back")
        idx, n, table, k, v, w = case
        if what == "index":
            idx[0, 0, 7] = 100
        elif what == "order":
            idx[0, 0, 20] = 3  # below its own slot
        else:
            table[0, 5] = 10 ** 6
        ws = va.Workspace(256)
        _run([100], *case, workspace=ws)
        with pytest.raises(va.VerifyAttnError) as ei:
            va.verify_attn_check_status(ws)
        assert ei.value.status == va.api.VA_ERR_DEVICE_BOUNDS


def test_captured_graph_replays():
    L, keep = [3000], [1000]
    idx, n, table, k, v, w = _make(0, L, keep, 2, 128, "bf16", 0, "random")
    kd, vd, wd = k.cuda(), v.cuda(), dev(w)
    a = dev(np.asarray(L, np.int32)), dev(idx), dev(n)
    sc, new = va.EvictScratch(1, 2, 1000), torch.zeros(1, dtype=torch.int32, device="cuda")
    va.verify_evict_kv_dense(kd, vd, *a, weight=wd, seqlens_out=new, scratch=sc)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        va.verify_evict_kv_dense(kd, vd, *a, weight=wd, seqlens_out=new, scratch=sc)
    k2, v2, w2 = _expect(L, idx, n, table, 0, k, v, w)
    for _ in range(3):
        kd.copy_(k), vd.copy_(v), wd.copy_(torch.from_numpy(w))
        g.replay()
        torch.cuda.synchronize()
        assert _same(kd.cpu(), k2) and _same(vd.cpu(), v2) and np.array_equal(wd.cpu().numpy(), w2)
    assert int(new) == 1000
