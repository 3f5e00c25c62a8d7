"""The score-shaping attention, the accumulated weight and the eviction as a
decoding loop uses them: verify, accept, commit, weigh, and cut the cache back
when it passes its budget, for several steps, against the plain fp64 statements
of every operator on the same state."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_verification_masked_gb300 as va
from tests import shaped
from tests.gpu_util import compare

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("page", [0, 16])
def test_decoding_with_a_bounded_cache(page):
    B, T, Hq, Hkv, budget, high = 2, 6, 8, 2, 96, 104
    c = shaped.make(40 + page, [100, 61], T, Hq, Hkv, page=page, draft="chain", softcap=20.0, slopes=True, gain=2.0,
                    extra=40)
    if page:  # room for what the steps append
        pages = c.k.shape[0]
        spare = np.arange(pages, pages + 2 * 4, dtype=np.int32).reshape(2, 4)
        c.table = np.concatenate([np.where(c.table < 0, pages - 1, c.table), spare], 1)
        # every entry its own page
        c.table = np.arange(c.table.size, dtype=np.int32).reshape(c.table.shape)
        c.cap = c.table.shape[1] * page
        rng = np.random.default_rng(0)
        c.k, c.v = (torch.from_numpy(rng.standard_normal((c.table.size, page, Hkv, 128)).astype(np.float32))
                    .to(torch.bfloat16) for _ in range(2))
    k, v = c.k.cuda(), c.v.cuda()
    table = shaped.dev(c.table) if page else None
    weight = np.zeros((B, Hkv, c.cap), np.float32)
    w = shaped.dev(weight)
    seqlens = shaped.dev(c.L)
    ws = va.Workspace.for_shape(va.make_shape(B, T, Hq, Hkv, 128, 0))
    sc = va.EvictScratch(B, Hkv, budget)
    rng = np.random.default_rng(3)
    evictions = 0
    for step in range(6):
        # the state as it is now, for the plain statements
        c.k, c.v, c.L = k.cpu(), v.cpu(), seqlens.cpu().numpy()
        c.q = torch.from_numpy(2 * rng.standard_normal((B, T, Hq, 128)).astype(np.float32)).to(torch.bfloat16)
        c.parent = np.stack([np.concatenate([[-1], [int(rng.integers(-1, t)) for t in range(1, T)]]) for _ in range(B)])
        c.parent = c.parent.astype(np.int32)
        depth = np.zeros((B, T), int)
        c.draft = np.zeros((B, T, T), bool)
        for b in range(B):
            for t in range(T):
                j = t
                while j >= 0:
                    c.draft[b, t, j] = True
                    j = c.parent[b, j]
                depth[b, t] = c.draft[b, t].sum() - 1
        c.pos = (c.L[:, None] + depth).astype(np.int32)
        # verify
        q, parent, mod = c.q.cuda(), shaped.dev(c.parent), shaped.mod_of(va, c)
        kv = (k, v, table) if page else (k, v)
        attend = va.verify_attn_paged_mod if page else va.verify_attn_dense_mod
        out, lse = attend(q, *kv, seqlens, mod, tree_parent=parent, workspace=ws, scale=c.scale)
        ro, rl = shaped.attend(c)
        compare(out, lse, {"out": ro, "lse": rl})
        # accept and commit
        tokens = rng.integers(0, 2, (B, T)).astype(np.int32)
        target = rng.integers(0, 2, (B, T + 1)).astype(np.int32)
        path, n_acc, _ = va.verify_accept_greedy(parent, shaped.dev(tokens), shaped.dev(target))
        commit = va.verify_commit_kv_paged if page else va.verify_commit_kv_dense
        new = commit(*kv, seqlens, path, n_acc)
        # weigh
        before = w.cpu().numpy()
        c.k = k.cpu()
        p_h, a_h = path.cpu().numpy(), n_acc.cpu().numpy()
        weigh = va.verify_accumulate_weight_paged if page else va.verify_accumulate_weight_dense
        weigh(q, *((k, table) if page else (k,)), seqlens, lse, w, mod=mod, path=path, n_accept=n_acc, decay=0.9,
              scale=c.scale, workspace=ws)
        want = shaped.accumulate(c, p_h, a_h, lse.cpu().numpy().astype(np.float64), 0.9, before)
        got = w.cpu().numpy()
        for b in range(B):
            n = int(c.L[b]) + int(a_h[b])
            assert np.allclose(got[b, :, :n], want[b, :, :n], rtol=2e-4, atol=1e-7)
        seqlens = new
        # cut back what has passed the high mark
        if int(seqlens.max()) >= high:
            evictions += 1
            idx, n = va.verify_build_index(seqlens, w, w, 4, 16, 0, budget, workspace=ws)
            L_h, w_h = seqlens.cpu().numpy(), w.cpu().numpy()
            want_idx, want_n = oracle.build_verify_index(w_h, w_h, L_h, 4, 16, 0, budget)
            assert np.array_equal(n.cpu().numpy(), want_n) and np.array_equal(idx.cpu().numpy(), want_idx)
            c.k, c.v = k.cpu(), v.cpu()
            evict = va.verify_evict_kv_paged if page else va.verify_evict_kv_dense
            seqlens = evict(*kv, seqlens, idx, n, weight=w, scratch=sc, workspace=ws)
            for b in range(B):
                for h in range(Hkv):
                    src = want_idx[b, h, : want_n[b, h]]
                    d = shaped.Case()
                    d.table, d.page = c.table, c.page
                    for old, now in ((c.k, k.cpu()), (c.v, v.cpu())):
                        rows = c.rows(old, b, h, int(L_h[b]))[src]
                        assert np.array_equal(d.rows(now, b, h, len(src)), rows)
                    assert np.array_equal(w.cpu().numpy()[b, h, : len(src)], w_h[b, h, src])
            assert np.array_equal(seqlens.cpu().numpy(), want_n[:, 0])
        va.verify_attn_check_status(ws)
    assert evictions >= 1
