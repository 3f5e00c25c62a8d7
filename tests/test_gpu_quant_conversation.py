"""The norm with rotation, the cache held in 8 or 4 bits, the attention over it, the
acceptance, the commit and the eviction together, as a serving loop runs them: a chunk
of prompts, steps of token trees, and a cache that is cut back.  After every step the
cache holds bit for bit what the definition gives for the rows that were written and
moved, and the attention is right on those rows."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
import workloads as W
from tests import quantized as Q
from tests.test_gpu_attn_quant import LSE, dev

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("fmt,D,page", [("e2m1", 128, 0), ("e4m3", 128, 16), ("e2m1", 64, 4), ("e4m3", 64, 0)])
def test_prompt_steps_and_eviction(fmt, D, page):
    rng = np.random.default_rng(D + page)
    B, Hq, Hkv, T, base = 3, 8, 2, 11, 500000.0
    L = [150, 0, 37]
    width, nb = 20 * 16, va.kv_row_bytes(fmt, D)
    if page:
        per = width // page
        table = dev(rng.permutation(B * per).reshape(B, per))
        shape, t = (B * per, page, Hkv, nb), [table]
        flat = lambda x: x[table.long()].reshape(B, width, Hkv, nb)  # noqa: E731
        name = "paged"
    else:
        shape, t, name = (B, width, Hkv, nb), [], "dense"
        flat = lambda x: x  # noqa: E731
    kc, vc = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    f = {n: getattr(va, f"verify_{n}_{name}") for n in ("quantize_kv", "dequantize_kv", "commit_kv", "evict_kv")}
    attend = getattr(va, f"verify_attn_{name}_quant")
    wq, wk = (torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).bfloat16().cuda() for _ in range(2))
    ws = va.Workspace.for_shape(va.make_shape(B, T, Hq, Hkv, D, 0))
    want = np.zeros((2, B, width, Hkv, nb), np.uint8)

    def project(n):
        x = torch.from_numpy(rng.standard_normal((B, n, Hq + 2 * Hkv, D)).astype(np.float32)).bfloat16().cuda()
        return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]

    def expect(rows, at, count):
        for i, x in enumerate(rows):
            b = Q.store(x.double().cpu().numpy(), fmt)
            for s in range(B):
                want[i, s, at[s]:at[s] + count[s]] = b[s, :count[s]]

    def check_cache():
        for i, x in enumerate((kc, vc)):
            Q.same_bytes(flat(x).cpu().numpy(), want[i], fmt, D)

    # the prompts, as one padded chunk
    n = max(L)
    q, k, v = project(n)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, n).contiguous()
    _, k = va.verify_norm_rope(q, k, wq, wk, pos, rope_base=base)
    zero = dev([0] * B)
    f["quantize_kv"](k, v, kc, vc, *t, zero, fmt, n_tokens=dev(L), workspace=ws)
    expect((k, v), [0] * B, L)
    check_cache()
    out = f["dequantize_kv"](kc, vc, *t, zero, fmt, n=n, n_tokens=dev(L), workspace=ws)
    for i in range(2):
        for b in range(B):
            assert torch.equal(out[i][b, :L[b]].cpu(), torch.from_numpy(Q.read(want[i, b, :L[b]], fmt, D)).bfloat16())

    for step in range(4):
        parent = np.stack([W.random_parents(T, rng) for _ in range(B)])
        depth = np.stack([W.chain_depths(p) for p in parent])
        pos = dev(np.asarray(L)[:, None] + depth)
        q, k, v = project(T)
        va.verify_norm_rope(q, k, wq, wk, pos, rope_base=base, q_out=q, k_out=k)  # in place, in the projection
        q = q.contiguous()
        seq = dev(L)
        f["quantize_kv"](k, v, kc, vc, *t, seq, fmt, workspace=ws)
        expect((k, v), L, [T] * B)
        check_cache()
        o, lse = attend(q, kc, vc, *t, seq, fmt, tree_parent=dev(parent), workspace=ws)
        G, qn = Hq // Hkv, q.double().cpu().numpy()
        for b in range(B):
            sees = np.zeros((T, T), bool)
            for i in range(T):
                j = i
                while j >= 0:
                    sees[i, j] = True
                    j = parent[b, j]
            vis = np.concatenate([np.ones((T, L[b]), bool), sees], 1)
            for h in range(Hq):
                kk, vv = (Q.read(want[i, b, :L[b] + T, h // G], fmt, D) for i in range(2))
                z = np.where(vis, qn[b, :, h] @ kk.T / np.sqrt(D), -np.inf)
                m = z.max(1, keepdims=True)
                e = np.exp(z - m)
                s = e.sum(1, keepdims=True)
                assert np.abs(lse[b, h].double().cpu().numpy() - (m + np.log(s))[:, 0]).max() <= LSE
                ref, mag = e @ vv / s, e @ np.abs(vv) / s
                err = np.abs(o[b, :, h].double().cpu().numpy() - ref)
                assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag).all()  # (see test_gpu_attn_quant)
        draft = rng.integers(0, 3, size=(B, T))
        target = rng.integers(0, 3, size=(B, T + 1))
        path, acc, _ = va.verify_accept_greedy(dev(parent), dev(draft), dev(target))
        new = f["commit_kv"](kc, vc, *t, seq, path, acc, workspace=ws)
        pn, an = path.cpu().numpy(), acc.cpu().numpy()
        for i in range(2):
            for b in range(B):
                moved = want[i, b, [L[b] + pn[b, j] for j in range(an[b])]].copy()
                want[i, b, L[b]:L[b] + an[b]] = moved
        L = [x + int(a) for x, a in zip(L, an)]
        assert new.tolist() == L
        check_cache()

    keep = [min(x, 100) for x in L]
    idx = np.full((B, Hkv, 100), -1, np.int32)
    for b in range(B):
        for h in range(Hkv):
            idx[b, h, :keep[b]] = np.sort(rng.permutation(L[b])[:keep[b]])
    kept = f["evict_kv"](kc, vc, *t, dev(L), dev(idx), dev([[x] * Hkv for x in keep]), workspace=ws)
    va.verify_attn_check_status(ws)
    assert kept.tolist() == keep
    for i, x in enumerate((kc, vc)):
        got = flat(x).cpu().numpy()
        for b in range(B):
            for h in range(Hkv):
                assert np.array_equal(got[b, :keep[b], h], want[i, b, idx[b, h, :keep[b]], h])
