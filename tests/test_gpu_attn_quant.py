"""Attention over caches held in 8 or 4 bits against fp64 on the rows' exact values.

Tolerance, from the arithmetic.  Products of halves are exact in fp32 and a score's
128 additions leave at most 2^-16 of scale * sum |q_i k_i|, for these inputs below 16:
2.5e-4 of a score, so a weight is off by at most that plus 2^-12 (its rounding to half)
and twice as much after the division by the row sum (the sum itself has no rounded
weights, but its own scores' errors): 2 * 2.5e-4 + 2^-12 < 2^-10.  An output is then off
by 2^-10 sum w |v|, and by 2^-8 of itself when it is rounded to bf16; an lse by 2.5e-4
and a few fp32 roundings: 4e-4.
"""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
import workloads as W
from speculative_decoding_verification_masked_gb300 import api
from tests import quantized as Q

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

LSE = 4e-4


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


class Case:
    """A call's inputs, on the host and on the device.  mode: chain, tree, mask, empty
    (a mask with empty rows); page 0: dense.  Slots behind the draft rows, and pages
    that no sequence owns, hold 0xff bytes (NaN everywhere)."""

    def __init__(self, seed, fmt, D, L, T, Hq, Hkv, page=0, mode="chain", k=None, v=None, q=None):
        rng = np.random.default_rng(seed)
        self.fmt, self.D, self.L, self.T, self.Hq, self.Hkv, self.page = fmt, D, list(L), T, Hq, Hkv, page
        B = len(L)
        nb = Q.row_bytes(fmt, D)
        self.q = torch.from_numpy(rng.standard_normal((B, T, Hq, D)).astype(np.float32) if q is None else q).bfloat16()
        rows = {}
        for name, given in (("k", k), ("v", v)):
            rows[name] = [Q.store((given(rng, L[b] + T) if given is not None else
                                   rng.standard_normal((L[b] + T, Hkv, D)) * np.exp(0.3 * rng.standard_normal((L[b] + T, Hkv, 1)))),
                                  fmt) for b in range(B)]
        self.rows = rows
        if page:
            need = [-(-(n + T) // page) for n in L]
            perm = rng.permutation(sum(need) + 1).astype(np.int32)
            table = np.full((B, max(need)), -1, np.int32)
            for b, n in enumerate(need):
                table[b, :n], perm = perm[:n], perm[n:]
            shape = (sum(need) + 1, page, Hkv, nb)
        else:
            table, shape = None, (B, max(L) + T + 3, Hkv, nb)
        self.cache = {}
        for name in ("k", "v"):
            x = np.full(shape, 255, np.uint8)
            for b in range(B):
                slot = np.arange(L[b] + T)
                if page:
                    x[table[b, slot // page], slot % page] = rows[name][b]
                else:
                    x[b, : L[b] + T] = rows[name][b]
            self.cache[name] = torch.from_numpy(x).cuda()
        self.table = dev(table) if page else None
        self.parent = self.mask = None
        self.sees = np.tril(np.ones((T, T), bool))[None].repeat(B, 0)
        if mode == "tree":
            par = np.stack([W.random_parents(T, rng) for _ in range(B)])
            self.parent = dev(par)
            self.sees[:] = False
            for b in range(B):
                for i in range(T):
                    j = i
                    while j >= 0:
                        self.sees[b, i, j] = True
                        j = par[b, j]
        elif mode in ("mask", "empty"):
            self.sees = rng.random((B, T, T)) < 0.5
            if mode == "empty":
                self.sees[:, ::2] = False
                self.sees[:, :, T // 2:] = False  # the draft's second half is seen by nobody
            words = np.zeros((B, T, (T + 31) // 32), np.uint32)
            for j in range(T):
                words[:, :, j // 32] |= (self.sees[:, :, j].astype(np.uint32) << np.uint32(j % 32))
            self.mask = torch.from_numpy(words.view(np.int32)).cuda()

    def run(self, workspace=None, **kw):
        kw = dict(dict(tree_parent=self.parent, tree_mask=self.mask, workspace=workspace), **kw)
        qd, L = self.q.cuda(), dev(self.L)
        if self.page:
            return va.verify_attn_paged_quant(qd, self.cache["k"], self.cache["v"], self.table, L, self.fmt, **kw)
        return va.verify_attn_dense_quant(qd, self.cache["k"], self.cache["v"], L, self.fmt, **kw)

    def reference(self):
        B, T, Hq, D = self.q.shape
        G = Hq // self.Hkv
        q = self.q.double().numpy()
        out, mag, lse = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq, D)), np.full((B, Hq, T), -np.inf)
        for b in range(B):
            vis = np.concatenate([np.ones((T, self.L[b]), bool), self.sees[b]], 1)
            for h in range(Hq):
                k, v = (Q.read(self.rows[x][b][:, h // G], self.fmt, D) for x in ("k", "v"))
                z = np.where(vis, q[b, :, h] @ k.T / np.sqrt(D), -np.inf)
                some = vis.any(1)
                m = z[some].max(1)
                e = np.exp(z[some] - m[:, None])
                l = e.sum(1)
                lse[b, h, some] = m + np.log(l)
                v = np.where(vis.any(0)[:, None], v, 0.0)
                out[b, some, h] = e @ v / l[:, None]
                mag[b, some, h] = e @ np.abs(v) / l[:, None]
        return out, mag, lse

    def check(self, out, lse):
        ro, mag, rl = self.reference()
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(l), np.isneginf(rl)), "rows that see nothing differ"
        fin = np.isfinite(rl)
        assert bool(np.isfinite(o).all()), "outputs that are not finite"
        worst = float(np.abs(l[fin] - rl[fin]).max(initial=0))
        assert worst <= LSE, f"lse off by {worst:.3e}"
        over = np.abs(o - ro) - (2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * mag)
        assert float(over.max()) <= 0, f"off by {np.abs(o - ro).max():.3e}, {over.max():.3e} over the bar"


FORMATS = [("e4m3", 128), ("e2m1", 128), ("e4m3", 64), ("e2m1", 64)]


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("page", [0, 1, 4, 8, 16, 128, 512])
def test_ragged_batches(fmt, D, page):
    c = Case(page, fmt, D, [0, 1, 127, 128, 129, 300, 700], 5, 8, 2, page, "tree")
    c.check(*c.run())


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 8, 1), (3, 5, 1), (8, 12, 3), (16, 4, 4), (13, 10, 2), (16, 4, 1),
                                      (33, 8, 4), (64, 2, 2), (64, 8, 2), (64, 7, 1)])
@pytest.mark.parametrize("mode", ["chain", "mask"])
def test_rows_from_one_to_several_blocks(fmt, D, T, Hq, Hkv, mode):
    c = Case(T, fmt, D, [45, 260], T, Hq, Hkv, 0, mode)
    c.check(*c.run())


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("L,T,Hq,Hkv,page", [(40000, 8, 8, 2, 0), (5001, 1, 4, 1, 64), (20000, 40, 4, 1, 16), (9000, 64, 8, 2, 0)])
def test_long_prefix_split_over_the_gpu(fmt, D, L, T, Hq, Hkv, page):
    c = Case(L, fmt, D, [L], T, Hq, Hkv, page, "tree")
    c.check(*c.run())


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("page", [0, 16])
def test_rows_that_see_nothing_and_hidden_bytes(fmt, D, page):
    """Empty mask rows with and without a prefix; draft keys that nobody sees hold 0xff."""
    c = Case(3, fmt, D, [0, 4, 200], 9, 4, 2, page, "empty")
    T = c.T
    for name in ("k", "v"):
        for b, n in enumerate(c.L):
            for j in range(T // 2, T):
                slot = n + j
                if page:
                    c.cache[name][c.table[b, slot // page].long(), slot % page] = 255
                else:
                    c.cache[name][b, slot] = 255
    out, lse = c.run()
    c.check(out, lse)
    assert (out[0, ::2] == 0).all() and torch.isneginf(lse[0, :, ::2]).all()


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("T,Hq", [(4, 4), (10, 2), (16, 4), (64, 4)])
def test_references_that_move(fmt, D, T, Hq):
    """Scores that rise and fall by far more than 2^8 along the prefix, value rows whose
    scales differ by 2^16, the largest of them late."""
    def keys(rng, n):
        x = rng.standard_normal((n, 1, D))
        return x * (1 + 3 * np.abs(np.sin(np.arange(n) / 200.0)))[:, None, None]

    def vals(rng, n):
        return rng.standard_normal((n, 1, D)) * 2.0 ** rng.integers(-8, 8, size=(n, 1, 1)) * (1 + np.arange(n) / 100)[:, None, None]

    c = Case(T, fmt, D, [900, 130, 37], T, Hq, 1, 0, "chain", keys, vals)
    c.q = (c.q.float() * 0.6).bfloat16()
    c.check(*c.run())


@pytest.mark.parametrize("fmt,D", FORMATS)
def test_rows_on_a_few_keys(fmt, D):
    """A few keys carry every row; their values are 30 times the others'."""
    def keys(rng, n):
        x = rng.standard_normal((n, 2, D)) * 0.5
        x[5::97] = 1.0
        return x

    def vals(rng, n):
        x = rng.standard_normal((n, 2, D)) * 0.3
        x[5::97] *= 30
        return x

    rng = np.random.default_rng(0)
    q = (rng.standard_normal((2, 8, 8, D)) * 0.3 + 12.0 / np.sqrt(D)).astype(np.float32)
    c = Case(7, fmt, D, [650, 3000], 8, 8, 2, 0, "chain", keys, vals, q)
    c.check(*c.run())


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("T", [4, 40])
def test_a_nan_stays_in_its_rows(fmt, D, T):
    """A NaN in a query row, and a draft row stored as NaN, make the rows that hold or see
    them NaN and no others."""
    c = Case(1, fmt, D, [300, 20], T, 4, 2, 0, "chain")
    plain, plain_lse = c.run()
    c.q[0, 1, 2, 7] = float("nan")
    out, lse = c.run()
    assert torch.isnan(out[0, 1, 2]).all() and torch.isnan(lse[0, 2, 1])
    rest = torch.ones(out.shape[:3], dtype=torch.bool)
    rest[0, 1, 2] = False
    assert torch.equal(out[rest], plain[rest])
    c.q[0, 1, 2, 7] = 0.5
    at = Q.row_bytes(fmt, D) - 16 + (0 if fmt == "e4m3" else D // 16)
    for name in ("k", "v"):
        save = c.cache[name].clone()
        c.cache[name][1, 20 + 2, 1] = 0
        c.cache[name][1, 20 + 2, 1, at:at + 4] = torch.tensor([0, 0, 192, 127], dtype=torch.uint8)
        out, lse = c.run()
        nan = torch.isnan(out).any(-1)
        want = torch.zeros_like(nan)
        want[1, 2:, 2:] = True
        assert torch.equal(nan, want) and (name == "v" or torch.equal(torch.isnan(lse), want.transpose(1, 2)))
        c.cache[name] = save


def test_large_and_small_queries():
    """Queries of 2^30 and 2^-30 beside one another, and scales to match."""
    c = Case(2, "e2m1", 128, [200], 4, 4, 2)
    for f in (2.0 ** 60, 2.0 ** -60):
        d = Case(2, "e2m1", 128, [200], 4, 4, 2)
        d.q = (c.q.float() * f).bfloat16()
        out, lse = d.run(scale=1 / (f * 128 ** 0.5))
        c.check(out, lse)


@pytest.mark.parametrize("shift", [4, 8])
def test_unaligned_outputs(shift):
    c = Case(5, "e2m1", 128, [30, 0], 5, 4, 2, 16, "tree")
    out = torch.zeros(2 * 5 * 4 * 128 + 16, dtype=torch.bfloat16, device="cuda")[shift:][: 2 * 5 * 4 * 128].view(2, 5, 4, 128)
    got, lse = c.run(out=out)
    assert got.data_ptr() == out.data_ptr()
    c.check(got, lse)


def test_one_workspace_for_many_shapes_and_the_same_bits_again():
    ws = va.Workspace(64 << 20)
    for i, (fmt, D) in enumerate(FORMATS * 2):
        c = Case(i, fmt, D, [3000, 10, 700], 6 + 11 * (i % 3), 8, 2, 16 * (i % 2), "tree")
        a = c.run(ws)
        b = c.run(ws)
        c.check(*a)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        va.verify_attn_check_status(ws)


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("T,page", [(1, 0), (4, 64), (4, 4), (8, 0), (16, 64), (32, 0)])
def test_every_block_size_over_many_tiles_from_memory(fmt, D, T, page):
    """Caches past the L2, dozens of tiles to a CTA: stages go round many times, and rows
    land out of order.  The same bits every time."""
    g = torch.Generator("cuda").manual_seed(T)
    Hq, Hkv, L, ps = 32, 8, 131072, page or 131072 + 128
    nb, n = va.kv_row_bytes(fmt, D), (L + 128) // ps
    x = [torch.randn(n, ps, Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2)]
    cache = [torch.zeros(n, ps, Hkv, nb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    zero = torch.zeros(n, dtype=torch.int32, device="cuda")
    va.verify_quantize_kv_dense(*x, *cache, zero, fmt)
    rows = [torch.empty_like(y) for y in x]
    va.verify_dequantize_kv_dense(*cache, zero, fmt, k_out=rows[0], v_out=rows[1])
    table = torch.randperm(n, generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(1, T, Hq, D, generator=g, device="cuda").bfloat16()
    lens = torch.full((1,), L, dtype=torch.int32, device="cuda")
    ws = va.Workspace(64 << 20)

    def call():
        if page:
            return va.verify_attn_paged_quant(q, *cache, table[None], lens, fmt, workspace=ws)
        return va.verify_attn_dense_quant(q, *cache, lens, fmt, workspace=ws)

    out, lse = call()
    for _ in range(8):
        o, l = call()
        assert torch.equal(o, out) and torch.equal(l, lse)
    va.verify_attn_check_status(ws)
    k, v = (y[table.long()].reshape(-1, Hkv, D) if page else y[0] for y in rows)
    seen = torch.arange(L + T, device="cuda")[None] <= L + torch.arange(T, device="cuda")[:, None]
    for h in range(Hkv):
        kh, vh = k[: L + T, h].double(), v[: L + T, h].double()
        z = torch.einsum("tgd,kd->gtk", q[0, :, 4 * h:4 * h + 4].double(), kh) / D ** 0.5
        z = z.masked_fill(~seen, -torch.inf)
        w = torch.softmax(z, -1)
        want, mag = ((w @ y).transpose(0, 1) for y in (vh, vh.abs()))
        over = (out[0, :, 4 * h:4 * h + 4].double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -10 * mag)
        assert float(over.max()) <= 0
        assert float((lse[0, 4 * h:4 * h + 4].double() - torch.logsumexp(z, -1)).abs().max()) <= LSE


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("B,T", [(256, 1), (256, 16), (255, 32), (257, 4)])
def test_as_many_segments_as_a_call_takes(fmt, D, B, T):
    """2048 segments, whose plan takes 8 KB from the ring of stages; more are refused."""
    g = torch.Generator("cuda").manual_seed(B)
    Hq, Hkv, N = 16, 8, 300
    x = [torch.randn(B, N, Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2)]
    cache = [torch.zeros(B, N, Hkv, va.kv_row_bytes(fmt, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    va.verify_quantize_kv_dense(*x, *cache, zero, fmt)
    k, v = va.verify_dequantize_kv_dense(*cache, zero, fmt, N)
    q = torch.randn(B, T, Hq, D, generator=g, device="cuda").bfloat16()
    lens = torch.randint(0, N - T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if B * Hkv > 2048:
        with pytest.raises(va.VerifyAttnError):
            va.verify_attn_dense_quant(q, *cache, lens, fmt)
        return
    out, lse = va.verify_attn_dense_quant(q, *cache, lens, fmt)
    for b in range(0, B, 13):
        n = int(lens[b]) + T
        kb, vb = (y[b, :n].double().repeat_interleave(Hq // Hkv, 1) for y in (k, v))
        z = torch.einsum("thd,khd->htk", q[b].double(), kb) / D ** 0.5
        seen = torch.arange(n, device="cuda")[None] <= n - T + torch.arange(T, device="cuda")[:, None]
        z = z.masked_fill(~seen, -torch.inf)
        w = torch.softmax(z, -1)
        want, mag = (torch.einsum("htk,khd->thd", w, y) for y in (vb, vb.abs()))
        assert float(((out[b].double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -10 * mag)).max()) <= 0
        assert float((lse[b].double() - torch.logsumexp(z, -1)).abs().max()) <= LSE


def test_bad_lengths_and_pages_are_recorded():
    c = Case(1, "e2m1", 128, [100, 60], 4, 4, 2, 16)
    ws = va.Workspace(16 << 20)
    good, _ = c.run(ws)
    for L in ([100, -1], [100, 1 << 30]):
        save, c.L = c.L, L
        out, _ = c.run(ws)
        c.L = save
        with pytest.raises(va.VerifyAttnError) as e:
            va.verify_attn_check_status(ws)
        assert e.value.status == 6
        assert torch.equal(out[0], good[0])
    for page in (16, 4):
        d = Case(1, "e2m1", 128, [100, 60], 4, 4, 2, page)
        good, _ = d.run(ws)
        for entry in (-1, 1 << 20):
            save = d.table.clone()
            d.table[1, 1] = entry
            out, _ = d.run(ws)
            d.table = save
            with pytest.raises(va.VerifyAttnError) as e:
                va.verify_attn_check_status(ws)
            assert e.value.status == 6
            assert torch.equal(out[0], good[0])


def test_captured_calls_and_two_streams():
    """Two captured graphs, replayed at once on two streams with a workspace each, and
    plain calls between them."""
    cases = [Case(1, "e2m1", 128, [4000], 8, 8, 2, 0, "chain"), Case(2, "e4m3", 128, [900, 50], 40, 4, 2, 16, "tree")]
    graphs, outs = [], []
    for c in cases:
        ws = va.Workspace(16 << 20)
        qd, L = c.q.cuda(), dev(c.L)
        o, l = torch.empty_like(qd), torch.empty(len(c.L), c.Hq, c.T, device="cuda")
        f = va.verify_attn_paged_quant if c.page else va.verify_attn_dense_quant
        cache = (c.cache["k"], c.cache["v"]) + ((c.table,) if c.page else ())
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        f(qd, *cache, L, c.fmt, tree_parent=c.parent, out=o, lse=l, workspace=ws, stream=s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            f(qd, *cache, L, c.fmt, tree_parent=c.parent, out=o, lse=l, workspace=ws, stream=s)
        graphs.append((g, s, qd, ws))
        outs.append((o, l))
    for _ in range(20):
        for g, s, _, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, (o, l) in zip(cases, outs):
        c.check(o, l)
        want = c.run()
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_a_cache_past_two_billion_bytes():
    """Rows past 2^31 bytes of the pool, dense and paged."""
    fmt, D, Hkv, T, page = "e4m3", 128, 8, 3, 64
    c = Case(4, fmt, D, [500], T, 16, Hkv, page)
    n = (2 << 30) // (page * Hkv * 144) + 40
    pool = {x: torch.full((n, page, Hkv, 144), 255, dtype=torch.uint8, device="cuda") for x in ("k", "v")}
    for x in ("k", "v"):
        pool[x][n - c.cache[x].shape[0]:] = c.cache[x]
    c.table += n - c.cache["k"].shape[0]
    c.cache = pool
    c.check(*c.run())
    d = Case(4, fmt, D, [5, 500], T, 16, Hkv)
    cap = (2 << 30) // (Hkv * 144) + 600
    big = {x: torch.full((2, cap, Hkv, 144), 255, dtype=torch.uint8, device="cuda") for x in ("k", "v")}
    for x in ("k", "v"):
        big[x][:, : d.cache[x].shape[1]] = d.cache[x]
    d.cache = big
    d.check(*d.run())


def test_refused_tensors():
    c = Case(1, "e2m1", 128, [10], 2, 4, 2)
    f, q, k, v, L = va.verify_attn_dense_quant, c.q.cuda(), c.cache["k"], c.cache["v"], dev([10])
    for args in ((q.float(), k, v, L, "e2m1"), (q.cpu(), k, v, L, "e2m1"), (q, k.view(torch.int8), v, L, "e2m1"),
                 (q, k, v[:, :-1], L, "e2m1"), (q, k, v, L.long(), "e2m1"), (q, k, v, L, "e4m3"), (q, k, v, L, 1),
                 (q, k[..., ::2], v, L, "e2m1")):
        with pytest.raises((TypeError, ValueError, va.VerifyAttnError)):
            f(*args)
    with pytest.raises(va.VerifyAttnError):
        f(q, k, v, L, "e2m1", workspace=va.Workspace(1024))
