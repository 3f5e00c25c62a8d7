"""Plain fp64 statements of score-shaping attention, the accumulated attention
weight and the eviction, one (sequence, query head) at a time, and the inputs
their GPU tests share."""
import numpy as np
import torch

import workloads as W


def scores(q, keys, scale, softcap, slope, away):
    """q [D], keys [N][D], away [N] = pos_q - pos_k, all fp64."""
    z = scale * (keys @ q)
    if softcap:
        z = softcap * np.tanh(z / softcap)
    return z - slope * np.abs(away)


def visible_prefix(L, pos, window, start):
    j = np.arange(L)
    ok = j >= start
    if window:
        ok &= pos - j < window
    return ok


def attend(c):
    """(out [B][T][Hq][D], lse [B][Hq][T]) of a case (see make), in fp64."""
    q = c.q.double().numpy()
    B, T, Hq, D = q.shape
    group = Hq // c.Hkv
    out, lse = np.zeros((B, T, Hq, D)), np.full((B, Hq, T), -np.inf)
    for b in range(B):
        L = int(c.L[b])
        pos = c.pos[b]
        for h in range(Hq):
            keys, vals = c.rows(c.k, b, h // group, L + T), c.rows(c.v, b, h // group, L + T)
            for t in range(T):
                away = pos[t] - np.concatenate([np.arange(L), pos])
                see = np.concatenate([visible_prefix(L, pos[t], c.window, c.start[b]), c.draft[b, t]])
                if c.window:
                    see &= away < c.window
                if not see.any():
                    continue
                z = scores(q[b, t, h], keys[see], c.scale, c.softcap, c.slopes[h], away[see])
                m = z.max()
                e = np.exp(z - m)
                lse[b, h, t] = m + np.log(e.sum())
                out[b, t, h] = (e / e.sum()) @ vals[see]
    return out, lse


def accumulate(c, path, n_accept, lse, decay, weight):
    """The totals after a step, in fp64; weight [B][Hkv][stride]."""
    w = weight.astype(np.float64).copy()
    q = c.q.double().numpy()
    B, T, Hq, D = q.shape
    group = Hq // c.Hkv
    for b in range(B):
        L, a = int(c.L[b]), int(n_accept[b])
        w[b, :, :L] *= decay
        w[b, :, L:L + a] = 0.0
        for h in range(Hq):
            keys = c.rows(c.k, b, h // group, L + a)
            for i in range(a):
                t = int(path[b, i])
                if np.isneginf(lse[b, h, t]):
                    continue
                n = L + i + 1
                see = np.concatenate([visible_prefix(L, L + i, c.window, c.start[b]), np.ones(i + 1, bool)])
                away = L + i - np.arange(n)
                if c.window:
                    see &= away < c.window
                z = scores(q[b, t, h], keys[:n][see], c.scale, c.softcap, c.slopes[h], away[see])
                w[b, h // group, np.flatnonzero(see)] += np.exp(z - lse[b, h, t])
    return w


class Case:
    """A call's inputs on the CPU; rows() reads logical slots of either layout."""

    def rows(self, x, b, h, n):
        if self.table is None:
            return x[b, :n, h].double().numpy()
        j = np.arange(n)
        pages = torch.from_numpy(self.table[b][j // self.page].astype(np.int64))
        return x[pages, torch.from_numpy(j % self.page), h].double().numpy()


def make(seed, L, T, Hq, Hkv, D=128, dtype="bf16", page=0, draft="chain", softcap=0.0, window=0, slopes=False,
         start=None, gain=1.0, extra=3):
    """Inputs for prefixes L; `draft`: chain, tree, block, or empty (a mask whose
    even rows see nothing); start: per-sequence document starts."""
    rng = np.random.default_rng(seed)
    c = Case()
    B = len(L)
    c.B, c.T, c.Hq, c.Hkv, c.D = B, T, Hq, Hkv, D
    c.L = np.asarray(L, np.int32)
    c.page, c.softcap, c.window, c.scale = page, softcap, window, 1.0 / np.sqrt(D)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def normal(*shape, g=1.0):
        return torch.from_numpy((g * rng.standard_normal(shape)).astype(np.float32)).to(dt)

    c.q = normal(B, T, Hq, D, g=gain)
    if page:
        need = [-(-(n + T) // page) for n in L]
        c.table = np.full((B, max(need)), -1, np.int32)
        perm = rng.permutation(sum(need) + 2)
        for b, n in enumerate(need):
            c.table[b, :n], perm = perm[:n], perm[n:]
        shape = (sum(need) + 2, page, Hkv, D)
        c.cap = max(need) * page
    else:
        c.table = None
        c.cap = max(L) + T + extra
        shape = (B, c.cap, Hkv, D)
    c.k, c.v = normal(*shape), normal(*shape)
    c.has_slopes = slopes
    c.slopes = (2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)).astype(np.float32) if slopes else np.zeros(Hq, np.float32)
    c.has_start = start is not None
    c.start = np.asarray(start if start is not None else [0] * B, np.int32)
    c.parent = c.words = None
    off = np.tile(np.arange(T), (B, 1))
    c.draft = np.tile(np.tril(np.ones((T, T), bool)), (B, 1, 1))
    if draft == "tree":
        c.parent = np.stack([W.random_parents(T, rng) for _ in range(B)]).astype(np.int32)
        off = np.stack([W.chain_depths(p) for p in c.parent])
        for b in range(B):
            c.draft[b] = False
            for t in range(T):
                j = t
                while j >= 0:
                    c.draft[b, t, j] = True
                    j = c.parent[b, j]
    elif draft in ("block", "empty"):
        rows = W.block_draft_mask(T, 4, "causal")
        c.draft = np.tile(rows, (B, 1, 1)).astype(bool)
        if draft == "empty":
            c.draft[:, ::2] = False
        c.words = W.pack_bits(c.draft)
    c.pos = (c.L[:, None] + off).astype(np.int32)
    return c


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def mod_of(va, c):
    return va.ScoreMod(softcap=c.softcap, window=c.window, slopes=dev(c.slopes) if c.has_slopes else None,
                       key_start=dev(c.start) if c.has_start else None, token_pos=dev(c.pos))


def run_attend(va, c, mod=None, **kw):
    mod = mod or mod_of(va, c)
    kw.setdefault("scale", c.scale)
    if c.parent is not None:
        kw["tree_parent"] = dev(c.parent)
    if c.words is not None:
        kw["tree_mask"] = dev(c.words.view(np.int32))
    if c.table is not None:
        return va.verify_attn_paged_mod(c.q.cuda(), c.k.cuda(), c.v.cuda(), dev(c.table), dev(c.L), mod, **kw)
    return va.verify_attn_dense_mod(c.q.cuda(), c.k.cuda(), c.v.cuda(), dev(c.L), mod, **kw)


def run_weight(va, c, lse, weight, mod=None, **kw):
    mod = mod or mod_of(va, c)
    if c.table is not None:
        return va.verify_accumulate_weight_paged(c.q.cuda(), c.k.cuda(), dev(c.table), dev(c.L), lse, weight, mod=mod,
                                                 scale=c.scale, **kw)
    return va.verify_accumulate_weight_dense(c.q.cuda(), c.k.cuda(), dev(c.L), lse, weight, mod=mod, scale=c.scale,
                                             **kw)
