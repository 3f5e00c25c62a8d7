"""Workloads of the score-shaping attention, the accumulated attention weight
and the cache eviction, in plain torch and through the library's entry points.

* ``attend`` -- verification attention whose scores are capped by a tanh, get a
  bias that falls with distance, or are cut by a sliding window or a document
  start (``verify_attn_dense_mod``, ``verify_attn_paged_mod``);
* ``weigh``  -- the attention weight the accepted tokens gave to every cached
  key, added to a running total per kv-head (``verify_accumulate_weight_*``);
* ``evict``  -- the rows of a keep set moved to the front of the cache, in
  place, with their accumulated weights (``verify_evict_kv_*``).
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CASE = dict(layout="dense", B=1, T=1, Hq=32, Hkv=8, D=128, dtype="bf16", lo=512, hi=512, page=16, draft="chain",
             softcap=0.0, window=0, slopes=False, start=False, gain=1.0, decay=1.0, accept=1, budget=0)


def _case(name=None, **kw):
    c = dict(_CASE)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # a short draft chain of a target with capped scores, one long conversation: latency of decoding
        _case("attend chain capped", op="attend", T=8, lo=32768, hi=32768, softcap=50.0, gain=4.0),
        # a 64-node token tree over a 128K prefix, capped scores: the largest single call
        _case("attend tree capped", op="attend", T=64, lo=131072, hi=131072, draft="tree", softcap=30.0, gain=3.0),
        # a serving batch on 16-row pages whose layer attends inside a sliding window; block-masked drafts
        _case("attend paged window", op="attend", layout="paged", B=64, T=16, lo=2048, hi=8192, draft="block",
              window=1024),
        # single-token decoding with a slope per head (no grouped heads), ragged batch
        _case("attend slopes one token", op="attend", B=8, T=1, Hkv=32, lo=4096, hi=16384, slopes=True),
        # packed documents on 64-row pages, 64-wide heads, odd lengths down to a few keys, every rule at once
        _case("attend documents d64", op="attend", layout="paged", B=16, T=5, D=64, lo=3, hi=4097, page=64,
              softcap=30.0, slopes=True, start=True, window=2048, gain=2.0),
        # the smallest configuration: fp32, one kv-head, an 8-node tree; launch latency
        _case("attend tiny", op="attend", T=8, Hq=4, Hkv=1, D=64, dtype="fp32", lo=512, hi=512, draft="tree",
              slopes=True, window=300),
        # the weights of the accepted part of the draft chain over one long conversation
        _case("weigh chain capped", op="weigh", T=8, lo=32768, hi=32768, softcap=50.0, gain=4.0, accept=5),
        # the weights of a serving batch: ragged lengths and acceptance, aged by a decay
        _case("weigh paged", op="weigh", layout="paged", B=64, T=16, lo=2048, hi=8192, decay=0.98),
        # 64 tokens of one chunk over a 128K prefix: as many rows as a call takes
        _case("weigh chunk", op="weigh", T=64, lo=131072, hi=131072, accept=64),
        # long conversations cut back to 8192 rows a kv-head
        _case("evict dense", op="evict", B=16, lo=16384, hi=32768, budget=8192),
        # a serving batch on 16-row pages cut back to the verify-set size
        _case("evict paged", op="evict", layout="paged", B=64, lo=2048, hi=8192, budget=2048),
        # the smallest configuration: fp32, one kv-head
        _case("evict tiny", op="evict", Hq=4, Hkv=1, D=64, dtype="fp32", lo=512, hi=512, budget=256),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["attend", "weigh", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    D = 64 if dtype == "fp32" else rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8] if Hkv < 8 else [1, 2, 4])
    T = log(1, 64)
    B = log(1, 64)
    # keys in all: at most 2^20 rows of all kv-heads (fp32: 2^17) and 2^26 scores
    rows = (1 << 17) if dtype == "fp32" else (1 << 20)
    most = max(64, min(131072, rows // (B * Hkv), (1 << 28) // (B * Hq * T)))
    hi = log(32, most)
    lo = max(1, hi - int(hi * rng.random())) if B > 1 else hi
    c = _case(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, lo=lo, hi=hi,
              layout=rng.choice(["dense", "paged"]), page=rng.choice([1, 4, 8, 16, 64, 256]))
    if op == "evict":
        c["T"] = 1
        c["budget"] = max(2, int(hi * rng.uniform(0.1, 0.9)))
        return c
    if rng.random() < 0.6:
        c["softcap"] = rng.choice([15.0, 30.0, 50.0])
        c["gain"] = rng.uniform(1.0, 5.0)
    if rng.random() < 0.4:
        c["window"] = log(8, 2 * hi)
    c["slopes"] = rng.random() < 0.4
    c["start"] = rng.random() < 0.4
    if op == "attend":
        c["draft"] = rng.choice(["chain", "tree", "block"])
    else:
        c["accept"] = rng.randint(1, T)
        c["decay"] = rng.choice([1.0, rng.uniform(0.5, 1.0)])
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread (hi alone for one)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _accepted(c):
    return _spread(1, c["T"], c["B"]) if c["B"] > 1 else [c["accept"]]


def _starts(c, lens):
    return [3 * n // 8 if c["start"] else 0 for n in lens]


def _lowest(c, lens):
    """Lowest slot any row of a sequence sees (the draft's first token is at offset 0)."""
    return [min(n, max(s, n - c["window"] + 1 if c["window"] else 0)) for n, s in zip(lens, _starts(c, lens))]


def _random_tree(T, g):
    """Parents of a random token tree: node i hangs off an earlier node or the prefix."""
    r = torch.rand(T, generator=g)
    return [-1 if i == 0 else int(r[i].item() * (i + 1)) - 1 for i in range(T)]


def _depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[c["dtype"]]
    B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]

    def normal(*shape):
        out = torch.empty(*shape, dtype=dt, device="cuda")
        return out.normal_(generator=gd)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32).cuda()

    order = torch.randperm(B, generator=g).tolist()
    lens = [_spread(c["lo"], c["hi"], B)[i] for i in order]
    cap = c["hi"] + T
    s = {"case": c, "seqlens": i32(lens), "lens": lens, "scale": 1.0 / math.sqrt(D)}
    if c["layout"] == "paged":
        need = [-(-(n + T) // c["page"]) for n in lens]
        used = torch.arange(max(need)) < torch.tensor(need)[:, None]
        table = torch.full(used.shape, -1, dtype=torch.int32)
        table[used] = torch.randperm(sum(need), generator=g).int()
        s["page_table"] = table.cuda()
        s["k"] = normal(sum(need), c["page"], Hkv, D)
        s["v"] = normal(sum(need), c["page"], Hkv, D)
        cap = max(need) * c["page"]
    else:
        s["k"] = normal(B, cap, Hkv, D)
        s["v"] = normal(B, cap, Hkv, D)
    s["cap"] = cap

    if c["op"] == "evict":
        # the keep set of every (sequence, kv-head): 4 first rows, the newest
        # eighth of the budget and the best of the others by accumulated weight
        weight = torch.rand(B, Hkv, cap, generator=gd, device="cuda")
        n_keep = torch.tensor([min(n, c["budget"]) for n in lens], device="cuda")
        L = s["seqlens"].long()[:, None, None]
        slot = torch.arange(cap, device="cuda")
        fixed = (slot < min(4, c["budget"])) | (slot >= L - c["budget"] // 8)
        key = torch.where(slot < L, weight + 2.0 * fixed, -1.0)
        best = key.topk(min(c["budget"], cap), dim=-1).indices
        j = torch.arange(best.shape[-1], device="cuda")
        best = torch.where(j < n_keep[:, None, None], best, cap).sort(dim=-1).values
        idx = torch.full((B, Hkv, c["budget"]), -1, dtype=torch.int32, device="cuda")
        idx[..., : best.shape[-1]] = torch.where(best < cap, best, -1).int()
        s["indices"] = idx
        s["n_indices"] = n_keep.int()[:, None].expand(B, Hkv).contiguous()
        s["weight"] = weight
        s["seqlens_out"] = torch.empty_like(s["seqlens"])
    else:
        s["q"] = normal(B, T, Hq, D).mul_(c["gain"])
        s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)).float() if c["slopes"] else None
        s["key_start"] = i32(_starts(c, lens)) if c["start"] else None
        if c["op"] == "attend":
            offset = [list(range(T)) for _ in range(B)]
            s["parent"] = s["mask"] = None
            if c["draft"] == "tree":
                trees = [_random_tree(T, g) for _ in range(B)]
                offset = [_depths(p) for p in trees]
                s["parent"] = i32(trees)
            elif c["draft"] == "block":  # bidirectional inside 4-token blocks, causal across them
                words = [[[sum(1 << (j % 32) for j in range(32 * w, min(T, 32 * w + 32)) if j // 4 <= i // 4)
                           for w in range((T + 31) // 32)] for i in range(T)] for _ in range(B)]
                m = torch.tensor(words, dtype=torch.int64)
                s["mask"] = (m - (m >= 1 << 31) * (1 << 32)).int().cuda()
            s["token_pos"] = i32([[n + o for o in row] for n, row in zip(lens, offset)])
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(B, Hq, T, dtype=torch.float32, device="cuda")
        else:
            acc = [_accepted(c)[i] for i in order]
            path = [sorted(torch.randperm(T, generator=g)[:a].tolist()) + [-1] * (T - a) for a in acc]
            s["path"], s["n_accept"] = i32(path), i32(acc)
            # totals as a few earlier steps leave them: a step gives a key about
            # (rows of its kv-head) / (keys) of weight
            s["weight"] = torch.rand(B, Hkv, cap, generator=gd, device="cuda").mul_(8.0 * Hq // Hkv * T / c["hi"])
            # log-sum-exp of the rows as the verification call returned them
            lse = torch.zeros(B, Hq, T, dtype=torch.float32, device="cuda")
            sc, seen, node = _accepted_scores(s)
            v = torch.logsumexp(sc.masked_fill(~seen, -math.inf), -1)  # [B][Hkv][group][T] by accepted rank
            s["lse"] = lse.scatter(2, node[:, None, :].expand(B, Hq, T), v.reshape(B, Hq, T)).contiguous()
    if own:
        import speculative_decoding_verification_masked_gb300 as va

        if c["op"] == "evict":
            s["scratch"] = va.EvictScratch(B, Hkv, c["budget"])
        else:
            s["mod"] = va.ScoreMod(softcap=c["softcap"], window=c["window"], slopes=s["slopes"],
                                   key_start=s["key_start"], token_pos=s.get("token_pos"))
            if c["op"] == "attend":
                s["workspace"] = va.Workspace.for_shape(va.make_shape(B, T, Hq, Hkv, D, 0 if dt is torch.bfloat16 else 2))
    return s


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------

def _rows_of(s, x):
    """The cache or pages x as logical slots [B][cap][Hkv][D]."""
    if s["case"]["layout"] == "dense":
        return x
    t = s["page_table"].long().clamp(min=0)
    return x[t].reshape(t.shape[0], -1, *x.shape[2:])


def _shape_scores(s, raw, dist):
    """Cap and distance bias on raw [B][Hkv][group][rows][slots]; dist [B][rows][slots]."""
    c = s["case"]
    if c["softcap"]:
        raw = c["softcap"] * torch.tanh(raw / c["softcap"])
    if s["slopes"] is not None:
        raw = raw - s["slopes"].view(1, c["Hkv"], -1, 1, 1) * dist.abs()[:, None, None].float()
    return raw


def _in_reach(s, dist, slot):
    """Window and document start: [B][rows][slots]."""
    ok = torch.ones_like(dist, dtype=torch.bool)
    if s["case"]["window"]:
        ok &= dist < s["case"]["window"]
    if s["key_start"] is not None:
        L = s["seqlens"].long()[:, None, None]
        ok &= (slot >= L) | (slot >= s["key_start"].long()[:, None, None])
    return ok


def _products(q, k):
    """q [B][T][Hq][D] on k [B][N][Hkv][D], in fp32: [B][Hkv][group][T][N]."""
    B, T, Hq, D = q.shape
    N, Hkv = k.shape[1:3]
    qg = q.float().reshape(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    return (qg @ k.float().permute(0, 2, 3, 1)).reshape(B, Hkv, Hq // Hkv, T, N)


def _accepted_scores(s):
    """Scores of the accepted rows over the committed slots, who sees what, and
    the draft node of every accepted row (any node past the accepted ones)."""
    c = s["case"]
    B, T, Hq, D = s["q"].shape
    rank = torch.arange(T, device="cuda")
    live = rank < s["n_accept"].long()[:, None]
    # nodes of the accepted rows first, then the others, so that `node` is a permutation
    used = torch.zeros(B, T + 1, device="cuda").scatter(1, torch.where(live, s["path"].long(), T), 1.0)[:, :T]
    rest = torch.argsort(used, dim=1, stable=True)
    node = torch.where(live, s["path"].long(), rest.gather(1, (rank - s["n_accept"].long()[:, None]).clamp(min=0)))
    q = s["q"].gather(1, node[:, :, None, None].expand(B, T, Hq, D))
    raw = _products(q, _rows_of(s, s["k"])) * s["scale"]
    slot = torch.arange(s["cap"], device="cuda")[None, None, :]
    dist = s["seqlens"].long()[:, None, None] + rank[None, :, None] - slot
    seen = (dist >= 0) & _in_reach(s, dist, slot)
    return _shape_scores(s, raw, dist), seen[:, None, None], node


def _attend(s):
    c = s["case"]
    B, T, Hq, D = s["q"].shape
    k, v = _rows_of(s, s["k"]), _rows_of(s, s["v"])
    raw = _products(s["q"], k) * s["scale"]
    slot = torch.arange(s["cap"], device="cuda")[None, None, :]
    L = s["seqlens"].long()[:, None, None]
    draft = (slot - L).clamp(0, T - 1)  # draft token of a slot behind the prefix
    pos = s["token_pos"].long()
    kpos = torch.where(slot < L, slot, pos[:, None, :].gather(2, draft))
    dist = pos[:, :, None] - kpos
    eye = torch.eye(T, dtype=torch.float64, device="cuda")
    if s["parent"] is not None:  # ancestors: powers of (I + parent matrix)
        up = (s["parent"].long()[:, :, None] == torch.arange(T, device="cuda")).double()
        among = torch.linalg.matrix_power(eye + up, T) > 0
    elif s["mask"] is not None:
        j = torch.arange(T, device="cuda")
        among = ((s["mask"].long()[:, :, j // 32] >> (j % 32)) & 1) > 0
    else:
        among = torch.ones(B, T, T, dtype=torch.bool, device="cuda").tril()
    seen = (slot < L) | ((slot < L + T) & among.gather(2, draft.expand(B, T, -1)))
    seen = (seen & _in_reach(s, dist, slot))[:, None, None]
    sc = _shape_scores(s, raw, dist).masked_fill(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m.masked_fill(m == -math.inf, 0.0))
    l = p.sum(-1, keepdim=True)
    o = (p.reshape(B, c["Hkv"], -1, s["cap"]) @ v.float().transpose(1, 2)).reshape(*p.shape[:-1], D)
    o = torch.where(l > 0, o / l, 0.0)  # [B][Hkv][group][T][D]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D))
    s["lse"].copy_((m + torch.log(l)).reshape(B, Hq, T))
    return s["out"], s["lse"]


def _weigh(s):
    c = s["case"]
    B, T, Hq, D = s["q"].shape
    sc, seen, node = _accepted_scores(s)
    live = torch.arange(T, device="cuda") < s["n_accept"].long()[:, None]
    lse = s["lse"].gather(2, node[:, None, :].expand(B, Hq, T)).reshape(B, c["Hkv"], -1, T, 1)
    p = torch.where(seen & live[:, None, None, :, None], torch.exp(sc - lse), 0.0).sum((2, 3))
    slot = torch.arange(s["cap"], device="cuda")
    L = s["seqlens"].long()[:, None, None]
    end = L + s["n_accept"].long()[:, None, None]
    w = torch.where(slot < L, c["decay"] * s["weight"] + p, torch.where(slot < end, p, s["weight"]))
    s["weight"].copy_(w)
    return s["weight"]


def _evict(s):
    n = s["n_indices"].long()
    B, Hkv, m = s["indices"].shape
    src = s["indices"].long()
    j = torch.arange(m, device="cuda")
    kept = j < n[:, :, None]
    b = torch.arange(B, device="cuda")[:, None, None].expand(B, Hkv, m)[kept]
    h = torch.arange(Hkv, device="cuda")[None, :, None].expand(B, Hkv, m)[kept]
    to, at = j.expand(B, Hkv, m)[kept], src[kept]
    s["weight"][b, h, to] = s["weight"][b, h, at]
    if s["case"]["layout"] == "paged":
        t, ps = s["page_table"].long(), s["case"]["page"]
        for x in (s["k"], s["v"]):
            x[t[b, to // ps], to % ps, h] = x[t[b, at // ps], at % ps, h]
    else:
        for x in (s["k"], s["v"]):
            x[b, to, h] = x[b, at, h]
    s["seqlens_out"].copy_(n[:, 0])
    return s["k"], s["v"], s["weight"], s["seqlens_out"]


def _calls(s):
    import speculative_decoding_verification_masked_gb300 as va

    c = s["case"]
    if c["op"] == "attend":
        kw = dict(tree_parent=s["parent"], tree_mask=s["mask"], out=s["out"], lse=s["lse"], workspace=s["workspace"],
                  scale=s["scale"])
        if c["layout"] == "paged":
            return va.verify_attn_paged_mod(s["q"], s["k"], s["v"], s["page_table"], s["seqlens"], s["mod"], **kw)
        return va.verify_attn_dense_mod(s["q"], s["k"], s["v"], s["seqlens"], s["mod"], **kw)
    if c["op"] == "weigh":
        kw = dict(mod=s["mod"], path=s["path"], n_accept=s["n_accept"], decay=c["decay"], scale=s["scale"])
        if c["layout"] == "paged":
            return va.verify_accumulate_weight_paged(s["q"], s["k"], s["page_table"], s["seqlens"], s["lse"],
                                                     s["weight"], **kw)
        return va.verify_accumulate_weight_dense(s["q"], s["k"], s["seqlens"], s["lse"], s["weight"], **kw)
    kw = dict(weight=s["weight"], seqlens_out=s["seqlens_out"], scratch=s["scratch"])
    if c["layout"] == "paged":
        va.verify_evict_kv_paged(s["k"], s["v"], s["page_table"], s["seqlens"], s["indices"], s["n_indices"], **kw)
    else:
        va.verify_evict_kv_dense(s["k"], s["v"], s["seqlens"], s["indices"], s["n_indices"], **kw)
    return s["k"], s["v"], s["weight"], s["seqlens_out"]


def run(state):
    if own:
        return _calls(state)
    return {"attend": _attend, "weigh": _weigh, "evict": _evict}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    lens = _spread(c["lo"], c["hi"], c["B"])
    row = c["D"] * es
    if c["op"] == "evict":
        moved = sum(min(n, c["budget"]) for n in lens) * c["Hkv"]
        return {"bytes": moved * (4 * row + 4 + 8), "flops": 0}
    keys = sum(n - a for n, a in zip(lens, _lowest(c, lens)))
    if c["op"] == "attend":
        keys += c["B"] * c["T"]
        qo = c["B"] * c["T"] * c["Hq"]
        return {"bytes": keys * c["Hkv"] * 2 * row + qo * (2 * row + 4), "flops": 4 * c["Hq"] * c["T"] * keys * c["D"]}
    acc = _accepted(c)
    total = sum(lens) + sum(acc)  # every total is read and written where it is aged
    new = sum(acc)
    touched = total if c["decay"] != 1.0 else keys + new
    flops = sum(2 * c["Hq"] * a * (n - lo + a) * c["D"] for n, lo, a in zip(lens, _lowest(c, lens), acc))
    return {"bytes": (keys + new) * c["Hkv"] * row + new * c["Hq"] * (row + 4) + touched * c["Hkv"] * 8, "flops": flops}


def _head_rows(s, x, b, h, n):
    """Rows of logical slots 0 .. n-1 of kv-head h of sequence b, in 64 bits."""
    if s["case"]["layout"] == "dense":
        return x[b, :n, h].double()
    ps = s["case"]["page"]
    at = torch.arange(n, device="cuda")
    return x[s["page_table"][b].long()[at // ps], at % ps, h].double()


def exact(case, seed):
    """The operators' definitions, one (sequence, kv-head) at a time, in 64 bits."""
    s = prepare(case, seed)
    c = s["case"]
    B, T, Hkv = c["B"], c["T"], c["Hkv"]
    G = c["Hq"] // Hkv
    if c["op"] == "evict":
        new = {x: s[x].double() for x in ("k", "v", "weight")}
        for b in range(B):
            for h in range(Hkv):
                n = int(s["n_indices"][b, h])
                src = s["indices"][b, h, :n].long()
                to = torch.arange(n, device="cuda")
                new["weight"][b, h, :n] = s["weight"][b, h][src].double()
                for x in ("k", "v"):
                    rows = _head_rows(s, s[x], b, h, s["lens"][b])[src]
                    if c["layout"] == "dense":
                        new[x][b, :n, h] = rows
                    else:
                        t = s["page_table"][b].long()
                        new[x][t[to // c["page"]], to % c["page"], h] = rows
        return new["k"], new["v"], new["weight"], s["n_indices"][:, 0].clone()

    def shaped(rows, keys, h, qpos, kpos):
        z = torch.einsum("tgd,nd->gtn", rows, keys) / math.sqrt(c["D"])
        if c["softcap"]:
            u = torch.exp(-2 * (z / c["softcap"]).abs())
            z = c["softcap"] * torch.sign(z) * (1 - u) / (1 + u)
        away = (qpos[:, None] - kpos[None, :]).double()
        if c["slopes"]:
            z = z - s["slopes"][h * G:(h + 1) * G].double()[:, None, None] * away.abs()
        near = away < c["window"] if c["window"] else torch.ones_like(away, dtype=torch.bool)
        return z, near

    if c["op"] == "attend":
        out = torch.zeros(B, T, c["Hq"], c["D"], dtype=torch.float64, device="cuda")
        lse = torch.empty(B, c["Hq"], T, dtype=torch.float64, device="cuda")
        for b in range(B):
            L = s["lens"][b]
            sees = torch.zeros(T, T, dtype=torch.bool)
            parent = s["parent"][b].tolist() if s["parent"] is not None else None
            for i in range(T):
                if parent is not None:
                    j = i
                    while j >= 0:
                        sees[i, j] = True
                        j = parent[j]
                elif s["mask"] is not None:
                    sees[i] = torch.tensor([j // 4 <= i // 4 for j in range(T)])
                else:
                    sees[i, : i + 1] = True
            pos = s["token_pos"][b].long()
            kpos = torch.cat([torch.arange(L, device="cuda"), pos])
            old = torch.arange(L, device="cuda") >= (int(s["key_start"][b]) if c["start"] else 0)
            vis = torch.cat([old[None].expand(T, L), sees.cuda()], 1)
            for h in range(Hkv):
                keys, vals = (_head_rows(s, s[x], b, h, L + T) for x in ("k", "v"))
                z, near = shaped(s["q"][b, :, h * G:(h + 1) * G].double(), keys, h, pos, kpos)
                z = torch.where(vis & near, z, -math.inf)
                t = torch.logsumexp(z, -1)
                lse[b, h * G:(h + 1) * G] = t
                w = torch.exp(z - t.clamp(min=-1e300)[..., None])
                out[b, :, h * G:(h + 1) * G] = torch.einsum("gtn,nd->tgd", w, vals)
        return out, lse
    weight = s["weight"].double()
    for b in range(B):
        L, a = s["lens"][b], int(s["n_accept"][b])
        if a == 0:
            weight[b, :, :L] *= c["decay"]
            continue
        node = s["path"][b, :a].long()
        qpos, kpos = L + torch.arange(a, device="cuda"), torch.arange(L + a, device="cuda")
        low = int(s["key_start"][b]) if c["start"] else 0
        vis = (kpos[None, :] <= qpos[:, None]) & ((kpos >= low) | (kpos >= L))[None, :]
        for h in range(Hkv):
            z, near = shaped(s["q"][b][node][:, h * G:(h + 1) * G].double(), _head_rows(s, s["k"], b, h, L + a), h,
                             qpos, kpos)
            p = torch.exp(z - s["lse"][b, h * G:(h + 1) * G][:, node].double()[..., None])
            p = torch.where(vis & near, p, 0.0).sum((0, 1))
            weight[b, h, :L] = c["decay"] * weight[b, h, :L] + p[:L]
            weight[b, h, L:L + a] = p[L:]
    return weight
