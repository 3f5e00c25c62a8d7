"""Workloads of the per-head norm with rotation and of the caches held in 8 or 4
bits, in plain torch and through the library's entry points.

* ``norm``   -- RMS norm of every query and key head and the rotary embedding, in
  one pass over a projection's output (``verify_norm_rope``);
* ``write``  -- rows of K and V quantised into a cache at the slots after each
  prefix (``verify_quantize_kv_*``), and those slots read back;
* ``read``   -- a range of slots of such a cache read back (``verify_dequantize_kv_*``);
* ``attend`` -- verification attention over such a cache (``verify_attn_*_quant``).

A quantised row (one token, one kv-head) is a run of bytes: "e4m3" has D codes,
the row scale as fp32 and zeros up to 16 bytes more than the codes; "e2m1" has
D/2 bytes of codes (element 2j in the low half of byte j), D/16 group scales in
e4m3, the row scale as fp32 and zeros up to the next multiple of 16 (D 128: 80,
D 64: 48 bytes).  Row scales are powers of two.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_FORMATS = ["e4m3", "e2m1"]
_EPS, _BASE = 1e-6, 500000.0
_CASE = dict(B=1, T=1, Hq=32, Hkv=8, D=128, dtype="bf16", lo=512, hi=512, layout="dense", page=16, fmt="e2m1",
             draft="chain", fused=True, far=False, ragged=False)


def _case(name=None, **kw):
    c = dict(_CASE)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # the smallest configuration: fp32, one kv-head, 8 drafted tokens; launch latency
        _case("norm tiny", op="norm", T=8, Hq=4, Hkv=1, D=64, dtype="fp32", far=True),
        # a verification step of a serving batch, q and k inside the fused projection
        _case("norm step", op="norm", B=64, T=16, lo=2048, hi=8192),
        # one long prompt
        _case("norm prompt", op="norm", T=16384, lo=0, hi=0),
        # a chunk of four prompts of different lengths into 4-bit rows
        _case("write chunk e2m1", op="write", B=4, T=4096, lo=0, hi=12288, ragged=True),
        # the drafted rows of a serving batch into 8-bit pages
        _case("write step e4m3 paged", op="write", B=64, T=16, lo=2048, hi=8192, layout="paged", fmt="e4m3"),
        # two long prefixes read back for a pass that wants 16-bit keys
        _case("read prefix e2m1", op="read", B=2, T=32768, lo=32768, hi=32768),
        # ragged 64-wide heads out of 8-bit pages, to fp32
        _case("read ragged e4m3 d64", op="read", B=16, T=1001, D=64, dtype="fp32", lo=3, hi=4097, layout="paged", page=64,
              fmt="e4m3", ragged=True),
        # a short draft chain over one long conversation held in 4 bits: latency of decoding
        _case("attend chain e2m1", op="attend", T=8, lo=32768, hi=32768),
        # a 64-node token tree over a 128K prefix in 4 bits: the largest single call
        _case("attend tree e2m1", op="attend", T=64, lo=131072, hi=131072, draft="tree"),
        # a serving batch in 8-bit pages, block-masked drafts
        _case("attend paged e4m3", op="attend", B=64, T=16, lo=2048, hi=8192, layout="paged", fmt="e4m3", draft="block"),
        # single-token decoding of a ragged batch in 4-bit pages
        _case("attend one token e2m1", op="attend", B=64, T=1, lo=1024, hi=16384, layout="paged", page=64),
        # short sequences, one of them empty, 64-wide heads, odd lengths, 4-row pages
        _case("attend short e4m3 d64", op="attend", B=5, T=5, Hq=16, Hkv=4, D=64, lo=0, hi=701, layout="paged", page=4,
              fmt="e4m3", draft="tree"),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["norm", "write", "read", "attend", "attend"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8] if Hkv < 8 else [1, 2, 4])
    c = _case(op=op, Hkv=Hkv, Hq=Hq, D=rng.choice([64, 128, 128]), layout=rng.choice(["dense", "paged"]),
              page=rng.choice([1, 4, 8, 16, 64, 256]), fmt=rng.choice(_FORMATS), fused=rng.random() < 0.7,
              far=rng.random() < 0.3, ragged=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "norm":
        c["D"] = rng.choice([64, 96, 128, 128, 256])
        c["B"] = log(1, 64)
        # at most 2^26 elements of q and k
        c["T"] = log(1, max(1, min(16384, (1 << 26) // (c["B"] * (Hq + Hkv) * c["D"]))))
        c["lo"] = c["hi"] = log(1, 131072)
    elif op in ("write", "read"):
        c["B"] = log(1, 64)
        c["T"] = log(1, max(1, min(32768, (1 << 25) // (c["B"] * Hkv * c["D"]))))
        c["hi"] = log(1, max(1, min(16384, (1 << 27) // (c["B"] * Hkv * c["D"]))))
        c["lo"] = c["hi"] - int(c["hi"] * rng.random()) if c["B"] > 1 else c["hi"]
    else:
        c["dtype"] = "bf16"
        c["T"], c["B"] = log(1, 64), log(1, 64)
        # at most 2^20 rows of all kv-heads and 2^28 scores
        most = max(64, min(131072, (1 << 20) // (c["B"] * Hkv), (1 << 28) // (c["B"] * Hq * c["T"])))
        c["hi"] = log(32, most)
        c["lo"] = max(0, c["hi"] - int(c["hi"] * rng.random())) if c["B"] > 1 else c["hi"]
        c["draft"] = rng.choice(["chain", "tree", "block"])
    return c


# ---------------------------------------------------------------------------
# rows in 8 or 4 bits
# ---------------------------------------------------------------------------

def _row_bytes(fmt, D):
    return D + 16 if fmt == "e4m3" else -(-(D // 2 + D // 16 + 4) // 16) * 16


def _used_bytes(fmt, D):
    return D + 4 if fmt == "e4m3" else D // 2 + D // 16 + 4


def _scale_at(fmt, D):
    return D if fmt == "e4m3" else D // 2 + D // 16


def _pow2(e):
    """2^e in fp32, from the bits (a power function may be off by a unit)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _round_e4m3(y):
    """Nearest e4m3 value (ties to even) of y with |y| <= 448, exactly."""
    ex = torch.frexp(y).exponent.clamp(min=-5)
    return torch.round(y * _pow2(4 - ex)) * _pow2(ex - 4)


def _e4m3_bits(v):
    """The byte of a value that _round_e4m3 returned."""
    a = v.abs()
    f = torch.frexp(a)
    normal = (f.exponent + 6) * 8 + ((f.mantissa * 2 - 1) * 8).int()
    return torch.where(a < 2.0 ** -6, (a * 512).int(), normal) + 128 * torch.signbit(v).int()


def _quantize(x, fmt):
    """Codes of fp32 rows x [..., D] (e4m3: the bytes; e2m1: 4-bit codes), the group
    scales, the row scales, and the values that they stand for."""
    amax = x.abs().amax(-1, keepdim=True)
    f = torch.frexp(amax)
    top, mant = (8, 0.875) if fmt == "e4m3" else (11, 0.65625)  # 448 and 6 * 448
    e = f.exponent - 1 - top + (f.mantissa > mant).int()
    e = torch.where(amax > 0, e, -126).clamp(min=-126)
    s = _pow2(e)
    y = x / s
    if fmt == "e4m3":
        v = _round_e4m3(y)
        return _e4m3_bits(v), None, s, v * s
    y = y.unflatten(-1, (-1, 16))
    g = _round_e4m3(y.abs().amax(-1, keepdim=True).double() / 6).float()
    a = y.abs()
    i = ((a > 0.25 * g).int() + (a >= 0.75 * g) + (a > 1.25 * g) + (a >= 1.75 * g) + (a > 2.5 * g) + (a >= 3.5 * g)
         + (a > 5 * g))
    i = torch.where(g > 0, i, 0)
    v = (torch.where(i < 4, 0.5 * i, torch.where(i < 6, i - 2.0, 2.0 * i - 8.0)) * g).copysign(y) * s[..., None]
    return (i + 8 * torch.signbit(y).int()).flatten(-2), _e4m3_bits(g[..., 0]), s, v.flatten(-2)


def _pack(x, fmt):
    """Quantised rows [..., row bytes] of x [..., D]."""
    D = x.shape[-1]
    code, group, s, _ = _quantize(x.float(), fmt)
    rows = torch.zeros(*x.shape[:-1], _row_bytes(fmt, D), dtype=torch.uint8, device=x.device)
    if fmt == "e4m3":
        rows[..., :D] = code.to(torch.uint8)
    else:
        rows[..., :D // 2] = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
        rows[..., D // 2:D // 2 + D // 16] = group.to(torch.uint8)
    at = _scale_at(fmt, D)
    rows[..., at:at + 4] = s.contiguous().view(torch.uint8)
    return rows


def _values_e4m3():
    v = [(c & 7) / 512 if c & 0x78 == 0 else (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10) for c in range(128)]
    return v + [-a for a in v]


def _unpack(rows, fmt, D):
    """The fp32 values of quantised rows."""
    table = torch.tensor(_values_e4m3(), device=rows.device)
    at = _scale_at(fmt, D)
    s = rows[..., at:at + 4].contiguous().view(torch.float32)
    if fmt == "e4m3":
        return table.index_select(0, rows[..., :D].int().flatten()).view(*rows.shape[:-1], D) * s
    v4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    v4 = v4 + [-a for a in v4]
    pairs = torch.tensor([[v4[c & 15], v4[c >> 4]] for c in range(256)], device=rows.device)
    v = pairs.index_select(0, rows[..., :D // 2].int().flatten()).view(*rows.shape[:-1], D // 16, 16)
    g = table.index_select(0, rows[..., D // 2:at].int().flatten()).view(*rows.shape[:-1], D // 16, 1)
    return (v * g * s[..., None]).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread (hi alone for one)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _counts(c):
    """Rows of every sequence that are written or read."""
    return _spread(max(1, c["T"] // 3), c["T"], c["B"]) if c["ragged"] else [c["T"]] * c["B"]


def _random_tree(T, g):
    """Parents of a random token tree: node i hangs off an earlier node or the prefix."""
    r = torch.rand(T, generator=g)
    return [-1 if i == 0 else int(r[i].item() * (i + 1)) - 1 for i in range(T)]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[c["dtype"]]
    B, T, Hq, Hkv, D, fmt = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["fmt"]

    def normal(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda").normal_(generator=gd)

    def rows(*shape):
        """K or V as projections give them: tokens of different size, a few loud channels."""
        loud = 1 + 3 * (torch.rand(D, generator=gd, device="cuda") < 0.05)
        return (normal(*shape, D, dtype=torch.float32) * loud
                * torch.exp(0.3 * normal(*shape, 1, dtype=torch.float32))).to(dt)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32).cuda()

    order = torch.randperm(B, generator=g).tolist()
    lens = [_spread(c["lo"], c["hi"], B)[i] for i in order]
    count = [_counts(c)[i] for i in order]
    s = {"case": c, "lens": lens, "count": count, "seqlens": i32(lens), "n_tokens": i32(count) if c["ragged"] else None}

    if c["op"] == "norm":
        s["wq"], s["wk"] = (1 + 0.2 * normal(D, dtype=torch.float32)).to(dt), (1 + 0.2 * normal(D, dtype=torch.float32)).to(dt)
        if c["fused"]:  # q, k and v side by side as one projection leaves them
            x = normal(B, T, Hq + 2 * Hkv, D)
            s["q"], s["k"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = normal(B, T, Hq, D), normal(B, T, Hkv, D)
        if c["far"]:  # ids that are not consecutive, up to a million
            s["positions"] = torch.randint(0, 1 << 20, (B, T), generator=gd, device="cuda", dtype=torch.int32)
        else:
            s["positions"] = s["seqlens"][:, None] + torch.arange(T, dtype=torch.int32, device="cuda")
        s["q_out"] = torch.empty(B, T, Hq, D, dtype=dt, device="cuda")
        s["k_out"] = torch.empty(B, T, Hkv, D, dtype=dt, device="cuda")
        return s

    # slots of every sequence, and the shape of a cache or pool of rows
    slots = [max(n, r) if c["op"] == "read" else n + T for n, r in zip(lens, count)]
    if c["layout"] == "paged":
        need = [-(-n // c["page"]) for n in slots]
        used = torch.arange(max(need)) < torch.tensor(need)[:, None]
        table = torch.full(used.shape, -1, dtype=torch.int32)
        table[used] = torch.randperm(sum(need), generator=g).int()
        s["page_table"] = table.cuda()
        shape = (sum(need), c["page"], Hkv)
    else:
        shape = (B, max(slots), Hkv)
    if c["op"] == "write":
        if c["fused"]:
            x = rows(B, T, Hq + 2 * Hkv)
            s["k"], s["v"] = x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        else:
            s["k"], s["v"] = rows(B, T, Hkv), rows(B, T, Hkv)
        for x in ("k_cache", "v_cache"):
            s[x] = torch.zeros(*shape, _row_bytes(fmt, D), dtype=torch.uint8, device="cuda")
        s["start"] = s["seqlens"]
    else:
        for x in ("k_cache", "v_cache"):
            cache = torch.empty(*shape, _row_bytes(fmt, D), dtype=torch.uint8, device="cuda")
            flat = cache.view(-1, Hkv, cache.shape[-1])
            for i in range(0, flat.shape[0], 1 << 16):
                part = flat[i:i + (1 << 16)]
                part.copy_(_pack(rows(part.shape[0], Hkv), fmt))
            s[x] = cache
        if c["op"] == "read":  # the last rows of every sequence
            s["start"] = i32([n - r for n, r in zip(slots, count)])
    if c["op"] in ("write", "read"):
        s["k_out"] = torch.zeros(B, T, Hkv, D, dtype=dt, device="cuda")
        s["v_out"] = torch.zeros(B, T, Hkv, D, dtype=dt, device="cuda")
        return s

    s["q"] = normal(B, T, Hq, D)
    s["scale"] = 1.0 / math.sqrt(D)
    s["parent"] = s["mask"] = None
    if c["draft"] == "tree":
        s["parent"] = i32([_random_tree(T, g) for _ in range(B)])
    elif c["draft"] == "block":  # bidirectional inside 4-token blocks, causal across them
        words = [[[sum(1 << (j % 32) for j in range(32 * w, min(T, 32 * w + 32)) if j // 4 <= i // 4)
                   for w in range((T + 31) // 32)] for i in range(T)] for _ in range(B)]
        m = torch.tensor(words, dtype=torch.int64)
        s["mask"] = (m - (m >= 1 << 31) * (1 << 32)).int().cuda()
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(B, Hq, T, dtype=torch.float32, device="cuda")
    if own:
        import speculative_decoding_verification_masked_gb300 as va

        s["workspace"] = va.Workspace.for_shape(va.make_shape(B, T, Hq, Hkv, D, 0))
    return s


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------

def _rows_of(s, x):
    """The cache or pages x as logical slots [B][slots][Hkv][row bytes]."""
    if s["case"]["layout"] == "dense":
        return x
    t = s["page_table"].long().clamp(min=0)
    return x[t].reshape(t.shape[0], -1, *x.shape[2:])


def _norm(s):
    D = s["case"]["D"]
    i = torch.arange(D // 2, device="cuda", dtype=torch.float64)
    angle = s["positions"].double()[:, :, None, None] * _BASE ** (-2 * i / D)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    for x, w, out in ((s["q"], s["wq"], s["q_out"]), (s["k"], s["wk"], s["k_out"])):
        y = x.float()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + _EPS) * w.float()
        a, b = y[..., :D // 2], y[..., D // 2:]
        out.copy_(torch.cat([a * cos - b * sin, b * cos + a * sin], -1))
    return s["q_out"], s["k_out"]


def _live(s):
    """The rows [B][T] of every sequence that count."""
    return torch.arange(s["case"]["T"], device="cuda") < torch.tensor(s["count"], device="cuda")[:, None]


def _write(s):
    live = _live(s)[:, :, None, None]
    for x, out in ((s["k"], s["k_out"]), (s["v"], s["v_out"])):
        v = _quantize(x.float(), s["case"]["fmt"])[3]
        out.copy_(torch.where(live, v, out.float()))
    return s["k_out"], s["v_out"]


def _read(s):
    c = s["case"]
    t = torch.arange(c["T"], device="cuda")
    live = _live(s)[:, :, None, None]
    slot = torch.where(live[:, :, 0, 0], s["start"].long()[:, None] + t, 0)
    b = torch.arange(c["B"], device="cuda")[:, None]
    for x, out in ((s["k_cache"], s["k_out"]), (s["v_cache"], s["v_out"])):
        if c["layout"] == "paged":
            rows = x[s["page_table"].long()[b, slot // c["page"]].clamp(min=0), slot % c["page"]]
        else:
            rows = x[b, slot]
        out.copy_(torch.where(live, _unpack(rows, c["fmt"], c["D"]), out.float()))
    return s["k_out"], s["v_out"]


def _attend(s):
    c = s["case"]
    B, T, Hq, D = s["q"].shape
    Hkv = c["Hkv"]
    k, v = (_unpack(_rows_of(s, s[x]), c["fmt"], D) for x in ("k_cache", "v_cache"))
    N = k.shape[1]
    q = s["q"].float().reshape(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    sc = ((q @ k.permute(0, 2, 3, 1)) * s["scale"]).view(B, Hkv, Hq // Hkv, T, N)
    slot = torch.arange(N, device="cuda")[None, None, :]
    L = s["seqlens"].long()[:, None, None]
    draft = (slot - L).clamp(0, T - 1)  # draft token of a slot behind the prefix
    if s["parent"] is not None:  # ancestors: powers of (I + parent matrix)
        up = (s["parent"].long()[:, :, None] == torch.arange(T, device="cuda")).double()
        among = torch.linalg.matrix_power(torch.eye(T, dtype=torch.float64, device="cuda") + up, T) > 0
    elif s["mask"] is not None:
        j = torch.arange(T, device="cuda")
        among = ((s["mask"].long()[:, :, j // 32] >> (j % 32)) & 1) > 0
    else:
        among = torch.ones(B, T, T, dtype=torch.bool, device="cuda").tril()
    seen = (slot < L) | ((slot < L + T) & among.gather(2, draft.expand(B, T, -1)))
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, -1, N) @ v.transpose(1, 2)).reshape(*p.shape[:-1], D) / l  # [B][Hkv][group][T][D]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D))
    s["lse"].copy_((m + torch.log(l)).reshape(B, Hq, T))
    return s["out"], s["lse"]


def _calls(s):
    import speculative_decoding_verification_masked_gb300 as va

    c = s["case"]
    if c["op"] == "norm":
        return va.verify_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], eps=_EPS, rope_base=_BASE,
                                   q_out=s["q_out"], k_out=s["k_out"])
    paged, fmt = c["layout"] == "paged", c["fmt"]
    cache = (s["k_cache"], s["v_cache"], s["page_table"]) if paged else (s["k_cache"], s["v_cache"])
    if c["op"] == "attend":
        f = va.verify_attn_paged_quant if paged else va.verify_attn_dense_quant
        return f(s["q"], *cache, s["seqlens"], fmt, tree_parent=s["parent"], tree_mask=s["mask"], out=s["out"],
                 lse=s["lse"], workspace=s["workspace"], scale=s["scale"])
    if c["op"] == "write":
        f = va.verify_quantize_kv_paged if paged else va.verify_quantize_kv_dense
        f(s["k"], s["v"], *cache, s["seqlens"], fmt, n_tokens=s["n_tokens"])
    f = va.verify_dequantize_kv_paged if paged else va.verify_dequantize_kv_dense
    return f(*cache, s["start"], fmt, n_tokens=s["n_tokens"], k_out=s["k_out"], v_out=s["v_out"])


def run(state):
    if own:
        return _calls(state)
    return {"norm": _norm, "write": _write, "read": _read, "attend": _attend}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    row, used = c["D"] * es, _used_bytes(c["fmt"], c["D"])
    if c["op"] == "norm":
        n = c["B"] * c["T"] * (c["Hq"] + c["Hkv"])
        return {"bytes": 2 * n * row + 2 * row + 4 * c["B"] * c["T"], "flops": 0}
    if c["op"] == "write":  # the rows in, their codes out, and read back
        return {"bytes": 2 * sum(_counts(c)) * c["Hkv"] * (2 * row + used), "flops": 0}
    if c["op"] == "read":
        return {"bytes": 2 * sum(_counts(c)) * c["Hkv"] * (row + used), "flops": 0}
    keys = sum(_spread(c["lo"], c["hi"], c["B"])) + c["B"] * c["T"]
    qo = c["B"] * c["T"] * c["Hq"]
    return {"bytes": 2 * keys * c["Hkv"] * used + qo * (2 * row + 4), "flops": 4 * c["Hq"] * c["T"] * keys * c["D"]}


def _nearest(y, values):
    """Nearest of the ascending `values` to each of y, ties to the even index."""
    v = torch.tensor(values, dtype=torch.float64, device=y.device)
    hi = torch.searchsorted(v, y).clamp(1, len(values) - 1)
    lo = hi - 1
    below, above = y - v[lo], v[hi] - y
    return v[torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)]


def _two(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _stored(x, fmt):
    """What rows x [..., D] (64 bits) are stored as."""
    out = torch.empty_like(x)
    e4m3 = _values_e4m3()[:127]
    flat, res = x.reshape(-1, x.shape[-1]), out.view(-1, x.shape[-1])
    for i in range(0, flat.shape[0], 1 << 16):
        r = flat[i:i + (1 << 16)]
        amax = r.abs().amax(-1, keepdim=True)
        most = 448.0 if fmt == "e4m3" else 6 * 448.0
        e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 1.0) / most))
        e = torch.where(amax > most * _two(e), e + 1, torch.where(amax <= most * _two(e - 1), e - 1, e))
        s = _two(torch.where(amax > 0, e, -126.0).clamp(min=-126.0))
        y = r.abs() / s
        if fmt == "e4m3":
            v = _nearest(y, e4m3)
        else:
            y = y.unflatten(-1, (-1, 16))
            g = _nearest(y.amax(-1, keepdim=True) / 6, e4m3)
            q = y / torch.where(g > 0, g, 1.0)
            v = (_nearest(q, [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]) * g).flatten(-2)
        res[i:i + (1 << 16)] = torch.sign(r) * v * s
    return out


def _decoded(rows, fmt, D):
    """Quantised rows in 64 bits, field by field."""
    def e4m3(b):
        b = b.long()
        ex, m = (b >> 3) & 15, (b & 7).double()
        v = torch.where(ex == 0, m / 512, (1 + m / 8) * _two(ex - 7))
        return torch.where(b >= 128, -v, v)

    at = _scale_at(fmt, D)
    word = rows[..., at:at + 4].long()
    s = _two(((word[..., 3:] & 127) * 2 + (word[..., 2:3] >> 7)) - 127)  # a power of two
    if fmt == "e4m3":
        return e4m3(rows[..., :D]) * s
    b = rows[..., :D // 2].long()
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    ex, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(ex == 0, m / 2, (1 + m / 2) * _two(ex - 1))
    return torch.where(c >= 8, -v, v) * e4m3(rows[..., D // 2:at]).repeat_interleave(16, -1) * s


def _slots(s, x, b, at):
    """Rows of logical slots `at` of sequence b: [n][Hkv][row bytes]."""
    if s["case"]["layout"] == "dense":
        return x[b, at]
    ps = s["case"]["page"]
    return x[s["page_table"][b].long()[at // ps], at % ps]


def exact(case, seed):
    """The operators' definitions in 64 bits, one sequence (and kv-head) at a time."""
    s = prepare(case, seed)
    c = s["case"]
    B, T, Hkv, D = c["B"], c["T"], c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    if c["op"] == "norm":
        half = torch.arange(D, device="cuda") % (D // 2)
        freq = torch.exp(-2 * half.double() / D * math.log(_BASE))
        res = []
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            for b in range(B):
                for t in range(0, T, 2048):
                    y = x[b, t:t + 2048].double()
                    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + _EPS) * w.double()
                    a = s["positions"][b, t:t + 2048].double()[:, None, None] * freq
                    turned = torch.cat([-y[..., D // 2:], y[..., :D // 2]], -1)
                    out[b, t:t + 2048] = y * torch.cos(a) + turned * torch.sin(a)
            res.append(out)
        return tuple(res)
    if c["op"] in ("write", "read"):
        res = []
        for x in ("k", "v"):
            out = torch.zeros(B, T, Hkv, D, dtype=torch.float64, device="cuda")
            for b, n in enumerate(s["count"]):
                if c["op"] == "write":
                    out[b, :n] = _stored(s[x][b, :n].double(), c["fmt"])
                else:
                    at = int(s["start"][b]) + torch.arange(n, device="cuda")
                    out[b, :n] = _decoded(_slots(s, s[x + "_cache"], b, at), c["fmt"], D)
            res.append(out)
        return tuple(res)
    out = torch.zeros(B, T, c["Hq"], D, dtype=torch.float64, device="cuda")
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
        vis = torch.cat([torch.ones(T, L, dtype=torch.bool), sees], 1).cuda()
        at = torch.arange(L + T, device="cuda")
        rows = {x: _slots(s, s[x], b, at) for x in ("k_cache", "v_cache")}
        for h in range(Hkv):
            keys, vals = (_decoded(rows[x][:, h], c["fmt"], D) for x in ("k_cache", "v_cache"))
            z = torch.einsum("tgd,nd->gtn", s["q"][b, :, h * G:(h + 1) * G].double(), keys) / math.sqrt(D)
            z = torch.where(vis, z, -math.inf)
            t = torch.logsumexp(z, -1)
            lse[b, h * G:(h + 1) * G] = t
            out[b, :, h * G:(h + 1) * G] = torch.einsum("gtn,nd->tgd", torch.exp(z - t[..., None]), vals)
    return out, lse
