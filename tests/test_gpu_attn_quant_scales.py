"""Attention over caches held in 8 or 4 bits where rows differ widely in size: value
rows, among them rows that only some of the draft sees, and queries.

Tolerance, from the arithmetic (fp32 rounds by 2^-24 of a value, half by 2^-11, or by 2^-25
below 2^-14; bf16 by 2^-8).  With s the scale, sums over a row's elements i and the keys j
that a row sees, c_j the value row in units of its own scale and u the largest value scale
that the row sees:
  a score    128 additions: 2^-16 s sum_i |q_i k_i|; the query rounded to half, its block's
             largest element M at 2^14 or above: 2^-39 M s sum_i |k_i|; e = the largest of
             both over the keys, and 2^-22 of the largest score
  a weight   e, 2^-22 of the exponential, 2^-11 of the rounding; 2^-25 where it is
             small, beside 2^6 at the row's largest, and relative to u: 2^-31 u / l in all
             for l = sum_j exp(score_j - largest)
  an output  that of its weights and of l (e again); one addition in fp32 a key, n in all;
             and 2^-8 of itself
  an lse     e, n additions, and 2^-20 of its size
so   |out - exact| <= (2.1 e + 2^-20 + 2^-11 + n 2^-23) sum_j w_j |v_j| + 2^-31 u sum_j |c_j| / l + 2^-8 |exact|
     |lse - exact| <= 1.1 e + n 2^-23 + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

from tests import quantized as Q
from tests.test_gpu_attn_quant import FORMATS, Case

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

# (T, Hq, Hkv): blocks of 16, 32, 64 rows, several blocks, 128 rows (4 bits, d128)
BLOCKS = [(4, 8, 2), (10, 4, 2), (16, 8, 2), (29, 8, 2), (64, 4, 2), (64, 4, 1)]


def row_scales(rows, fmt, D):
    at = D if fmt == "e4m3" else D // 2 + D // 16
    return np.ascontiguousarray(rows[..., at:at + 4]).view("<f4")[..., 0].astype(np.float64)


def check(c, out, lse, scale=None):
    """Every row of case c within the bars above."""
    B, T, Hq, D = c.q.shape
    G = Hq // c.Hkv
    s = D ** -0.5 if scale is None else scale
    q = c.q.double().numpy()
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all() and not np.isnan(l).any()
    for b in range(B):
        vis = np.concatenate([np.ones((T, c.L[b]), bool), c.sees[b]], 1)
        n = vis.shape[1]
        for h in range(Hq):
            k, v = (Q.read(c.rows[x][b][:, h // G], c.fmt, D) for x in ("k", "v"))
            vs = row_scales(c.rows["v"][b][:, h // G], c.fmt, D)
            top = np.abs(q[b, :, h // G * G:(h // G + 1) * G]).max()  # (of the kv-head: at least the block's)
            z = np.where(vis, q[b, :, h] @ k.T * s, -np.inf)
            some = vis.any(1)
            assert np.array_equal(np.isneginf(l[b, h]), ~some) and not o[b, ~some, h].any()
            z, see = z[some], vis[some]
            m = z.max(1, keepdims=True)
            w = np.exp(z - m)
            tot = w.sum(1, keepdims=True)
            e = np.where(see, 2.0 ** -16 * (np.abs(q[b, some, h]) @ np.abs(k).T) * s, 0).max(1)
            e = e + np.where(see, 2.0 ** -39 * top * s * np.abs(k).sum(1), 0).max(1)
            e = (e + 2.0 ** -22 * np.abs(np.where(see, z, 0)).max(1))[:, None]
            u = np.where(see, vs, 0).max(1, keepdims=True)
            want = w @ v / tot
            bar = (2.1 * e + 2.0 ** -20 + 2.0 ** -11 + n * 2.0 ** -23) * (w @ np.abs(v) / tot)
            bar = bar + 2.0 ** -31 * u * (see @ (np.abs(v) / vs[:, None])) / tot + 2.0 ** -8 * np.abs(want)
            over = np.abs(o[b, some, h] - want) - bar
            assert over.max() <= 0, f"sequence {b}, head {h}: {over.max():.3e} over a bar of {bar.flat[over.argmax()]:.3e}"
            want = (m + np.log(tot))[:, 0]
            off = np.abs(l[b, h, some] - want) - (1.1 * e[:, 0] + n * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(want)))
            assert off.max() <= 0, f"sequence {b}, head {h}: lse {off.max():.3e} over the bar"


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 4, 2), (10, 4, 2), (16, 8, 2), (64, 4, 2)])
@pytest.mark.parametrize("up", [15, 24, 25, 26])
def test_a_large_value_row_of_next_to_no_weight(fmt, D, T, Hq, Hkv, up):
    """Weights keep what the documented 2^-31 of the largest value scale leaves of them."""
    def keys(rng, n):
        x = 0.3 * rng.standard_normal((n, Hkv, D))
        x[7] = -4.0  # a score of -4 sqrt(D)
        return x

    def vals(rng, n):
        x = rng.standard_normal((n, Hkv, D))
        x[7] *= 2.0 ** up
        return x

    rng = np.random.default_rng(up)
    q = (1 + 0.3 * rng.standard_normal((2, T, Hq, D))).astype(np.float32)
    c = Case(up, fmt, D, [40, 333], T, Hq, Hkv, 0, "chain", keys, vals, q)
    check(c, *c.run())


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("T,Hq,Hkv", BLOCKS)
@pytest.mark.parametrize("mode", ["tree", "mask"])
@pytest.mark.parametrize("up", [15, 30, 100])
def test_large_value_rows_on_other_branches(fmt, D, T, Hq, Hkv, mode, up):
    """Draft rows that some rows of a block see and others do not, with values 2^15 to 2^100
    times the others': a row is as exact as the keys that it sees let it be.  Prefixes that put
    the draft into the first tile, into two tiles, and into parts of a split segment."""
    def vals(rng, n):
        x = rng.standard_normal((n, Hkv, D))
        f = np.zeros(T)
        for t, more in ((2, up), (T // 2, up / 2), (T - 1, up)):
            f[t] += more
        x[n - T:] *= (2.0 ** np.minimum(f, 100))[:, None, None]  # (2^150 is past the row scale's fp32)
        return x

    c = Case(up + T, fmt, D, [0, 100, 300, 4500], T, Hq, Hkv, 16 if T == 29 else 0, mode, None, vals)
    check(c, *c.run())


def quiet_keys(D, loud):
    """Keys that are zero in their first `loud` elements."""
    def keys(rng, n, Hkv=2):
        x = rng.standard_normal((n, Hkv, D))
        x[..., :loud] = 0
        return x

    return keys


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("T,Hq,Hkv", BLOCKS)
@pytest.mark.parametrize("top", [10, 20, 30])
def test_queries_of_very_different_size_in_a_block(fmt, D, T, Hq, Hkv, top):
    """Rows whose largest elements are 1 to 2^top times those that meet a key: one power of two
    for a block of rows leaves the small ones what the documented 2^-39 of its largest does."""
    rng = np.random.default_rng(top + T)
    q = rng.standard_normal((3, T, Hq, D)).astype(np.float32)
    q[..., :16] *= 2.0 ** rng.choice([0, top // 2, top - 1, top], size=(3, T, Hq, 1))
    q[:, :, ::2, 16:] *= 2.0 ** -5
    c = Case(top * T, fmt, D, [0, 77, 2500], T, Hq, Hkv, 0, "tree", lambda rng, n: quiet_keys(D, 16)(rng, n, Hkv), None, q)
    check(c, *c.run())


@pytest.mark.parametrize("fmt,D", FORMATS)
def test_the_worst_rounding_of_a_query(fmt, D):
    """An element of 1.5 2^-38 beside one of 1: half a unit of the scaled query, 2^-39 of the
    largest, in a score that is nothing else."""
    q = np.zeros((1, 1, 1, D), np.float32)
    q[..., 0], q[..., 1] = 1, 1.5 * 2.0 ** -38

    def keys(rng, n):
        x = np.zeros((n, 1, D))
        x[..., 1] = 1
        return x

    c = Case(1, fmt, D, [0], 1, 1, 1, 0, "chain", keys, None, q)
    check(c, *c.run(scale=2.0 ** 38), scale=2.0 ** 38)


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("L,T,Hq,Hkv", [(300, 4, 4, 2), (20, 40, 4, 2), (20000, 4, 4, 2), (20000, 16, 8, 2), (20000, 64, 4, 1)])
@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("where", ["prefix", "draft"])
def test_a_key_stored_as_nan_reaches_out_and_lse(fmt, D, L, T, Hq, Hkv, name, where):
    """A key or value row whose scale is NaN makes out and lse NaN in every row that sees it,
    through the parities' join and the merge of a split segment, and in no other."""
    c = Case(L + T, fmt, D, [L, 33], T, Hq, Hkv, 0, "chain")
    plain, plain_lse = (x.clone() for x in c.run())
    at = Q.row_bytes(fmt, D) - 16 + (0 if fmt == "e4m3" else D // 16)
    slot = L // 2 if where == "prefix" else L + 2
    row = c.cache[name][0, slot, Hkv - 1]
    row[:] = 0
    row[at:at + 4] = torch.tensor([0, 0, 192, 127], dtype=torch.uint8)
    out, lse = c.run()
    want = torch.zeros(2, T, Hq, dtype=torch.bool, device="cuda")
    want[0, 0 if where == "prefix" else 2:, Hq - Hq // Hkv:] = True
    assert torch.equal(torch.isnan(out).all(-1), want) and torch.equal(torch.isnan(out).any(-1), want)
    assert torch.equal(torch.isnan(lse), want.transpose(1, 2))
    assert torch.equal(out[~want], plain[~want]) and torch.equal(lse.transpose(1, 2)[~want], plain_lse.transpose(1, 2)[~want])


@pytest.mark.parametrize("fmt,D", FORMATS)
@pytest.mark.parametrize("T,Hq,Hkv", BLOCKS)
def test_short_sequences_keep_their_lse(fmt, D, T, Hq, Hkv):
    """Small scores over a few keys, where the bar of an lse is 2^-20 and little more."""
    q = (2.0 ** -7 * np.random.default_rng(T).standard_normal((5, T, Hq, D))).astype(np.float32)
    c = Case(T, fmt, D, [0, 1, 9, 70, 200], T, Hq, Hkv, 0, "tree", None, None, q)
    check(c, *c.run())
