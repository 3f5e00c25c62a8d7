"""The per-head norm with rotation against fp64.

Tolerance, from the arithmetic (u = 2^-24): the sum of D squares is a tree of at most
16 + 4 steps in each lane and across lanes, so the mean is within 22 u and the factor
1 / sqrt within 11 u + 2 u; two products more are 2 u.  An angle is a 32-bit fraction of
a turn (off by 2^-32 turns, and by pos * 2^-55 turns for the 53 bits of its frequency)
rounded to 24 bits, its sine and cosine are within 2^-23, together below 2^-21 + pos 2^-52;
the rotation adds 2 u.  So before the last rounding an element is off by at most
(17 u + 2^-21 + |pos| 2^-51) (|y_i| + |y_j|) for its pair, and the fp64 angle of the
reference by another |pos| 2^-51: bars of 2^-19 + |pos| 2^-50 of the pair, plus 2^-8 of
the value for bf16.
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def reference(x, w, pos, eps, base):
    """(values, bound without the last rounding) in fp64; x [B][T][H][D]."""
    x = x.double().cpu()
    D = x.shape[-1]
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double().cpu()
    a, b = x[..., : D // 2], x[..., D // 2:]
    mag = (a.abs() + b.abs()).repeat(1, 1, 1, 2)
    bound = 2.0 ** -19 * mag
    if pos is not None:
        p = pos.double().cpu()[:, :, None, None]
        ang = p * base ** (-2 * torch.arange(D // 2, dtype=torch.float64) / D)
        bound = bound + p.abs() * 2.0 ** -50 * mag
        x = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    return x, bound


def check(got, x, w, pos, eps, base):
    want, bound = reference(x, w, pos, eps, base)
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * want.abs()
    err = (got.double().cpu() - want).abs()
    assert (err <= bound + 1e-37).all(), f"worst excess {(err - bound).max():.3e}"


def positions(kind, B, T, rng):
    if kind is None:
        return None
    lo, hi = {"near": (0, 4096), "far": (0, 1 << 24), "any": (-(1 << 31), 1 << 31)}[kind]
    return torch.from_numpy(rng.integers(lo, hi, size=(B, T)).astype(np.int32)).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [16, 64, 80, 96, 128, 256])
@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (3, 7, 8, 2), (2, 5, 33, 8), (1, 130, 5, 3)])
@pytest.mark.parametrize("kind", ["near", "any"])
def test_against_fp64(dtype, D, B, T, Hq, Hkv, kind):
    rng = np.random.default_rng(D + T)
    dt = TYPES[dtype]
    x = (torch.from_numpy(rng.standard_normal((B, T, Hq + 2 * Hkv, D)) * np.exp(rng.standard_normal((B, T, 1, 1))))
         .to(dt).cuda())
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]  # parts of one projection's output
    wq, wk = (torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).to(dt).cuda() for _ in range(2))
    pos = positions(kind, B, T, rng)
    before = x.clone()
    qo, ko = va.verify_norm_rope(q, k, wq, wk, pos, eps=1e-5, rope_base=500000.0)
    assert torch.equal(x, before) and qo.is_contiguous() and ko.is_contiguous()
    check(qo, q, wq, pos, 1e-5, 500000.0)
    check(ko, k, wk, pos, 1e-5, 500000.0)


@pytest.mark.parametrize("wq,wk,kind", [(False, False, "far"), (True, False, None), (False, True, "near"),
                                        (False, False, None)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_parts_left_out(dtype, wq, wk, kind):
    """No weight: those rows are only rotated; no positions: only normed; neither: copied."""
    rng = np.random.default_rng(1)
    dt = TYPES[dtype]
    q, k = (torch.from_numpy(rng.standard_normal((2, 6, h, 128))).to(dt).cuda() for h in (8, 4))
    w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(128)).to(dt).cuda() if on else None for on in (wq, wk)]
    pos = positions(kind, 2, 6, rng)
    qo, ko = va.verify_norm_rope(q, k, *w, pos)
    check(qo, q, w[0], pos, 1e-6, 10000.0)
    check(ko, k, w[1], pos, 1e-6, 10000.0)
    if kind is None and not wq:
        assert torch.equal(qo, q)


def test_in_place_and_strides():
    """In place inside a projection whose other parts stay as they are, time-major
    batches, a token broadcast to every sequence."""
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((4, 9, 14, 64))).bfloat16().cuda()
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(64)).bfloat16().cuda()
    pos = positions("far", 4, 9, rng)
    want = va.verify_norm_rope(x[:, :, :8], x[:, :, 8:10], w, w, pos)
    y = x.clone()
    va.verify_norm_rope(y[:, :, :8], y[:, :, 8:10], w, w, pos, q_out=y[:, :, :8], k_out=y[:, :, 8:10])
    assert torch.equal(y[:, :, :8], want[0]) and torch.equal(y[:, :, 8:10], want[1])
    assert torch.equal(y[:, :, 10:], x[:, :, 10:])
    t = x.transpose(0, 1).contiguous().transpose(0, 1)
    got = va.verify_norm_rope(t[:, :, :8], t[:, :, 8:10], w, w, pos)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    one = x[:1, :1].expand(4, 9, 14, 64)
    got = va.verify_norm_rope(one[:, :, :8], one[:, :, 8:10], w, w, pos)
    check(got[0], one[:, :, :8], w, pos, 1e-6, 10000.0)
    with pytest.raises(va.VerifyAttnError):  # outputs in one place
        va.verify_norm_rope(x[:, :, :8], x[:, :, 8:10], w, w, pos, q_out=one[:, :, :8], k_out=want[1])


def test_zero_rows_and_rows_that_are_not_finite():
    """A row of zeros stays zero; a NaN or infinity stays in its row."""
    x = torch.randn(1, 3, 6, 128, device="cuda")
    x[0, 1, 2] = 0
    x[0, 2, 3, 5], x[0, 0, 5, 100] = float("nan"), float("inf")
    w = torch.ones(128, device="cuda")
    pos = torch.tensor([[3, 4, 5]], dtype=torch.int32, device="cuda")
    q, k = va.verify_norm_rope(x[:, :, :4], x[:, :, 4:], w, w, pos)
    y = torch.cat([q, k], 2)
    assert (y[0, 1, 2] == 0).all() and torch.isnan(y[0, 2, 3]).any() and not torch.isfinite(y[0, 0, 5]).all()
    rest = torch.ones(1, 3, 6, dtype=torch.bool)
    rest[0, 2, 3] = rest[0, 0, 5] = False
    assert torch.isfinite(y[rest]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_without_positions_an_infinity_stays_in_its_place(dtype):
    """No rotation: what is not finite meets its row's sum of squares, not its partner.  Rows
    without a weight are copied as they are."""
    x = torch.randn(2, 3, 6, 128, device="cuda").to(TYPES[dtype])
    x[0, 1, 2, 7], x[1, 2, 3, 70], x[0, 0, 5, 3], x[1, 1, 4, 90] = (float(s) for s in ("inf", "nan", "-inf", "nan"))
    x[1, 0, 0, :64], x[1, 0, 1, 64:] = -0.0, -0.0
    w = torch.ones(128, device="cuda", dtype=x.dtype)
    q, k = va.verify_norm_rope(x[:, :, :4], x[:, :, 4:], None, w)
    assert torch.equal(q.nan_to_num(7.0), x[:, :, :4].nan_to_num(7.0)) and torch.equal(q.isnan(), x[:, :, :4].isnan())
    assert torch.equal(torch.signbit(q) & ~q.isnan(), torch.signbit(x[:, :, :4]) & ~q.isnan())
    nan = k[0, 0, 1].isnan()
    assert nan[3] and int(nan.sum()) == 1 and (k[0, 0, 1][~nan] == 0).all()  # (an infinite root)
    assert k[1, 1, 0].isnan().all()


def test_graph_and_refusals():
    x = torch.randn(2, 5, 10, 128, device="cuda").bfloat16()
    q, k = x[:, :, :8], x[:, :, 8:]
    w = torch.ones(128, device="cuda").bfloat16()
    pos = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty(2, 5, 8, 128, device="cuda").bfloat16(), torch.empty(2, 5, 2, 128, device="cuda").bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        va.verify_norm_rope(q, k, w, w, pos, q_out=qo, k_out=ko)
    with torch.cuda.graph(g, stream=s):
        va.verify_norm_rope(q, k, w, w, pos, q_out=qo, k_out=ko, stream=s)
    torch.cuda.synchronize()
    x.copy_(torch.randn_like(x))
    pos.copy_(torch.randint(0, 1000, (2, 5), dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    check(qo, q, w, pos, 1e-6, 10000.0)
    check(ko, k, w, pos, 1e-6, 10000.0)
    f = va.verify_norm_rope
    for bad in (dict(q_weight=w.float()), dict(q_weight=w[:64]), dict(positions=pos.long()), dict(positions=pos[:1]),
                dict(k=k.float()), dict(k=k[:, :4]), dict(q=q.transpose(1, 2)), dict(q=q.cpu()), dict(q_out=qo.float())):
        kw = dict(q=q, k=k, q_weight=w, k_weight=w, positions=pos)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError)):
            f(**kw)
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(rope_base=0.0), dict(rope_base=float("inf"))):
        with pytest.raises(va.VerifyAttnError):
            f(q, k, w, w, pos, **bad)
