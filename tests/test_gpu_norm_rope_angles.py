"""The angles of the norm with rotation: unit vectors come back as cosine and sine.

Bar, from the arithmetic: an angle is off by at most 2^-26 + 2^-32 + |position| 2^-55 of a
turn, 2 pi as much in either result, its cosine and sine by 2^-23 (two units below 1);
the factors 1 and 0 that they meet round nothing.  The fp64 angle of the reference is
reduced by whole turns first (|position| 2^-53 of it at most, and the same for its frequency).
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("D", [16, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("lo,hi", [(0, 1 << 10), (0, 1 << 20), (-(1 << 24), 1 << 24), (-(1 << 31), 1 << 31)])
def test_angles(D, base, lo, hi):
    rng = np.random.default_rng(D)
    T = 5000
    p = rng.integers(lo, hi, size=(1, T)).astype(np.int32)
    p[0, :4] = [lo, hi - 1, 1, 0]
    x = torch.zeros(1, T, 2, D, device="cuda")
    x[..., : D // 2] = 1  # (1, 0) in every pair: (cos, sin)
    q, k = va.verify_norm_rope(x[:, :, :1], x[:, :, 1:], positions=torch.from_numpy(p).cuda(), rope_base=base)
    assert torch.equal(q, k)
    got = q[0, :, 0].double().cpu().numpy()
    turns = np.longdouble(base) ** (-2 * np.arange(D // 2, dtype=np.longdouble) / D) / (2 * np.longdouble(np.pi))
    ang = 2 * np.pi * np.fmod(p[0, :, None].astype(np.float64) * turns.astype(np.float64), 1.0)
    bar = 2 * np.pi * (2.0 ** -26 + 2.0 ** -32 + np.abs(p[0, :, None].astype(np.float64)) * (2.0 ** -55 + 2.0 ** -53 + 2.0 ** -53)) + 2.0 ** -23
    assert (np.abs(got[:, : D // 2] - np.cos(ang)) <= bar).all()
    assert (np.abs(got[:, D // 2:] - np.sin(ang)) <= bar).all()


@pytest.mark.parametrize("token_major", [False, True])
def test_outputs_without_room_behind_the_last_row(token_major):
    """Output rows with gaps between them and none behind the last: what lies in the gaps stays."""
    B, T, H, D, gap = 3, 5, 4, 64, 32
    row = H * D
    near, far = row + gap, ((B if token_major else T) - 1) * (row + gap) + row
    strides = (near, far, D, 1) if token_major else (far, near, D, 1)
    x = torch.randn(B, T, 2 * H, D, device="cuda").bfloat16()
    w = torch.ones(D, device="cuda").bfloat16()
    pos = torch.arange(B * T, dtype=torch.int32, device="cuda").view(B, T)
    want = va.verify_norm_rope(x[:, :, :H], x[:, :, H:], w, w, pos)
    size = 1 + (B - 1) * strides[0] + (T - 1) * strides[1] + row - 1
    flat = torch.full((2, size + 16), 7.0, device="cuda").bfloat16()
    out = [f[:size].as_strided((B, T, H, D), strides) for f in flat]
    va.verify_norm_rope(x[:, :, :H], x[:, :, H:], w, w, pos, q_out=out[0], k_out=out[1])
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    for f, o in zip(flat, out):
        o.fill_(7.0)
        assert (f == 7.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_at_the_ends_of_the_range(dtype):
    """Squares past 2^128 give zeros, and squares below fp32's range count as none beside eps;
    the rows around them are what they were."""
    x = torch.randn(1, 4, 3, 64, device="cuda").to(dtype)
    w = torch.ones(64, device="cuda", dtype=dtype)
    plain = va.verify_norm_rope(x[:, :, :2], x[:, :, 2:], w, w)[0]
    x[0, 1, 0], x[0, 2, 1] = 2.0 ** 64, 2.0 ** -80
    out = va.verify_norm_rope(x[:, :, :2], x[:, :, 2:], w, w, eps=1e-6)[0]
    assert (out[0, 1, 0] == 0).all()
    want = torch.full((64,), 2.0 ** -80 * 1000, dtype=torch.float64)  # 1 / sqrt(1e-6)
    assert ((out[0, 2, 1].double().cpu() - want).abs() <= (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20) * want).all()
    same = torch.ones(4, 2, dtype=torch.bool)
    same[1, 0] = same[2, 1] = False
    assert torch.equal(out[0][same], plain[0][same])
