"""The capped score that a weight is made of, to the digits of fp32.

Each row's own key alone is visible (a window of one) and its product exact (one
element of q is not zero), so a weight is exp(s' - lse) with the kernel's score s',
and lse is set to the fp32 value next to s.  The polynomials are within 3.2e-8 of
tanh; Horner's last steps and the product with y round three times (2^-24 / sqrt 3
rms each, 6e-8 together); past 0.75 the rational form rounds about twice as often
(1.2e-7).  The exponential's 2^-22 is taken off as an absolute error.  That makes
7e-8 and 1.3e-7 rms of the score: bars of 1e-7 and 2e-7."""
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("cap", [15.0, 50.0])
@pytest.mark.parametrize("lo,hi,bar", [(0.1, 0.3, 1e-7), (0.3, 0.44, 1e-7), (0.44, 0.54, 1e-7), (0.55, 0.74, 1e-7),
                                       (0.76, 1.2, 2e-7), (1.2, 3.0, 2e-7)])
@pytest.mark.parametrize("dtype,D,T", [("bf16", 128, 16), ("bf16", 64, 8), ("fp32", 64, 8)])
def test_score_of_a_weight(dtype, D, T, lo, hi, bar, cap):
    g = torch.Generator().manual_seed(T)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    if dtype == "fp32":
        bar = 2e-7  # the rational form at every size
    B, H = 24, 2
    L = torch.randint(0, 300, (B,), generator=g).int()
    q = torch.zeros(B, T, H, D)
    col = torch.randint(D, (B, T, H), generator=g)
    q.scatter_(3, col[..., None], 2.0)
    u = torch.rand(B, 300 + T, H, D, generator=g) * (hi - lo) + lo
    k = (u * torch.where(torch.rand(u.shape, generator=g) < 0.5, -1.0, 1.0) * cap / 2).to(dt)
    at = (L[:, None] + torch.arange(T, dtype=torch.int32)).long()
    raw = 2.0 * k.double()[torch.arange(B)[:, None], at].gather(3, col[..., None])[..., 0]  # [B][T][H]
    s = cap * torch.tanh(raw / cap)
    lse = s.float()
    w = torch.zeros(B, H, 300 + T, device="cuda")
    va.verify_accumulate_weight_dense(q.to(dt).cuda(), k.cuda(), L.cuda(), lse.transpose(1, 2).contiguous().cuda(), w,
                                      mod=va.ScoreMod(softcap=cap, window=1), scale=1.0)
    got = w.cpu().double()[torch.arange(B)[:, None], :, at]  # [B][T][H]
    err = (got.log() + (lse.double() - s)).abs()
    rel = ((err - 2.0 ** -22).clamp(min=0) / s.abs())
    assert float((rel * rel).mean().sqrt()) <= bar, float((rel * rel).mean().sqrt())
