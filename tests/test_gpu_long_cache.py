"""Caches whose elements pass 2^31: the far sequence of a batch is read, weighed
and evicted at the right addresses.  The cache is zero but for a few rows, so the
results are known without a reference over all of it."""
import math

import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

B, CAP, HKV, D = 3, 1 << 20, 8, 128   # 3.2e9 elements, 6.4 GB a cache
L = CAP - 64
HOT = CAP - 100                       # the one key that stands out


def test_far_sequence():
    k = torch.zeros(B, CAP, HKV, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    q = torch.zeros(B, 2, 16, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    b = B - 1
    k[b, HOT, :, 0] = 64.0
    for h in range(HKV):
        v[b, HOT, h] = h + 1.0
    seqlens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    out, lse = va.verify_attn_dense_mod(q, k, v, seqlens, va.ScoreMod(softcap=30.0), scale=1.0)
    s = 30.0 * math.tanh(64.0 / 30.0)
    n = torch.arange(1, 3, device="cuda") + L - 1                # the other visible keys, all at score 0
    want = torch.log(torch.exp(torch.tensor(s, dtype=torch.float64)) + n.cpu().double())
    assert (lse[b].cpu().double() - want).abs().max() <= 1e-4
    p = torch.exp(s - want)                                      # weight of the one key
    heads = torch.arange(16) // 2 + 1
    got = out[b, :, :, 5].cpu().double()
    assert (got - p[:, None] * heads).abs().max() <= 2 ** -8 * 8  # half a bf16 step of values up to 8
    w = torch.zeros(B, HKV, CAP, device="cuda")
    va.verify_accumulate_weight_dense(q, k, seqlens, lse, w, mod=va.ScoreMod(softcap=30.0), scale=1.0)
    # two heads a kv-head, two rows; lse is off by at most 1e-4, so each term by 1e-4 of itself
    assert (w[b, :, HOT].cpu().double() - 2 * p.sum()).abs().max() <= 2e-4 * 4
    assert abs(float(w[b, 0].double().sum()) - 4.0) <= 1e-3
    idx = torch.tensor([0, HOT, L - 1], dtype=torch.int32, device="cuda").repeat(B, HKV, 1)
    v[b, L - 1] = -3.0
    new = va.verify_evict_kv_dense(k, v, seqlens, idx, torch.full((B, HKV), 3, dtype=torch.int32, device="cuda"), weight=w)
    assert new.tolist() == [3] * B
    assert (k[b, 1, :, 0] == 64.0).all() and (v[b, 1, :, 0].cpu() == torch.arange(1.0, HKV + 1)).all()
    assert (v[b, 2] == -3.0).all() and (v[0, 1] == 0).all()
    assert torch.equal(w[b, :, 1], w[b, :, HOT])
