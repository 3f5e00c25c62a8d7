"""A query row with a NaN gets NaN from the shaped attention, out and lse, whatever
the rules, the kernel and the length, and no other row is touched; the weights of
its kv-head are NaN wherever the row sees a key."""
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests import shaped

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

# a cap far above the scores and one that most of them pass: both forms of the tanh
RULES = {"none": {}, "window": dict(window=100), "slopes": dict(slopes=True), "cap": dict(softcap=20.0),
         "low cap": dict(softcap=1.0), "all": dict(softcap=2.0, slopes=True, window=150)}
FORMS = {
    "bf16 d128 3 rows": ("bf16", 128, 3, 2, 2, 0),
    "bf16 d128 20 rows pages of 16": ("bf16", 128, 5, 8, 2, 16),
    "bf16 d128 64 rows": ("bf16", 128, 16, 8, 2, 0),
    "bf16 d128 100 rows": ("bf16", 128, 25, 4, 1, 0),
    "bf16 d128 256 rows": ("bf16", 128, 64, 4, 1, 0),
    "bf16 d64 64 rows": ("bf16", 64, 16, 4, 1, 0),
    "bf16 d64 80 rows pages of 2": ("bf16", 64, 20, 4, 1, 2),
    "fp32 d64 8 rows": ("fp32", 64, 2, 4, 1, 0),
    "fp32 d64 32 rows": ("fp32", 64, 8, 4, 1, 0),
    "fp32 d64 72 rows": ("fp32", 64, 18, 4, 1, 0),
}


@pytest.mark.parametrize("L", [[40, 300], [9000]], ids=["short", "split over the blocks"])
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("form", FORMS)
def test_a_nan_row(form, rule, L):
    dtype, D, T, Hq, Hkv, page = FORMS[form]
    c = shaped.make(5, L, T, Hq, Hkv, D, dtype, page, **RULES[rule])
    clean, clean_lse = shaped.run_attend(va, c)
    c.q[0, 1, 1, :3] = float("nan")
    out, lse = shaped.run_attend(va, c)
    assert lse[0, 1, 1].isnan() and out[0, 1, 1].isnan().all()
    out[0, 1, 1], lse[0, 1, 1] = clean[0, 1, 1], clean_lse[0, 1, 1]
    # (the rows of a tile decide together how many bits their weights keep)
    assert (out.float() - clean.float()).abs().max() <= 2e-3 + 2 ** -8 * clean.float().abs().max()
    assert (lse - clean_lse).abs().max() <= 1e-5
    w = shaped.run_weight(va, c, clean_lse, torch.zeros(c.B, Hkv, c.cap, device="cuda"))
    g = 1 // (Hq // Hkv)
    seen = max(0, L[0] + 1 - c.window + 1) if c.window else 0  # accepted row 1 is at L + 1
    nan = w.isnan()
    assert nan[0, g, seen:L[0] + 2].all() and int(nan.sum()) == L[0] + 2 - seen
