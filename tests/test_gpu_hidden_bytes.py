"""What a key that no row sees holds does not matter, to the last bit: equal calls
over other bytes there, and after other work, give equal results.  The visible
scores stay small against the cap, the hidden ones are far past it."""
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests import shaped

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

L = [0, 5, 63, 130, 200, 301]
RULES = {
    "cap": dict(),
    "window": dict(window=70),
    "start": dict(start=[0, 2, 40, 129, 70, 300]),
    "slopes": dict(slopes=True, window=100),
}
# (dtype, D, T, Hq, Hkv, page)
FORMS = {
    "bf16 d128 3 rows": ("bf16", 128, 3, 2, 2, 0),
    "bf16 d128 20 rows pages of 16": ("bf16", 128, 5, 8, 2, 16),
    "bf16 d128 64 rows pages of 2": ("bf16", 128, 16, 8, 2, 2),
    "bf16 d128 100 rows": ("bf16", 128, 25, 4, 1, 0),
    "bf16 d128 256 rows pages of 8": ("bf16", 128, 64, 4, 1, 8),
    "bf16 d64 64 rows pages of 8": ("bf16", 64, 16, 4, 1, 8),
    "bf16 d64 80 rows": ("bf16", 64, 20, 4, 1, 0),
    "fp32 d64 32 rows pages of 4": ("fp32", 64, 8, 4, 1, 4),
}


def _scribble(c, value):
    """The case's K with `value` in every row that no query row sees."""
    k = c.k.clone()
    if c.table is not None:  # pages of no sequence, and the rows behind the last token
        used = torch.zeros(k.shape[:2], dtype=torch.bool)
    for b, n in enumerate(c.L.tolist()):
        lo = max(0, int(c.start[b]), n - c.window + 1 if c.window else 0)
        seen = range(min(lo, n), n + c.T)
        if c.table is None:
            k[b, :seen.start], k[b, seen.stop:] = value, value
        else:
            for j in seen:
                used[int(c.table[b][j // c.page]), j % c.page] = True
    if c.table is not None:
        k[~used] = value
    return k


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("form", FORMS)
def test_the_last_bits(form, rule):
    dtype, D, T, Hq, Hkv, page = FORMS[form]
    c = shaped.make(11, L, T, Hq, Hkv, D, dtype, page, softcap=50.0, **RULES[rule])
    noise = shaped.make(12, [700] * 8, T, Hq, Hkv, D, dtype, page, softcap=50.0, gain=500.0)
    weight = torch.rand(c.B, Hkv, c.cap, device="cuda")
    first = None
    for value in (0.0, 400.0, -30.0):
        c.k = _scribble(c, value)
        for busy in (False, True):
            if busy:  # other scores in every CTA's shared memory
                _, big = shaped.run_attend(va, noise)
                shaped.run_weight(va, noise, big, torch.zeros(8, Hkv, noise.cap, device="cuda"))
            out, lse = shaped.run_attend(va, c)
            w = shaped.run_weight(va, c, lse, weight.clone(), decay=0.5)
            if first is None:
                first = out, lse, w
            for got, want in zip((out, lse, w), first):
                assert torch.equal(got, want), (value, busy, float((got - want).abs().max()))
