"""An eviction whose blocks wait in vain for one of them: the documented error,
the lengths from before the call, and a scratch that serves the next call."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests.shaped import dev
from tests.test_gpu_evict import _expect, _make, _same

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("B,n", [(3, 1500), (40, 1500)])  # chunks of one turn of the blocks, and of several
@pytest.mark.parametrize("dtype,D,Hkv,page", [("bf16", 128, 4, 0), ("bf16", 128, 4, 16), ("fp32", 64, 2, 0)])
def test_lengths_and_scratch_after_a_lost_block(dtype, D, Hkv, page, B, n):
    L, keep = [2000 + b for b in range(B)], [n - b for b in range(B)]
    idx, n_idx, table, k, v, w = _make(B, L, keep, Hkv, D, dtype, page, "back")
    ws = va.Workspace(256)
    scratch = va.EvictScratch(B, Hkv, idx.shape[2])

    def run():
        kd, vd, wd = k.cuda(), v.cuda(), dev(w)
        args = (dev(np.asarray(L, np.int32)), dev(idx), dev(n_idx))
        new = torch.full((B,), -7, dtype=torch.int32, device="cuda")
        kw = dict(weight=wd, seqlens_out=new, scratch=scratch, workspace=ws)
        if page:
            va.verify_evict_kv_paged(kd, vd, dev(table), *args, **kw)
        else:
            va.verify_evict_kv_dense(kd, vd, *args, **kw)
        return kd, vd, wd, new

    lib = va.api.lib()
    assert lib.verify_attn_test_inject(2_000_000, 0) == 0
    try:
        kd, vd, wd, new = run()
        with pytest.raises(va.VerifyAttnError) as ei:
            va.verify_attn_check_status(ws)
        assert ei.value.status == va.api.VA_ERR_TIMEOUT
    finally:
        assert lib.verify_attn_test_inject(0, -1) == 0
    assert new.tolist() == L
    assert not scratch.buffer[scratch.offset:scratch.offset + scratch.nbytes].any()
    if not page:  # behind the kept rows nothing was touched
        for b in range(B):
            assert _same(kd[b, keep[b]:].cpu(), k[b, keep[b]:]) and _same(vd[b, keep[b]:].cpu(), v[b, keep[b]:])
            assert np.array_equal(wd[b, :, keep[b]:].cpu().numpy(), w[b, :, keep[b]:])
    kd, vd, wd, new = run()
    va.verify_attn_check_status(ws)
    k2, v2, w2 = _expect(L, idx, n_idx, table, page, k, v, w)
    assert _same(kd.cpu(), k2) and _same(vd.cpu(), v2) and np.array_equal(wd.cpu().numpy(), w2)
    assert new.tolist() == keep
