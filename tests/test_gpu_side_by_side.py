"""Shaped attention, accumulated weight and eviction at the same time, each on a
stream, workspace and scratch of its own: the launches whose blocks wait for one
another share the GPU with others, no wait runs out and every result is a lone
call's."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests import shaped
from tests.shaped import dev
from tests.test_gpu_evict import _make

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)


def test_three_streams():
    jobs = []
    for seed, (T, Hq, Hkv, D, dtype) in enumerate([(8, 8, 2, 128, "bf16"), (64, 4, 1, 128, "bf16"), (8, 8, 2, 64, "bf16"),
                                                   (8, 8, 2, 64, "fp32")]):
        c = shaped.make(seed, [6000, 500, 31], T, Hq, Hkv, D, dtype, 16, softcap=20.0, slopes=True)
        ws, ws2 = (va.Workspace.for_shape(va.make_shape(3, T, Hq, Hkv, D, 0 if dtype == "bf16" else 2)) for _ in range(2))
        q, k, v, table, L, mod = c.q.cuda(), c.k.cuda(), c.v.cuda(), dev(c.table), dev(c.L), shaped.mod_of(va, c)
        out, lse = torch.empty_like(q), torch.empty(3, Hq, T, device="cuda")
        lse0, w = torch.full_like(lse, 6.0), torch.zeros(3, Hkv, c.cap, device="cuda")

        def attend(s, a=(q, k, v, table, L, mod), o=out, l=lse, ws=ws):
            va.verify_attn_paged_mod(*a, out=o, lse=l, workspace=ws, stream=s)

        def weigh(s, a=(q, k, table, L, lse0, w), mod=mod, ws=ws2):
            va.verify_accumulate_weight_paged(*a, mod=mod, decay=0.0, workspace=ws, stream=s)

        jobs += [(attend, ws, (out, lse)), (weigh, ws2, (w,))]
    Lk, keep = [9000, 4000], [7000, 4000]
    idx, n, _, k, v, w = _make(3, Lk, keep, 2, 128, "bf16", 0, "front")  # nothing moves: the same call again and again
    n_idx, k, v, w, idx, L = dev(n), k.cuda(), v.cuda(), dev(w), dev(idx), dev(np.asarray(Lk, np.int32))
    ws, scratch, new = va.Workspace(256), va.EvictScratch(2, 2, idx.shape[2]), torch.empty(2, dtype=torch.int32, device="cuda")

    def evict(s):
        va.verify_evict_kv_dense(k, v, L, idx, n_idx, weight=w, seqlens_out=new, scratch=scratch, workspace=ws, stream=s)

    jobs.append((evict, ws, (k, v, w, new)))
    want = []
    for call, _, outs in jobs:
        call(None)
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs])
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(200):
        for (call, _, _), s in zip(jobs, streams):
            call(s)
    torch.cuda.synchronize()
    for (_, ws, outs), ref, s in zip(jobs, want, streams):
        va.verify_attn_check_status(ws, stream=s)
        for got, x in zip(outs, ref):
            assert torch.equal(got, x)
