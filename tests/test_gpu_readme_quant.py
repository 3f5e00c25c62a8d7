"""The README's example of a cache held in 4 bits runs, and its rows are those of the
definition."""
import os
import re

import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
import workloads as W
from tests import quantized as Q
from tests.test_gpu_quant import dev

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)


def test_the_example_runs():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        blocks = re.findall(r"```py\n(.*?)```", f.read(), flags=re.S)
    assert len(blocks) == 1
    rng = np.random.default_rng(0)
    B, T, Hq, Hkv, D, cap = 2, 8, 32, 8, 128, 700
    L = np.array([600, 300], np.int32)
    parent = np.stack([W.random_parents(T, rng) for _ in range(B)]).astype(np.int32)
    depth = np.stack([W.chain_depths(p) for p in parent])
    past = rng.standard_normal((2, B, cap, Hkv, D)).astype(np.float32)
    cache = torch.from_numpy(Q.store(past, "e2m1")).cuda()
    env = dict(va=va, Hq=Hq, Hkv=Hkv, parent=dev(parent), positions=dev(L[:, None] + depth), seqlens=dev(L),
               qkv=torch.from_numpy(rng.standard_normal((B, T, Hq + 2 * Hkv, D)).astype(np.float32)).bfloat16().cuda(),
               q_weight=torch.ones(D, device="cuda").bfloat16(), k_weight=torch.ones(D, device="cuda").bfloat16(),
               k_cache=cache[0].contiguous(), v_cache=cache[1].contiguous(), start=dev([44, 0]),
               ws=va.Workspace.for_shape(va.make_shape(B, T, Hq, Hkv, D, 0)),
               path=dev([list(range(T))] * B), n_acc=dev([1, 0]))
    exec(blocks[0], env)  # noqa: S102 -- the repository's own text
    va.verify_attn_check_status(env["ws"])
    assert torch.isfinite(env["out"].float()).all() and torch.isfinite(env["lse"]).all()
    assert env["new_len"].tolist() == [601, 300]
    want = torch.from_numpy(Q.read(Q.store(past[1, 0, 44:300], "e2m1"), "e2m1", D)).bfloat16()
    assert torch.equal(env["v16"][0].cpu(), want)
