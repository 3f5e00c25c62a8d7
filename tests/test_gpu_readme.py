"""The README's examples run, one after the other, on a step's inputs."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
import workloads as W
from tests.shaped import dev
from tests.test_readme_host import _blocks

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)


def test_the_examples_run():
    rng = np.random.default_rng(0)
    B, T, Hq, Hkv, D, cap = 2, 8, 32, 8, 128, 9100
    L = np.array([9000, 8700], np.int32)
    parent = np.stack([W.random_parents(T, rng) for _ in range(B)]).astype(np.int32)
    positions = (L[:, None] + np.stack([W.chain_depths(p) for p in parent])).astype(np.int32)
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)

    ws = va.Workspace.for_shape(va.make_shape(B, T, Hq, Hkv, D, 0))
    env = dict(q=normal(B, T, Hq, D), k_cache=normal(B, cap, Hkv, D), v_cache=normal(B, cap, Hkv, D), seqlens=dev(L),
               score_draft=torch.rand(B, Hkv, cap, device="cuda"), parent=dev(parent), positions=dev(positions),
               accepted_positions=dev(L[:, None] + np.arange(T, dtype=np.int32)),
               draft_tokens=dev(rng.integers(0, 2, (B, T)).astype(np.int32)),
               target_next=dev(rng.integers(0, 2, (B, T + 1)).astype(np.int32)),
               weight=torch.zeros(B, Hkv, cap, device="cuda"), ws=ws, cache_is_full=True)
    for block in _blocks():
        exec(block, env)  # noqa: S102 -- the repository's own text
        torch.cuda.synchronize()
        va.verify_attn_check_status(ws)
        assert torch.isfinite(env["out"].float()).all() and torch.isfinite(env["lse"]).all()
    assert env["new_len"].tolist() == [8192, 8192]
    assert torch.isfinite(env["weight"]).all() and float(env["weight"].sum()) > 0
