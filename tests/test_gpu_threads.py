"""Calls from host threads other than the first one."""
import sys
import threading

import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests import shaped

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

CALLS = 4000


def _attend(B, T, Hq, Hkv, D, dtype, plain=False):
    c = shaped.make(B + T, [40] * B, T, Hq, Hkv, D, dtype, softcap=0.0 if plain else 20.0)
    ws = va.Workspace.for_shape(va.make_shape(B, T, Hq, Hkv, D, 0 if dtype == "bf16" else 2))
    q, k, v, L = c.q.cuda(), c.k.cuda(), c.v.cuda(), shaped.dev(c.L)
    out, lse = torch.empty_like(q), torch.empty(B, Hq, T, device="cuda")
    mod = shaped.mod_of(va, c)

    def call(stream):
        if plain:
            va.verify_attn_dense(q, k, v, L, out=out, lse=lse, workspace=ws, stream=stream)
        else:
            va.verify_attn_dense_mod(q, k, v, L, mod, out=out, lse=lse, workspace=ws, stream=stream)

    return call, (out, lse)


def _weigh(B, T, Hq, Hkv, D):
    c = shaped.make(B + T, [40] * B, T, Hq, Hkv, D)
    q, k, L = c.q.cuda(), c.k.cuda(), shaped.dev(c.L)
    lse = torch.full((B, Hq, T), 8.0, device="cuda")
    weight = torch.zeros(B, Hkv, c.cap, device="cuda")

    def call(stream):
        va.verify_accumulate_weight_dense(q, k, L, lse, weight, decay=0.0, stream=stream)

    return call, (weight,)


def _commit(B, T, D):
    g = torch.Generator(device="cuda").manual_seed(T)
    k = torch.randn(B, 100, 2, D, generator=g, device="cuda")
    v = torch.randn(B, 100, 2, D, generator=g, device="cuda")
    L = torch.full((B,), 20, dtype=torch.int32, device="cuda")
    path = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
    n = torch.full((B,), T, dtype=torch.int32, device="cuda")
    new = torch.empty_like(L)

    def call(stream):
        va.verify_commit_kv_dense(k, v, L, path, n, seqlens_out=new, stream=stream)

    return call, (k, v, new)


FIRST = {
    "attend": lambda: _attend(2, 8, 8, 2, 128, "bf16"),
    "attend, rows on lanes": lambda: _attend(1, 64, 4, 1, 128, "bf16"),
    "attend, fp32": lambda: _attend(2, 8, 4, 1, 64, "fp32"),
    "plain": lambda: _attend(2, 8, 8, 2, 128, "bf16", True),
    "weights": lambda: _weigh(2, 8, 8, 2, 128),
    "commit": lambda: _commit(2, 64, 256),
}


@pytest.mark.parametrize("job", FIRST)
def test_first_call_of_a_thread(job):
    """A thread's very first use of the GPU is the call itself."""
    call, outs = FIRST[job]()
    call(None)
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    s, errors = torch.cuda.Stream(), []
    for x in outs:
        x.zero_() if job != "commit" else None
    torch.cuda.synchronize()

    def run():
        try:
            call(s)
        except Exception as e:  # noqa: BLE001 -- reported by the main thread
            errors.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert not errors, errors[0]
    s.synchronize()
    for got, ref in zip(outs, want):
        assert torch.equal(got, ref)


class _Recorder:
    """Stands in for the loaded library: notes a call's function and arguments."""

    def __init__(self, real):
        self.real, self.seen = real, None

    def __getattr__(self, name):
        f = getattr(self.real, name)

        def note(*args):
            self.seen = (f, args)
            return 0

        return note


def _c_call(call, stream):
    """The C call behind a Python call, to be made again and again with little around it."""
    real = va.api.lib()
    rec = _Recorder(real)
    va.api._lib = rec
    try:
        call(stream)
    finally:
        va.api._lib = real
    return rec.seen


# one kernel instance each, with different needs of shared memory (sequences, rows)
PAIRS = {
    "keys on lanes": lambda: (_attend(1, 8, 8, 2, 128, "bf16"), _attend(8, 8, 32, 8, 128, "bf16")),
    "keys on lanes, d64": lambda: (_attend(1, 4, 4, 1, 64, "bf16"), _attend(8, 4, 32, 8, 64, "bf16")),
    "rows on lanes": lambda: (_attend(1, 64, 4, 1, 128, "bf16"), _attend(8, 64, 32, 8, 128, "bf16")),
    "fp32": lambda: (_attend(1, 8, 4, 1, 64, "fp32"), _attend(8, 8, 32, 8, 64, "fp32")),
    "plain": lambda: (_attend(1, 8, 8, 2, 128, "bf16", True), _attend(8, 8, 32, 8, 128, "bf16", True)),
    "plain, d64": lambda: (_attend(1, 4, 4, 1, 64, "bf16", True), _attend(8, 4, 32, 8, 64, "bf16", True)),
    "plain, rows on lanes": lambda: (_attend(1, 64, 4, 1, 128, "bf16", True), _attend(8, 64, 32, 8, 128, "bf16", True)),
    "weights": lambda: (_weigh(1, 8, 8, 2, 128), _weigh(8, 32, 32, 8, 128)),
    "commit": lambda: (_commit(2, 64, 256), _commit(2, 49, 256)),
}


@pytest.mark.parametrize("pair", PAIRS)
def test_two_threads_of_one_kernel(pair):
    """What a launch sets on a kernel belongs to the process, not to the call: calls of
    different sizes at the same time all succeed and give what a lone call gives."""
    jobs = PAIRS[pair]()
    want, work = [], []
    for call, outs in jobs:
        call(None)
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs])
        s = torch.cuda.Stream()
        work.append((*_c_call(call, s), s))
    errors = []

    def run(f, args, s):
        for i in range(CALLS):
            status = f(*args)
            if status != 0:
                errors.append((i, status, va.api.lib().verify_attn_last_error().decode()))
                break
            if i % 200 == 199:
                s.synchronize()
        s.synchronize()

    old = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        threads = [threading.Thread(target=run, args=w) for w in work]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(old)
    assert not errors, errors[0]
    for (_, outs), w in zip(jobs, want):
        for got, ref in zip(outs, w):
            assert torch.equal(got, ref)
