"""The norm with rotation and caches held in 8 or 4 bits from several host threads: a
thread's first use of the GPU, and all of them at once, a stream each."""
import threading

import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests.test_gpu_attn_quant import Case, dev

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)


def _attend(fmt, D, T, page):
    c = Case(T, fmt, D, [900, 0, 333], T, 8, 2, page, "tree")
    ws = va.Workspace.for_shape(va.make_shape(3, T, 8, 2, D, 0))
    q, L = c.q.cuda(), dev(c.L)
    out, lse = torch.empty_like(q), torch.empty(3, 8, T, device="cuda")
    kw = dict(tree_parent=c.parent, out=out, lse=lse, workspace=ws)
    if page:
        return lambda s: va.verify_attn_paged_quant(q, c.cache["k"], c.cache["v"], c.table, L, fmt, stream=s, **kw), (out, lse)
    return lambda s: va.verify_attn_dense_quant(q, c.cache["k"], c.cache["v"], L, fmt, stream=s, **kw), (out, lse)


def _norm():
    x = torch.randn(2, 50, 10, 128, device="cuda").bfloat16()
    w, pos = torch.ones(128, device="cuda").bfloat16(), torch.arange(100, dtype=torch.int32, device="cuda").view(2, 50)
    out = [torch.empty(2, 50, h, 128, device="cuda").bfloat16() for h in (8, 2)]
    return lambda s: va.verify_norm_rope(x[:, :, :8], x[:, :, 8:], w, w, pos, q_out=out[0], k_out=out[1], stream=s), out


def _write_and_read(fmt):
    x = torch.randn(2, 2, 70, 4, 64, device="cuda")
    cache = torch.zeros(2, 2, 100, 4, va.kv_row_bytes(fmt, 64), dtype=torch.uint8, device="cuda")
    back, start = torch.zeros_like(x), dev([0, 30])

    def call(s):
        va.verify_quantize_kv_dense(x[0], x[1], cache[0], cache[1], start, fmt, stream=s)
        va.verify_dequantize_kv_dense(cache[0], cache[1], start, fmt, k_out=back[0], v_out=back[1], stream=s)

    return call, (cache, back)


JOBS = {
    "16 rows": lambda: _attend("e2m1", 128, 3, 0),
    "32 rows, boxes of pages": lambda: _attend("e4m3", 128, 8, 16),
    "64 rows, gathered": lambda: _attend("e4m3", 64, 13, 4),
    "128 rows": lambda: _attend("e2m1", 128, 50, 0),
    "norm": _norm,
    "e4m3": lambda: _write_and_read("e4m3"),
    "e2m1": lambda: _write_and_read("e2m1"),
}


def _run(jobs, times):
    """Every job in a thread of its own, `times` calls each; what they leave is what one call
    of the main thread leaves."""
    jobs = [JOBS[j]() for j in jobs]
    want = []
    for call, outs in jobs:
        call(None)
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs])
        for x in outs:
            x.zero_()
    streams, errors = [torch.cuda.Stream() for _ in jobs], []
    torch.cuda.synchronize()

    def work(call, s):
        try:
            for _ in range(times):
                call(s)
        except Exception as e:  # noqa: BLE001 -- shown below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(call, s)) for (call, _), s in zip(jobs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors[0]
    for (_, outs), w in zip(jobs, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))


@pytest.mark.parametrize("job", JOBS)
def test_first_call_of_a_thread(job):
    _run([job], 1)


def test_all_at_once():
    _run(list(JOBS), 300)
