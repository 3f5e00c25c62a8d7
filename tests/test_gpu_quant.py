"""Caches held in 8 or 4 bits: what is written is bit for bit what the definition
says (every rounding of it is exact, so there is no tolerance), reading back gives
exactly what the bytes stand for, and nothing else changes."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from tests import quantized as Q

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def make_cache(rng, L, T, Hkv, nbytes, page):
    """Two caches of random bytes, their page table and a map (b, slot) -> index of a row of heads."""
    B = len(L)
    if page:
        need = [-(-(n + T) // page) for n in L]
        perm = rng.permutation(sum(need) + 1).astype(np.int32)
        table = np.full((B, max(need)), -1, np.int32)
        for b, n in enumerate(need):
            table[b, :n], perm = perm[:n], perm[n:]
        shape = (sum(need) + 1, page, Hkv, nbytes)
        at = lambda b, slot: (table[b, slot // page], slot % page)  # noqa: E731
    else:
        table, shape = None, (B, max(L) + T + 2, Hkv, nbytes)
        at = lambda b, slot: (b, slot)  # noqa: E731
    k, v = (rng.integers(0, 256, size=shape).astype(np.uint8) for _ in range(2))
    return k, v, table, at


def call(what, *args, table=None, **kw):
    f = getattr(va, f"verify_{what}_kv_{'dense' if table is None else 'paged'}")
    head, tail = args[:-2], args[-2:]
    return f(*head, *([] if table is None else [dev(table)]), *tail, **kw)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("page,T,Hkv,ragged", [(0, 1, 1, False), (0, 37, 3, True), (1, 5, 8, False), (16, 64, 2, True),
                                               (256, 333, 4, True)])
def test_written_and_read(fmt, D, dtype, page, T, Hkv, ragged):
    rng = np.random.default_rng(T * 31 + D + page)
    L = [0, 7, 130]
    n = [T, 0, max(1, T // 2)] if ragged else [T] * 3
    k, v, table, at = make_cache(rng, L, T, Hkv, va.kv_row_bytes(fmt, D), page)
    assert k.shape[-1] == Q.row_bytes(fmt, D)
    x = Q.rows_in(rng, (3, T, 3 * Hkv, D), TYPES[dtype]).cuda()  # k and v inside one projection's output
    xk, xv = x[:, :, Hkv:2 * Hkv], x[:, :, 2 * Hkv:]
    kd, vd = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    ws = va.Workspace(4096)
    count = dev(n) if ragged else None
    call("quantize", xk, xv, kd, vd, dev(L), fmt, table=table, n_tokens=count, workspace=ws)
    va.verify_attn_check_status(ws)
    for name, cache, got, rows in (("k", k, kd, xk), ("v", v, vd, xv)):
        want = cache.copy()
        for b in range(3):
            stored = Q.store(rows[b, :n[b]].double().cpu().numpy(), fmt)
            for t in range(n[b]):
                want[at(b, L[b] + t)] = stored[t]
        Q.same_bytes(got.cpu().numpy(), want, fmt, D)

    out = [torch.full((3, T, Hkv, D), 7.0, dtype=TYPES[dtype], device="cuda") for _ in range(2)]
    call("dequantize", kd, vd, dev(L), fmt, table=table, n_tokens=count, k_out=out[0], v_out=out[1], workspace=ws)
    va.verify_attn_check_status(ws)
    for cache, got in ((kd, out[0]), (vd, out[1])):
        host = cache.cpu().numpy()
        for b in range(3):
            assert (got[b, n[b]:] == 7.0).all()
            if n[b] == 0:
                continue
            rows = np.stack([host[at(b, L[b] + t)] for t in range(n[b])])
            want = torch.from_numpy(Q.read(rows, fmt, D)).to(TYPES[dtype])
            assert torch.equal(torch.nan_to_num(got[b, :n[b]].cpu(), nan=9e9), torch.nan_to_num(want, nan=9e9))


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_many_random_rows_round_exactly(fmt):
    """fp32 rows of full mantissas, and neighbours of the borders by one unit."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((1, 4096, 4, 128)).astype(np.float32)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32)
    g = Q.E4M3[rng.integers(8, 126, size=(1, 2048, 4, 8, 1))].astype(np.float32)
    edge = (ties[rng.integers(0, 8, size=(1, 2048, 4, 8, 16))] * g).reshape(1, 2048, 4, 128)
    x[:, :2048] = np.nextafter(edge, np.where(rng.random(edge.shape) < 0.5, 0, np.inf).astype(np.float32))
    cache = torch.zeros(2, 1, 4096, 4, va.kv_row_bytes(fmt, 128), dtype=torch.uint8, device="cuda")
    xd = torch.from_numpy(x).cuda()
    va.verify_quantize_kv_dense(xd, xd, cache[0], cache[1], dev([0]), fmt)
    want = Q.store(x, fmt)
    Q.same_bytes(cache[0].cpu().numpy(), want, fmt, 128)
    Q.same_bytes(cache[1].cpu().numpy(), want, fmt, 128)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_row_that_is_not_finite_reads_back_as_nan(fmt, bad):
    x = torch.randn(1, 4, 2, 128, device="cuda").bfloat16()
    x[0, 2, 1, 77] = bad
    cache = torch.full((2, 1, 6, 2, va.kv_row_bytes(fmt, 128)), 255, dtype=torch.uint8, device="cuda")
    va.verify_quantize_kv_dense(x, x, cache[0], cache[1], dev([1]), fmt)
    k, v = va.verify_dequantize_kv_dense(cache[0], cache[1], dev([1]), fmt, n=4)
    for y in (k, v):
        nan = torch.isnan(y)
        assert nan[0, 2, 1].all() and nan.sum() == 128


@pytest.mark.parametrize("page", [0, 16])
def test_bad_lengths_and_pages(page):
    """A sequence that does not fit is left alone, a row of a bad page is not written;
    the others are as they should be."""
    fmt, Hkv, T = "e2m1", 2, 4
    rng = np.random.default_rng(1)
    L = [3, 14, 2, 40]
    k, v, table, at = make_cache(rng, L, T, Hkv, 80, page)
    x = torch.from_numpy(rng.standard_normal((4, T, Hkv, 128)).astype(np.float32)).bfloat16().cuda()
    want = Q.store(x.double().cpu().numpy(), fmt)
    for seq, count in ((L[:2] + [-1, 40], [T] * 4), (L[:2] + [1 << 30, 40], [T] * 4), (L, [T, T, T + 1, T]),
                       (L, [T, T, -1, T])):
        kd, vd, ws = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), va.Workspace(4096)
        call("quantize", x, x, kd, vd, dev(seq), fmt, table=table, n_tokens=dev(count), workspace=ws)
        expect = k.copy()
        for b in (0, 1, 3):
            for t in range(T):
                expect[at(b, L[b] + t)] = want[b, t]
        assert np.array_equal(kd.cpu().numpy(), expect)
        with pytest.raises(va.VerifyAttnError) as e:
            va.verify_attn_check_status(ws)
        assert e.value.status == 6
        out = [torch.full((4, T, Hkv, 128), 7.0, device="cuda") for _ in range(2)]
        call("dequantize", kd, vd, dev(seq), fmt, table=table, n_tokens=dev(count), k_out=out[0], v_out=out[1], workspace=ws)
        assert (out[0][2] == 7.0).all() and (out[0][[0, 1, 3]] != 7.0).any()
        with pytest.raises(va.VerifyAttnError):
            va.verify_attn_check_status(ws)
    if page:
        for entry in (-1, len(k)):
            t2 = table.copy()
            t2[1, 1] = entry  # slots 16, 17 of sequence 1
            kd, vd, ws = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), va.Workspace(4096)
            call("quantize", x, x, kd, vd, dev(L), fmt, table=t2, workspace=ws)
            expect = k.copy()
            for b in range(4):
                for t in range(T):
                    if not (b == 1 and L[b] + t >= 16):
                        expect[at(b, L[b] + t)] = want[b, t]
            assert np.array_equal(kd.cpu().numpy(), expect)
            with pytest.raises(va.VerifyAttnError):
                va.verify_attn_check_status(ws)


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("fmt,D", [("e4m3", 128), ("e2m1", 128), ("e4m3", 64), ("e2m1", 64)])
def test_commit_and_eviction_move_quantised_rows(fmt, D, page):
    rng = np.random.default_rng(3)
    L, T, Hkv = [20, 33], 6, 3
    k, v, table, at = make_cache(rng, L, T, Hkv, va.kv_row_bytes(fmt, D), page)
    kd, vd = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    path = np.array([[1, 3, 5, -1, -1, -1], [0, 4, -1, -1, -1, -1]], np.int32)
    n = [3, 2]
    pages = [] if table is None else [dev(table)]
    commit = va.verify_commit_kv_dense if table is None else va.verify_commit_kv_paged
    new = commit(kd, vd, *pages, dev(L), dev(path), dev(n))
    assert new.tolist() == [23, 35]
    want = k.copy()
    for b in range(2):
        for j in range(n[b]):
            want[at(b, L[b] + j)] = k[at(b, L[b] + path[b, j])]
    assert np.array_equal(kd.cpu().numpy(), want)
    idx = np.full((2, Hkv, 16), -1, np.int32)
    m = [16, 9]
    for b in range(2):
        for h in range(Hkv):
            idx[b, h, :m[b]] = np.sort(rng.permutation(int(new[b]))[:m[b]])
    evict = va.verify_evict_kv_dense if table is None else va.verify_evict_kv_paged
    kept = evict(kd, vd, *pages, new, dev(idx), dev([[x] * Hkv for x in m]))
    assert kept.tolist() == m
    got = kd.cpu().numpy()
    for b in range(2):
        for h in range(Hkv):
            for j in range(m[b]):
                assert np.array_equal(got[at(b, j)][h], want[at(b, idx[b, h, j])][h])


def test_streams_graphs_and_wrong_tensors():
    """A captured and replayed pair of calls on a stream of its own sees the inputs of
    the replay; tensors of other types, shapes and strides are refused."""
    fmt, T, Hkv = "e2m1", 9, 2
    x = torch.randn(2, T, Hkv, 128, device="cuda").bfloat16()
    cache = torch.zeros(2, 2, 40, Hkv, 80, dtype=torch.uint8, device="cuda")
    start = dev([0, 30])
    out = [torch.zeros(2, T, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        va.verify_quantize_kv_dense(x, x, cache[0], cache[1], start, fmt)  # (loads the kernels)
        va.verify_dequantize_kv_dense(cache[0], cache[1], start, fmt, k_out=out[0], v_out=out[1])
    with torch.cuda.graph(g, stream=s):
        va.verify_quantize_kv_dense(x, x, cache[0], cache[1], start, fmt, stream=s)
        va.verify_dequantize_kv_dense(cache[0], cache[1], start, fmt, k_out=out[0], v_out=out[1], stream=s)
    torch.cuda.synchronize()
    x.copy_(torch.randn_like(x))
    start.copy_(dev([3, 11]))
    g.replay()
    torch.cuda.synchronize()
    want = torch.from_numpy(Q.read(Q.store(x.double().cpu().numpy(), fmt), fmt, 128)).bfloat16()
    assert torch.equal(out[0].cpu(), want) and torch.equal(out[1].cpu(), want)

    f = va.verify_quantize_kv_dense
    for bad, kind in ((x.half(), TypeError), (x.transpose(1, 2), ValueError), (x[..., :64], ValueError),
                      (x.cpu(), ValueError)):
        with pytest.raises(kind):
            f(bad, x, cache[0], cache[1], start, fmt)
        with pytest.raises((TypeError, ValueError)):
            f(x, bad, cache[0], cache[1], start, fmt)
    with pytest.raises(ValueError):
        f(x, x, cache[0], cache[1], start, "int4")
    with pytest.raises(ValueError):
        f(x, x, cache[0], cache[1], start, "e4m3")  # rows of another size
    with pytest.raises(va.VerifyAttnError):  # every row of the output in one place
        va.verify_dequantize_kv_dense(cache[0], cache[1], start, fmt, k_out=out[0][:, :1].expand(2, T, Hkv, 128),
                                      v_out=out[1])
    with pytest.raises(va.VerifyAttnError):  # rows that are not 16-byte aligned
        y = torch.zeros(2 * T * Hkv * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(2, T, Hkv, 128)
        f(y, y, cache[0], cache[1], start, fmt)


def test_slots_past_two_billion_bytes():
    """Offsets past 32 bits: the last slots of a cache of 2.4 GB."""
    fmt, Hkv, cap = "e4m3", 8, (1 << 21) + 77
    cache = torch.zeros(1, cap, Hkv, 144, dtype=torch.uint8, device="cuda")
    x = torch.randn(1, 5, Hkv, 128, device="cuda").bfloat16()
    start = dev([cap - 5])
    va.verify_quantize_kv_dense(x, x, cache, cache, start, fmt)
    k, _ = va.verify_dequantize_kv_dense(cache, cache, start, fmt, n=5)
    want = torch.from_numpy(Q.read(Q.store(x.double().cpu().numpy(), fmt), fmt, 128)).bfloat16()
    assert torch.equal(k.cpu(), want) and not cache[0, :cap - 5].any()
