"""Refusals of the norm with rotation and of the caches held in 8 or 4 bits: bad
arguments come back with the documented status before anything touches a device."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from speculative_decoding_verification_masked_gb300 import api

FAKE = 1 << 20  # a non-NULL address validation never dereferences
BAD, UNSUPPORTED, WORKSPACE = api.VA_ERR_INVALID_ARG, api.VA_ERR_UNSUPPORTED, api.VA_ERR_WORKSPACE


def _shape(**kw):
    d = dict(B=2, T=8, Hq=32, Hkv=8, D=128, dtype=0, scale=0.088, rope_base=10000.0)
    d.update(kw)
    return api.VaShape(*d.values())


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def _rows(ptr=FAKE, batch=1 << 20, token=1 << 14):
    return api.VaRows(ptr, batch, token)


def _norm(shape, q=None, k=None, q_out=None, k_out=None, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, null=()):
    args = dict(q=q or _rows(), k=k or _rows(), q_out=q_out or _rows(), k_out=k_out or _rows())
    r = {n: None if n in null else ctypes.byref(a) for n, a in args.items()}
    return api.lib().verify_norm_rope(_ref(shape), r["q"], r["k"], qw, kw, eps, pos, r["q_out"], r["k_out"], None)


def _write(shape, fmt=0, k=None, v=None, cache=FAKE, cap=100, start=FAKE, count=None, ws=None):
    return api.lib().verify_quantize_kv_dense(_ref(shape), fmt, _ref(k or _rows()), _ref(v or _rows()), cache, FAKE, cap,
                                              start, count, ws, None)


def _write_paged(shape, fmt=1, page=16, pages=10, table=FAKE, width=4):
    return api.lib().verify_quantize_kv_paged(_ref(shape), fmt, _ref(_rows()), _ref(_rows()), FAKE, FAKE, pages, page, table,
                                              width, FAKE, None, None, None)


def _read(shape, fmt=0, k=None, v=None, cache=FAKE, cap=100, start=FAKE, ws=None):
    return api.lib().verify_dequantize_kv_dense(_ref(shape), fmt, cache, FAKE, cap, start, None, _ref(k or _rows()),
                                                _ref(v or _rows()), ws, None)


def _attn(shape, fmt=1, q=FAKE, k=FAKE, parent=None, mask=None, ws=FAKE, cap=100, out=FAKE):
    return api.lib().verify_attn_dense_quant(_ref(shape), fmt, q, k, FAKE, cap, FAKE, parent, mask, out, FAKE, ws, 1 << 40,
                                             None)


def _attn_paged(shape, fmt=1, page=16, pages=10, table=FAKE, width=4):
    return api.lib().verify_attn_paged_quant(_ref(shape), fmt, FAKE, FAKE, FAKE, pages, page, table, width, FAKE, None, None,
                                             FAKE, FAKE, FAKE, 1 << 40, None)


def test_row_sizes():
    want = {("e4m3", 128): 144, ("e4m3", 64): 80, ("e2m1", 128): 80, ("e2m1", 64): 48}
    for (fmt, D), n in want.items():
        assert va.kv_row_bytes(fmt, D) == n
    L = api.lib()
    assert L.verify_kv_row_bytes(2, 128) == 0 and L.verify_kv_row_bytes(-1, 128) == 0 and L.verify_kv_row_bytes(0, 96) == 0
    with pytest.raises(ValueError):
        va.kv_row_bytes("int4", 128)
    with pytest.raises(ValueError):
        va.kv_row_bytes("e4m3", 256)


@pytest.mark.parametrize("kw,code", [
    (dict(shape=None), BAD), (dict(shape=_shape(T=0)), BAD), (dict(shape=_shape(Hkv=0)), BAD),
    (dict(shape=_shape(dtype=1)), BAD), (dict(shape=_shape(D=72)), UNSUPPORTED), (dict(shape=_shape(D=272)), UNSUPPORTED),
    (dict(shape=_shape(B=1 << 16, T=1 << 16)), UNSUPPORTED), (dict(shape=_shape(Hq=65536)), UNSUPPORTED),
    (dict(shape=_shape(rope_base=0.0)), BAD), (dict(shape=_shape(rope_base=float("nan"))), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("inf")), BAD), (dict(qw=FAKE + 8), BAD), (dict(kw=FAKE + 2), BAD),
    (dict(pos=FAKE + 2), BAD), (dict(null=("q",)), BAD), (dict(null=("k",)), BAD), (dict(null=("q_out",)), BAD),
    (dict(null=("k_out",)), BAD), (dict(q=_rows(ptr=None)), BAD), (dict(q=_rows(ptr=FAKE + 2)), BAD),
    (dict(k=_rows(token=(1 << 14) + 4)), BAD), (dict(k=_rows(batch=-8)), BAD), (dict(k=_rows(batch=1 << 41)), BAD),
    (dict(q_out=_rows(token=32 * 128 - 8)), BAD), (dict(k_out=_rows(token=0)), BAD),
    (dict(k_out=_rows(batch=1 << 14, token=1 << 14)), BAD),
])
def test_norm_refusals(kw, code):
    kw = dict(dict(shape=_shape()), **kw)
    assert _norm(**kw) == code
    assert api.lib().verify_attn_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(shape=None), BAD), (dict(shape=_shape(B=0)), BAD), (dict(shape=_shape(dtype=1)), BAD), (dict(fmt=2), BAD),
    (dict(fmt=-1), BAD), (dict(shape=_shape(D=96)), UNSUPPORTED), (dict(shape=_shape(B=65536)), UNSUPPORTED),
    (dict(shape=_shape(T=1 << 28)), UNSUPPORTED), (dict(cache=None), BAD), (dict(cache=FAKE + 8), BAD), (dict(cap=0), BAD),
    (dict(start=None), BAD), (dict(start=FAKE + 2), BAD), (dict(k=_rows(ptr=FAKE + 4)), BAD), (dict(v=_rows(token=4)), BAD),
    (dict(ws=FAKE + 16), WORKSPACE),
])
@pytest.mark.parametrize("call", [_write, _read])
def test_write_and_read_refusals(call, kw, code):
    kw = dict(dict(shape=_shape()), **kw)
    assert call(**kw) == code
    assert api.lib().verify_attn_last_error()


def test_read_back_into_one_place_is_refused():
    assert _read(_shape(), k=_rows(token=0)) == BAD
    assert _read(_shape(), v=_rows(token=8 * 128 - 8)) == BAD
    assert _read(_shape(), v=_rows(batch=0)) == BAD


@pytest.mark.parametrize("kw", [dict(page=0), dict(page=12), dict(page=2048), dict(table=None), dict(pages=0), dict(width=0),
                                dict(page=1024, width=1 << 20)])
def test_page_refusals(kw):
    assert _write_paged(_shape(), **kw) == BAD
    assert _attn_paged(_shape(), **kw) in (BAD, UNSUPPORTED)


@pytest.mark.parametrize("kw,code", [
    (dict(shape=None), BAD), (dict(fmt=2), BAD), (dict(shape=_shape(T=65)), UNSUPPORTED),
    (dict(shape=_shape(dtype=2, D=64)), UNSUPPORTED), (dict(shape=_shape(D=96)), UNSUPPORTED),
    (dict(shape=_shape(Hq=30)), BAD), (dict(shape=_shape(scale=0.0)), BAD), (dict(q=FAKE + 8), BAD), (dict(k=FAKE + 8), BAD),
    (dict(k=None), BAD), (dict(out=FAKE + 4), BAD), (dict(parent=FAKE, mask=FAKE), BAD), (dict(ws=None), WORKSPACE),
    (dict(ws=FAKE + 16), WORKSPACE), (dict(cap=7), BAD), (dict(shape=_shape(B=300, Hkv=8)), UNSUPPORTED),
])
def test_attention_refusals(kw, code):
    kw = dict(dict(shape=_shape()), **kw)
    assert _attn(**kw) == code
    assert api.lib().verify_attn_last_error()


def test_tensors_off_the_gpu_are_refused():
    x = torch.zeros(1, 2, 4, 128)
    c = torch.zeros(1, 8, 4, 80, dtype=torch.uint8)
    n = torch.zeros(1, dtype=torch.int32)
    for f, args in ((va.verify_norm_rope, (x, x)), (va.verify_quantize_kv_dense, (x, x, c, c, n, "e2m1")),
                    (va.verify_dequantize_kv_dense, (c, c, n, "e2m1", 2)),
                    (va.verify_attn_dense_quant, (x, c, c, n, "e2m1")),
                    (va.verify_attn_paged_quant, (x, c, c, n, n, "e2m1"))):
        with pytest.raises(ValueError):
            f(*args)
        with pytest.raises(TypeError):
            f(None, *args[1:])
