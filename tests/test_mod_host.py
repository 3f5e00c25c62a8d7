"""Refusals of the score-shaping attention, the accumulated weight and the
eviction: bad arguments come back with the documented status before anything
touches a device."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_masked_gb300 as va
from speculative_decoding_verification_masked_gb300 import api

FAKE = 1 << 20  # a non-NULL address validation never dereferences
BAD, UNSUPPORTED, WORKSPACE = api.VA_ERR_INVALID_ARG, api.VA_ERR_UNSUPPORTED, api.VA_ERR_WORKSPACE


def _shape(**kw):
    d = dict(B=1, T=8, Hq=32, Hkv=8, D=128, dtype=0, scale=0.088, rope_base=0.0)
    d.update(kw)
    return api.VaShape(*d.values())


def _mod(softcap=0.0, window=0, slopes=None, key_start=None, token_pos=None):
    return api.VaScoreMod(softcap, window, slopes, key_start, token_pos)


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def _attn(shape, mod, parent=None, mask=None, q=FAKE, ws=FAKE, k=FAKE, max_len=100):
    return api.lib().verify_attn_dense_mod(_ref(shape), _ref(mod), q, k, FAKE, max_len, FAKE, parent, mask, FAKE, FAKE,
                                           ws, 1 << 30, None)


def _attn_paged(shape, mod, page=16, table=FAKE):
    return api.lib().verify_attn_paged_mod(_ref(shape), _ref(mod), FAKE, FAKE, FAKE, 10, page, table, 4, FAKE, None,
                                           None, FAKE, FAKE, FAKE, 1 << 30, None)


@pytest.mark.parametrize("kw", [dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
                                dict(softcap=1e-40), dict(softcap=3e38), dict(window=-1), dict(window=(1 << 23) + 1),
                                dict(slopes=FAKE + 2), dict(key_start=FAKE + 1), dict(token_pos=FAKE + 2)])
def test_bad_shaping(kw):
    assert _attn(_shape(), _mod(**kw)) == BAD
    assert _attn_paged(_shape(), _mod(**kw)) == BAD
    assert _weight(_shape(), _mod(**kw)) == BAD
    assert api.lib().verify_attn_last_error()


@pytest.mark.parametrize("draft", ["parent", "mask"])
@pytest.mark.parametrize("kw", [dict(window=8), dict(slopes=FAKE)])
def test_a_tree_or_mask_needs_positions(draft, kw):
    assert _attn(_shape(), _mod(**kw), **{draft: FAKE}) == BAD
    assert "token_pos" in api.lib().verify_attn_last_error().decode()


def test_attention_arguments():
    assert _attn(_shape(), None) == BAD
    assert _attn(None, _mod()) == BAD
    assert _attn(_shape(T=65), _mod()) == UNSUPPORTED
    assert _attn(_shape(D=96), _mod()) == UNSUPPORTED
    assert _attn(_shape(), _mod(), q=FAKE + 4) == BAD
    assert _attn(_shape(), _mod(), k=None) == BAD
    assert _attn(_shape(), _mod(), ws=FAKE + 16) == WORKSPACE
    assert _attn(_shape(), _mod(), parent=FAKE, mask=FAKE) == BAD
    assert _attn(_shape(), _mod(), max_len=3) == BAD
    assert _attn_paged(_shape(), _mod(), page=12) == BAD
    assert _attn_paged(_shape(), _mod(), table=None) == BAD


def _weight(shape, mod=None, q=FAKE, lse=FAKE, weight=FAKE, decay=1.0, stride=100, ws=None, max_len=100):
    return api.lib().verify_accumulate_weight_dense(_ref(shape), _ref(mod), q, FAKE, max_len, FAKE, FAKE, FAKE, lse,
                                                    decay, weight, stride, ws, None)


def test_weight_arguments():
    assert _weight(None) == BAD
    assert _weight(_shape(T=65)) == UNSUPPORTED
    assert _weight(_shape(D=96)) == UNSUPPORTED
    assert _weight(_shape(dtype=2)) == UNSUPPORTED
    assert _weight(_shape(B=300)) == UNSUPPORTED
    assert _weight(_shape(), q=None) == BAD
    assert _weight(_shape(), q=FAKE + 8) == BAD
    assert _weight(_shape(), lse=None) == BAD
    assert _weight(_shape(), weight=FAKE + 2) == BAD
    for decay in (-0.1, 1.5, float("nan")):
        assert _weight(_shape(), decay=decay) == BAD
    assert _weight(_shape(), stride=0) == BAD
    assert _weight(_shape(), max_len=0) == BAD
    assert _weight(_shape(), ws=FAKE + 16) == WORKSPACE
    paged = api.lib().verify_accumulate_weight_paged
    for pages, size, table, per in [(10, 12, FAKE, 4), (10, 2048, FAKE, 4), (0, 16, FAKE, 4), (10, 16, None, 4),
                                    (10, 16, FAKE, 0), (10, 1024, FAKE, 1 << 20)]:
        assert paged(_ref(_shape()), None, FAKE, FAKE, pages, size, table, per, FAKE, FAKE, FAKE, FAKE, 1.0, FAKE, 100,
                     None, None) == BAD


def _evict(shape, k=FAKE, idx=FAKE, m=16, weight=FAKE, stride=100, out=FAKE + 64, scratch=FAKE, nbytes=1 << 30,
           ws=None, max_len=100):
    return api.lib().verify_evict_kv_dense(_ref(shape), k, FAKE, max_len, FAKE, idx, FAKE, m, weight, stride, out,
                                           scratch, nbytes, ws, None)


def test_evict_arguments():
    assert _evict(None) == BAD
    assert _evict(_shape(B=0)) == BAD
    assert _evict(_shape(B=300)) == UNSUPPORTED
    assert _evict(_shape(D=4)) == UNSUPPORTED
    assert _evict(_shape(D=1024)) == UNSUPPORTED
    assert _evict(_shape(dtype=5)) == BAD
    assert _evict(_shape(), k=None) == BAD
    assert _evict(_shape(), k=FAKE + 8) == BAD
    assert _evict(_shape(), idx=None) == BAD
    assert _evict(_shape(), m=0) == BAD
    assert _evict(_shape(), weight=FAKE + 2) == BAD
    assert _evict(_shape(), stride=0) == BAD
    assert _evict(_shape(), out=None) == BAD
    assert _evict(_shape(), out=FAKE) == BAD  # seqlens itself
    assert _evict(_shape(), scratch=None) == WORKSPACE
    assert _evict(_shape(), scratch=FAKE + 8) == WORKSPACE
    assert _evict(_shape(), nbytes=8) == WORKSPACE
    assert _evict(_shape(), ws=FAKE + 8) == WORKSPACE
    assert _evict(_shape(), max_len=0) == BAD
    assert api.lib().verify_evict_kv_scratch_size(0, 1, 1) == 0
    assert api.lib().verify_evict_kv_scratch_size(1, 1, 0) == 0
    assert api.lib().verify_evict_kv_scratch_size(1000, 1000, 10) == 0
    assert api.lib().verify_evict_kv_scratch_size(4, 8, 8192) >= 256


def test_python_entry_points_refuse_cpu_tensors():
    q, k = torch.zeros(1, 2, 2, 64), torch.zeros(1, 8, 1, 64)
    L, lse, w = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 2), torch.zeros(1, 1, 8)
    idx = torch.zeros(1, 1, 4, dtype=torch.int32)
    for call in (lambda: va.verify_attn_dense_mod(q, k, k, L, va.ScoreMod()),
                 lambda: va.verify_attn_paged_mod(q, k, k, idx[0], L, va.ScoreMod()),
                 lambda: va.verify_accumulate_weight_dense(q, k, L, lse, w),
                 lambda: va.verify_accumulate_weight_paged(q, k, idx[0], L, lse, w),
                 lambda: va.verify_evict_kv_dense(k, k, L, idx, idx[:, :, 0]),
                 lambda: va.verify_evict_kv_paged(k, k, idx[0], L, idx, idx[:, :, 0])):
        with pytest.raises(ValueError, match="GPU"):
            call()
