"""Which strides of an output the norm with rotation takes: those that put every row in a
place of its own.  (Every call here is refused for its weights at the latest, before
anything touches a device.)"""
import itertools

import pytest

from speculative_decoding_verification_masked_gb300 import api
from tests.test_quant_host import BAD, FAKE, _norm, _rows, _shape


def taken(B, T, heads, D, batch, token):
    """Whether an output with these strides is refused for its rows."""
    assert _norm(_shape(B=B, T=T, Hq=heads, Hkv=1, D=D), q_out=_rows(batch=batch, token=token), qw=FAKE + 2) == BAD
    text = api.lib().verify_attn_last_error().decode()
    assert "rows in one place" in text or "weights" in text, text
    return "weights" in text


@pytest.mark.parametrize("B,T", [(1, 1), (1, 5), (4, 1), (2, 2), (3, 5), (7, 4)])
def test_strides_whose_rows_are_apart(B, T):
    """Against every pair of rows: one sequence after the other, one token after the other,
    with room left and with none."""
    D, heads = 16, 2
    row = heads * D
    steps = sorted({0, 8, row - 8, row, row + 8, 2 * row} | {n * s + d for n in (B - 1, B, T - 1, T) for s in (row, row + 8)
                                                           for d in (0, row - 8, row, row + 8)})
    for batch, token in itertools.product(steps, steps):
        at = sorted({(b, t): b * batch + t * token for b in range(B) for t in range(T)}.values())
        apart = all(y - x >= row for x, y in zip(at, at[1:]))
        nested = (T == 1 or token >= row) and (B == 1 or batch >= row) and (
            B == 1 or T == 1 or batch >= (T - 1) * token + row or token >= (B - 1) * batch + row)
        assert taken(B, T, heads, D, batch, token) == nested
        assert apart or not nested
