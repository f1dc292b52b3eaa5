"""CPU checks of how long a row of the table kda_attn_decode takes: its kernels count tokens, and runs of up to 256 of them, in
32 bits.  Nothing is launched where a call is refused; no call that is not refused is made."""
import ctypes

import pytest

from test_attn_abi import DEC, _lib

MOST = 2 ** 31 - 512


def _plan(width, pt):
    n = ctypes.c_size_t(0)
    return _lib().kda_attn_decode_plan(2, pt, width, 1, 1, 8, 8, 64, 64, ctypes.byref(n))


@pytest.mark.parametrize("pt", [32, 64, 128])
def test_rows_of_nearly_2_31_tokens_are_refused(pt):
    for width in range(MOST // pt + 1, 2 ** 31 // pt):
        assert width * pt < 2 ** 31
        assert _plan(width, pt) == 2
    for width in (MOST // pt + 1, 2 ** 31 // pt - 1):
        assert _lib().kda_attn_decode(*{**DEC, "R": 1, "W": width, "pt": pt, "B": 1, "K": 1, "rows": None}.values(), None) == 2


def test_rows_below_are_planned():
    assert [_plan(MOST // pt, pt) for pt in (32, 64, 128)] == [0, 0, 0]
    assert _plan(2 ** 26, 16) == 0
