"""Rows of queries up to 32-bit counts.  No GPU: every call below is refused before anything is launched."""

import ctypes

import pytest

import memory_bound_gemv_gb300 as mbg
from memory_bound_gemv_gb300 import decode

torch = pytest.importorskip("torch")

FAKE = 0x10000  # never dereferenced


def cache(heads):
    return decode._KvStruct(FAKE, FAKE, (16 * 8 * heads, 8 * heads, 8), (16 * 8 * heads, 8 * heads, 8), FAKE, 8, 100, 0, 0,
                            decode.ELEM_F16, 16, 8, 4, heads, 8)


@pytest.mark.parametrize("tokens,heads", [(33554431, 64), (33554429, 64), (2 ** 25 - 1, 64)])
def test_rows_that_fill_the_last_block_past_32_bits_are_refused(tokens, heads):
    """Rows are counted in blocks of 256, the next of which has to have a number as well: 2^31 - 64 rows do not fit."""
    kv = cache(1)
    at = ctypes.addressof(kv)
    assert tokens * heads < 2 ** 31 <= (tokens * heads + 255) // 256 * 256 + 256
    args = decode._PROMPT.pack(FAKE, 8 * heads, 8, FAKE, 8 * heads, 8, FAKE, FAKE, 0, FAKE, 1 << 50, tokens, heads, 0, 0, 1.0)
    assert mbg.lib().gemv_attn_prompt_workspace(at, tokens, heads) == 0
    assert mbg.lib().gemv_attn_prompt(at, args, None) == mbg.ERR_UNSUPPORTED
    assert mbg.lib().gemv_attn_prompt_workspace(at, (2 ** 31 - 2048) // heads, heads) > 0
