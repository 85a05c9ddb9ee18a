"""Refusals at the limits of the decode-step operators.  No GPU: nothing below is launched."""

import ctypes

import pytest

import memory_bound_gemv_gb300 as mbg
from memory_bound_gemv_gb300 import decode

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("shape", [(4, 16, 0, 64), (4, 0, 2, 64), (4, 16, 2, 0)])
def test_caches_without_heads_slots_or_elements_are_refused(shape):
    """A count of 0 heads would divide by zero in the compiled checks, which ends the process."""
    k, table = torch.zeros(shape, dtype=torch.float16), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="pages need slots, heads and elements"):
        mbg.PagedKV(k, k, table)


FAKE = 0x10000  # never dereferenced


@pytest.mark.parametrize("dim,heads", [(64, 2 ** 31 - 2), (64, 2 ** 25), (1, 2 ** 31 - 2), (256, 2 ** 23)])
def test_more_heads_or_tokens_than_32_bits_count_are_refused(dim, heads):
    s = decode._KvStruct(FAKE, FAKE, (32 * dim, 2 * dim, dim), (32 * dim, 2 * dim, dim), FAKE, 8, 100, FAKE, FAKE,
                         decode.ELEM_F16, 16, 8, 4, 2, dim)
    L, at = mbg.lib(), ctypes.addressof(s)
    unsupported = 3
    assert L.gemv_attn_paged_workspace(at, heads, 0) == 0 and L.gemv_attn_paged_workspace(at, heads, 1) == 0
    call = decode._ATTN.pack(FAKE, 0, dim, FAKE, 0, dim, FAKE, 0, 0, FAKE, 1 << 60, heads, 0, 1.0)
    assert L.gemv_attn_paged(at, call, None) == unsupported

    def rope(heads, tokens):
        return L.gemv_rope_append(at, decode._ROPE.pack(
            FAKE, 0, dim, FAKE, 0, dim, FAKE, 0, dim, FAKE, 0, dim, FAKE, 0, FAKE, FAKE, 0, FAKE, FAKE, 1, tokens, heads, 1,
            0, 0), None)

    assert rope(heads, 4) == rope(8, 2 ** 31 - 1) == rope(8, 2 ** 31 - 2 ** 20) == unsupported
