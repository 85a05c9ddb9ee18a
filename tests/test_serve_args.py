"""Refusals of the serving operators.  No GPU: every call below is refused before anything is launched."""

import ctypes

import pytest

import memory_bound_gemv_gb300 as mbg
from memory_bound_gemv_gb300 import decode

torch = pytest.importorskip("torch")

FAKE = 0x10000  # never dereferenced


@pytest.fixture
def kv():
    made = []

    def make(**change):
        s = decode._KvStruct(FAKE, FAKE, (16 * 2 * 64, 2 * 64, 64), (16 * 2 * 64, 2 * 64, 64), FAKE, 8, 100, FAKE, FAKE,
                             decode.ELEM_F16, 16, 8, 4, 2, 64)
        for k, v in change.items():
            setattr(s, k, v)
        made.append(s)
        return ctypes.addressof(s)

    return make


def assign(at, lengths=FAKE, fresh=FAKE, shared=0, lengths_out=FAKE, ring=FAKE, size=100, state=FAKE, state_out=FAKE,
           starts=FAKE, slots=FAKE, seq=FAKE, room=64):
    return mbg.lib().gemv_kv_assign(at, decode._ASSIGN.pack(lengths, fresh, shared, lengths_out, ring, size, state, state_out,
                                                            starts, slots, seq, room), None)


def test_assign_refusals(kv):
    for change in (dict(lengths=0), dict(fresh=0), dict(lengths_out=0), dict(ring=0), dict(size=-1), dict(state=0),
                   dict(state_out=0), dict(starts=0), dict(slots=0), dict(seq=0), dict(room=-1)):
        assert assign(kv(), **change) == mbg.ERR_INVALID_VALUE, change
    for name in ("lengths", "fresh", "shared", "lengths_out", "ring", "state", "state_out", "starts", "slots", "seq"):
        assert assign(kv(), **{name: FAKE + 2}) == mbg.ERR_MISALIGNED, name
    assert assign(kv(), room=2 ** 31 - 1) == assign(kv(), size=2 ** 31) == mbg.ERR_UNSUPPORTED
    assert assign(kv(table_stride=7)) == mbg.ERR_INVALID_VALUE  # rows of the table lie on one another
    assert assign(kv(page_table=None)) == mbg.ERR_INVALID_VALUE
    assert assign(kv(page_table=FAKE + 1)) == mbg.ERR_MISALIGNED
    assert assign(kv(batch=65536)) == assign(kv(head_dim=257)) == mbg.ERR_UNSUPPORTED
    assert mbg.lib().gemv_kv_assign(kv(), None, None) == mbg.ERR_INVALID_VALUE
    assert mbg.lib().gemv_kv_assign(None, bytes(decode._ASSIGN.size), None) == mbg.ERR_INVALID_VALUE


def test_norm_rope_refusals(kv):
    def call(q_weight=FAKE, k_weight=FAKE, q_elem=1, k_elem=1, tokens=4):
        two = (128, 64)
        args = decode._ROPE.pack(FAKE, *two, FAKE, *two, FAKE, *two, FAKE, *two, FAKE, 4, FAKE, 0, 0, FAKE, FAKE, 0, tokens,
                                 8, 1, 64, 0)
        return mbg.lib().gemv_rope_append_norm(kv(), args, decode._HEAD_NORM.pack(q_weight, k_weight, q_elem, k_elem, 0, 1e-6),
                                               None)

    assert call(q_elem=2) == call(k_elem=7) == mbg.ERR_INVALID_VALUE
    assert call(q_weight=FAKE + 1) == call(k_weight=FAKE + 2, k_elem=0) == mbg.ERR_MISALIGNED
    assert call(tokens=5) == call(tokens=-1) == mbg.ERR_INVALID_VALUE
    assert call(tokens=0) == mbg.OK
    assert mbg.lib().gemv_rope_append_norm(kv(), bytes(decode._ROPE.size), None, None) == mbg.ERR_INVALID_VALUE


def test_sinks_refusals(kv):
    args = decode._ATTN.pack(FAKE, 128, 64, FAKE, 128, 64, FAKE, 0, 0, FAKE, 1 << 40, 8, 0, 1.0)
    assert mbg.lib().gemv_attn_paged_sinks(kv(), args, -1, None) == mbg.ERR_INVALID_VALUE
    assert mbg.lib().gemv_attn_paged_sinks(kv(batch=0), args, 4, None) == mbg.OK


def test_struct_layouts_match():
    assert decode._ASSIGN.size == 12 * 8
    assert decode._HEAD_NORM.size == 2 * 8 + 4 * 4


def test_page_pool():
    for bad in (dict(), dict(pages=3, ring=torch.zeros(3, dtype=torch.int32)), dict(ring=torch.zeros(3, dtype=torch.int32)),
                dict(pages=-1), dict(pages=4, state=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            mbg.PagePool(device="cpu", **bad)
    with pytest.raises(ValueError, match="CUDA"):
        mbg.PagePool(4, device="cpu")


TWO, NEG = (128, 64), (-1, 64)


def prompt(at, q=FAKE, qs=TWO, out=FAKE, os=TWO, starts=FAKE, lengths=FAKE, lse=0, ws=FAKE, n=1 << 40, tokens=9, heads=8,
           window=0, sinks=0):
    return mbg.lib().gemv_attn_prompt(at, decode._PROMPT.pack(q, *qs, out, *os, starts, lengths, lse, ws, n, tokens, heads,
                                                              window, sinks, 1.0), None)


def test_prompt_refusals(kv):
    need = mbg.lib().gemv_attn_prompt_workspace(kv(), 9, 8)
    assert need > 0 and need % 256 == 0
    for change in (dict(q=0), dict(out=0), dict(starts=0), dict(lengths=0), dict(ws=0), dict(heads=0), dict(heads=7),
                   dict(window=-1), dict(sinks=-1), dict(tokens=-1), dict(qs=NEG), dict(os=NEG), dict(n=need - 1)):
        assert prompt(kv(), **change) == mbg.ERR_INVALID_VALUE, change
    for change in (dict(q=FAKE + 1), dict(out=FAKE + 1), dict(starts=FAKE + 2), dict(lengths=FAKE + 2), dict(lse=FAKE + 2),
                   dict(ws=FAKE + 16)):
        assert prompt(kv(), **change) == mbg.ERR_MISALIGNED, change
    for change in (dict(tokens=2 ** 31), dict(tokens=2 ** 24, heads=2 ** 8), dict(heads=2 ** 25)):
        assert prompt(kv(), **change) == mbg.ERR_UNSUPPORTED, change
        assert mbg.lib().gemv_attn_prompt_workspace(kv(), change.get("tokens", 9), change.get("heads", 8)) == 0
    assert prompt(kv(batch=0)) == prompt(kv(), tokens=0) == mbg.OK
    assert prompt(kv(elem=0)) == prompt(kv(k=None)) == mbg.ERR_INVALID_VALUE
    assert prompt(None) == mbg.lib().gemv_attn_prompt(kv(), None, None) == mbg.ERR_INVALID_VALUE
    assert mbg.lib().gemv_attn_prompt_workspace(None, 9, 8) == mbg.lib().gemv_attn_prompt_workspace(kv(), -1, 8) == 0


def shared(at, prefix=FAKE, sinks=0, q=FAKE, lengths=FAKE, heads=8, window=0, sums=0, ws=FAKE, n=1 << 40):
    args = decode._ATTN.pack(q, *TWO, FAKE, *TWO, lengths, 0, sums, ws, n, heads, window, 1.0)
    return mbg.lib().gemv_attn_shared(at, args, prefix, sinks, None)


def test_shared_refusals(kv):
    L = mbg.lib()
    need = L.gemv_attn_shared_workspace(kv(), 8)
    assert need > L.gemv_attn_paged_workspace(kv(), 8, 0)
    for change in (dict(prefix=None), dict(sinks=-1), dict(window=-1), dict(heads=7), dict(heads=0), dict(q=0),
                   dict(lengths=0), dict(ws=0), dict(sums=FAKE), dict(n=need - 1)):
        assert shared(kv(), **change) == mbg.ERR_INVALID_VALUE, change
    for change in (dict(prefix=FAKE + 2), dict(q=FAKE + 1), dict(ws=FAKE + 128)):
        assert shared(kv(), **change) == mbg.ERR_MISALIGNED, change
    assert shared(kv(batch=0)) == mbg.OK
    assert shared(kv(batch=65535), heads=2 ** 17) == mbg.ERR_UNSUPPORTED
    assert L.gemv_attn_shared_workspace(kv(batch=65535), 2 ** 17) == L.gemv_attn_shared_workspace(kv(), 7) == 0
    assert L.gemv_attn_shared(kv(), None, FAKE, 0, None) == mbg.ERR_INVALID_VALUE


def test_prompt_layout_matches():
    assert decode._PROMPT.size == 2 * 24 + 3 * 8 + 2 * 8 + 8 + 4 * 4
