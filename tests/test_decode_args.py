"""Refusals of the decode-step operators, and their host-side tables.  No GPU:
every call below is refused before anything is launched."""

import ctypes
import math

import pytest

import memory_bound_gemv_gb300 as mbg
from memory_bound_gemv_gb300 import decode

torch = pytest.importorskip("torch")

FAKE = 0x10000  # never dereferenced


def kv(**change):
    s = decode._KvStruct(FAKE, FAKE, (16 * 2 * 64, 2 * 64, 64), (16 * 2 * 64, 2 * 64, 64), FAKE, 8, 100, FAKE, FAKE,
                         decode.ELEM_F16, 16, 8, 4, 2, 64)
    for k, v in change.items():
        setattr(s, k, v)
    return s


def at(s):
    return ctypes.addressof(s)


TWO = (128, 64)
NEG = (-1, 64)


def attn(s, q=FAKE, qs=TWO, lengths=FAKE, out=FAKE, os=TWO, heads=8, scale=1.0, window=0, lse=0, sums=0, ws=FAKE,
         n=1 << 40):
    args = decode._ATTN.pack(q, *qs, out, *os, lengths, lse, sums, ws, n, heads, window, scale)
    return mbg.lib().gemv_attn_paged(at(s), args, None)


def rope(s=None, elem=0, q=FAKE, qs=TWO, k=FAKE, ks=TWO, v=FAKE, vs=TWO, out=FAKE, os=TWO, tokens=4, heads=8,
         pos=FAKE, ps=4, axes=1, slots=FAKE, seq=0, stamps=0, turns=FAKE, axis=FAKE, rot=64, pairs=0):
    args = decode._ROPE.pack(q, *qs, k, *ks, v, *vs, out, *os, pos, ps, slots, seq, stamps, turns, axis, elem, tokens,
                             heads, axes, rot, pairs)
    return mbg.lib().gemv_rope_append(at(s or kv()), args, None)


BAD_CACHES = [(dict(elem=0), 1), (dict(elem=7), 1), (dict(batch=-1), 1), (dict(kv_heads=0), 1), (dict(head_dim=0), 1),
              (dict(page_size=0), 1), (dict(max_pages=-1), 1), (dict(num_pages=-1), 1), (dict(table_stride=-8), 1),
              (dict(head_dim=257), 3), (dict(page_size=1 << 20, max_pages=1 << 20), 3), (dict(batch=65536), 3),
              (dict(num_pages=1 << 31), 3), (dict(k=None), 1), (dict(v=None), 1), (dict(page_table=None), 1),
              (dict(k=FAKE + 1), 2), (dict(page_table=FAKE + 2), 2), (dict(scores=FAKE + 2), 2),
              (dict(stamps=FAKE + 1), 2)]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_every_call_checks_the_cache(change, status):
    L, s = mbg.lib(), kv(**change)
    assert attn(s) == status
    assert L.gemv_kv_evict_plan(at(s), FAKE, 64, 0, 0, FAKE, 64, FAKE, None) == status
    assert L.gemv_kv_evict_apply(at(s), FAKE, 64, FAKE, FAKE, 64, None) == status
    assert rope(s) == status


def test_attn_refusals():
    s = kv()
    for change in (dict(q=0), dict(lengths=0), dict(out=0), dict(ws=0), dict(heads=0), dict(heads=7),
                   dict(window=-1), dict(qs=NEG), dict(os=NEG), dict(n=16)):
        assert attn(s, **change) == mbg.ERR_INVALID_VALUE, change
    for change in (dict(q=FAKE + 1), dict(out=FAKE + 1), dict(lengths=FAKE + 2), dict(lse=FAKE + 2),
                   dict(sums=FAKE + 1), dict(ws=FAKE + 16)):
        assert attn(s, **change) == mbg.ERR_MISALIGNED, change
    assert attn(kv(scores=None), sums=FAKE) == mbg.ERR_INVALID_VALUE
    assert attn(kv(batch=0)) == mbg.OK
    assert mbg.lib().gemv_attn_paged(at(kv()), None, None) == mbg.ERR_INVALID_VALUE
    assert mbg.lib().gemv_attn_paged(None, bytes(decode._ATTN.size), None) == mbg.ERR_INVALID_VALUE


def test_attn_workspace_sizes():
    L = mbg.lib()
    need = L.gemv_attn_paged_workspace(at(kv()), 8, 0)
    assert need > 0 and need % 256 == 0
    # the logits of every slot come with the weights: 4 heads per cached head
    assert L.gemv_attn_paged_workspace(at(kv()), 8, 1) >= need + 4 * 2 * 128 * 4 * 4
    assert attn(kv(), n=need - 1) == mbg.ERR_INVALID_VALUE
    assert L.gemv_attn_paged_workspace(at(kv()), 7, 0) == 0
    assert L.gemv_attn_paged_workspace(at(kv(head_dim=300)), 8, 0) == 0
    assert L.gemv_attn_paged_workspace(None, 8, 0) == 0


def test_evict_refusals():
    L, s = mbg.lib(), kv()

    def plan(s=s, lengths=FAKE, keep=64, sinks=0, recent=0, moves=FAKE, most=64, counts=FAKE):
        return L.gemv_kv_evict_plan(at(s), lengths, keep, sinks, recent, moves, most, counts, None)

    for change in (dict(keep=0), dict(sinks=-1), dict(recent=-1), dict(most=-1), dict(most=63), dict(lengths=None),
                   dict(moves=None), dict(counts=None), dict(s=kv(scores=None)), dict(s=kv(stamps=None))):
        assert plan(**change) == mbg.ERR_INVALID_VALUE, change
    for change in (dict(lengths=FAKE + 1), dict(moves=FAKE + 4), dict(counts=FAKE + 2)):
        assert plan(**change) == mbg.ERR_MISALIGNED, change
    assert plan(s=kv(batch=0)) == mbg.OK

    def apply(s=s, moves=FAKE, most=64, counts=FAKE, lengths=FAKE, keep=64):
        return L.gemv_kv_evict_apply(at(s), moves, most, counts, lengths, keep, None)

    for change in (dict(moves=None), dict(most=-1), dict(counts=None), dict(keep=0)):
        assert apply(**change) == mbg.ERR_INVALID_VALUE, change
    for change in (dict(moves=FAKE + 4), dict(counts=FAKE + 1), dict(lengths=FAKE + 2)):
        assert apply(**change) == mbg.ERR_MISALIGNED, change
    assert apply(s=kv(batch=0)) == mbg.OK


def test_rope_refusals():
    for change in (dict(elem=2), dict(qs=NEG), dict(ks=NEG), dict(vs=NEG), dict(os=NEG), dict(tokens=-1),
                   dict(heads=-1), dict(axes=0), dict(rot=63), dict(rot=66), dict(rot=-2), dict(ps=-1), dict(tokens=5),
                   dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(pos=0), dict(slots=0), dict(turns=0),
                   dict(axis=0)):
        assert rope(**change) == mbg.ERR_INVALID_VALUE, change
    for change in (dict(q=FAKE + 2), dict(k=FAKE + 1), dict(v=FAKE + 2), dict(out=FAKE + 1), dict(pos=FAKE + 2),
                   dict(slots=FAKE + 1), dict(seq=FAKE + 2), dict(stamps=FAKE + 1), dict(turns=FAKE + 4)):
        assert rope(**change) == mbg.ERR_MISALIGNED, change
    assert rope(tokens=0) == mbg.OK
    assert mbg.lib().gemv_rope_append(at(kv()), None, None) == mbg.ERR_INVALID_VALUE


def test_norm_refusals():
    L = mbg.lib()
    names = ("y", "x", "gate", "post_weight", "pre_weight", "pre_bias", "out", "h")

    def norm(rows=3, width=64, flags=2, **change):
        ops = {n: (FAKE, 64, 1) for n in names}
        ops.update(change)
        flat = [v for n in names for v in ops[n]]
        return L.gemv_norm_residual(decode._NORM.pack(*flat, rows, width, 1.0, 1e-6, flags), None)

    assert norm(rows=-1) == norm(width=-1) == norm(flags=8) == mbg.ERR_INVALID_VALUE
    assert norm(rows=0) == norm(width=0) == mbg.OK
    for n in ("y", "x", "out"):
        assert norm(**{n: (0, 64, 1)}) == mbg.ERR_INVALID_VALUE, n
    for n in names:
        assert norm(**{n: (FAKE, 64, 3)}) == mbg.ERR_INVALID_VALUE, n
        assert norm(**{n: (FAKE, -64, 1)}) == mbg.ERR_INVALID_VALUE, n
        if n not in ("x", "out"):  # these two share a type
            assert norm(**{n: (FAKE + 2, 64, 0)}) == mbg.ERR_MISALIGNED, n
    assert norm(out=(FAKE, 64, 0)) == mbg.ERR_INVALID_VALUE  # not x's type
    assert norm(out=(FAKE, 0, 1)) == norm(h=(FAKE, 63, 1)) == mbg.ERR_INVALID_VALUE  # written rows overlap
    assert norm(rows=1 << 31) == norm(width=(1 << 24) + 1, out=(FAKE, 1 << 30, 1), h=(FAKE, 1 << 30, 1)) == 3
    assert L.gemv_norm_residual(None, None) == mbg.ERR_INVALID_VALUE


def test_struct_layouts_match():
    """The packed arguments and the cache structure have the sizes of C's structures on a 64-bit machine."""
    assert decode._NORM.size == 8 * 24 + 2 * 8 + 3 * 4 + 4
    assert decode._ATTN.size == 2 * 24 + 5 * 8 + 3 * 4 + 4
    assert decode._ROPE.size == 4 * 24 + 7 * 8 + 6 * 4
    assert ctypes.sizeof(decode._KvStruct) == 2 * 8 + 6 * 8 + 5 * 8 + 6 * 4


def test_binding_refuses_cpu_tensors():
    h = torch.float16
    with pytest.raises(ValueError):
        mbg.PagedKV(torch.zeros(4, 16, 2, 64, dtype=h), torch.zeros(4, 16, 2, 64, dtype=h),
                    torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        mbg.PagedKV(torch.zeros(4, 16, 2, 64), torch.zeros(4, 16, 2, 64), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        mbg.PagedKV(torch.zeros(4, 64, dtype=h), torch.zeros(4, 64, dtype=h), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        mbg.gemv_norm_residual(torch.zeros(2, 8), torch.zeros(2, 8))
    with pytest.raises(ValueError):
        mbg.gemv_norm_residual(torch.zeros(2, 8), torch.zeros(2, 8), kind="group")
    with pytest.raises(ValueError):
        mbg.gemv_norm_residual(torch.zeros(2, 8), torch.zeros(2, 8), post_weight=torch.zeros(8))


def test_rope_table():
    t = mbg.RopeTable(128, sections=[16, 24, 24], theta=10000.0, device="cpu")
    assert t.axes == 3 and t.axis.tolist() == [0] * 16 + [1] * 24 + [2] * 24
    for i in (0, 1, 20, 63):
        f = 10000.0 ** (-2.0 * i / 128)
        steps = f / (2 * math.pi) * 2.0 ** 64
        # half a step of the fixed point, and the quotient's and its constant's roundings in 64 bits
        assert abs(t.turns[i].item() % (1 << 64) - steps) <= 0.5 + 4 * 2.0 ** -53 * steps
    # a product with a far position wraps as the angle does
    i, pos = 5, 1_999_993
    turns = (t.turns[i].item() * pos) % (1 << 64) / 2.0 ** 64
    exact = math.fmod(pos * 10000.0 ** (-2.0 * i / 128) / (2 * math.pi), 1.0)
    assert abs(turns - exact) < 1e-9
    p = mbg.RopeTable(16, sections=[2, 6], theta=100.0, per_axis=True, device="cpu")
    f = [100.0 ** (-j / 2) for j in range(2)] + [100.0 ** (-j / 6) for j in range(6)]
    got = [(v % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for v in p.turns.tolist()]
    assert max(abs(a - b) for a, b in zip(f, got)) < 1e-15
    for bad in (dict(rot_dim=7), dict(rot_dim=8, sections=[3]), dict(rot_dim=8, sections=[5, -1]),
                dict(rot_dim=8, sections=[]), dict(rot_dim=8, theta=0.0), dict(rot_dim=8, frequencies=[1.0]),
                dict(rot_dim=4, frequencies=[1.0, 7.0]), dict(rot_dim=4, frequencies=[1.0, -1.0])):
        with pytest.raises(ValueError):
            mbg.RopeTable(device="cpu", **bad)
