"""Slots whose page does not exist are left out of the attention of many tokens, as out of the one-token attention.

The reference is the definition in 64 bits over the other slots; tolerances as in test_gpu_serve_attn."""

import pytest

import memory_bound_gemv_gb300 as mbg
from test_gpu_decode import BF16, F16, close, make_cache, no_device_error, normal, rows_of  # noqa: F401
from test_gpu_serve_attn import attend, hidden_of, ints, shared_cache

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FRESH, LENGTHS = [200, 1, 40], [420, 300, 40]


def prompt_without(cache, lost, fresh, lengths, group, window, sinks, rows=None):
    """lost: (sequence, table entry, what it becomes).  Attends before its entries are lost (for the reference) and after."""
    hq, d, page = cache.kv_heads * group, cache.head_dim, cache.page_size
    starts = [0]
    for f in fresh:
        starts.append(starts[-1] + f)
    q = normal(4, (starts[-1], hq, d), cache.dtype, 1.5)
    want = []
    for b, n in enumerate(lengths):
        k, v = rows_of(cache, b, list(range(n)))
        m = fresh[b]
        hid = hidden_of(torch.arange(n - m + 1, n + 1, device="cuda"), n, window, sinks)
        for s, entry, _ in lost:
            if s == b:
                hid[:, entry * page:(entry + 1) * page] = True
        want.append(attend(q[starts[b]:starts[b + 1]], k, v, hid, d ** -0.5, cache.dtype))
    for b, entry, what in lost:
        cache.page_table[b, entry] = what
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = mbg.gemv_attn_prompt(cache, q, ints(starts), ints(lengths), window=window, sinks=sinks, lse=lse)
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    for b, (ref, tol, rl, lt) in enumerate(want):
        close(out[starts[b]:starts[b + 1]], ref, tol, f"out of {b}")
        close(lse[starts[b]:starts[b + 1]], rl, lt, f"lse of {b}")
    return out


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hk,group,dim,page,window,sinks,shift", [
    (2, 4, 128, 16, 0, 0, 0), (1, 2, 64, 8, 0, 0, 0), (2, 1, 80, 24, 150, 40, 0), (1, 12, 64, 7, 0, 0, 0), (1, 3, 128, 1, 0, 0, 0),
    (2, 2, 256, 16, 0, 0, 0), (1, 3, 192, 32, 120, 30, 0), (1, 2, 128, 128, 0, 0, 0), (1, 2, 40, 16, 0, 0, 0), (1, 3, 200, 7, 0, 0, 0),
    (2, 2, 77, 5, 0, 0, 1)])
def test_prompt_leaves_out_slots_without_a_page(dtype, hk, group, dim, page, window, sinks, shift):
    cache = make_cache(21, LENGTHS, hk, dim, page, dtype, shift=shift)
    lost = [(0, 0, -1), (0, 200 // page, 1 << 20), (0, 419 // page, -1), (1, 299 // page, cache.k.shape[0])]
    prompt_without(cache, lost, FRESH, LENGTHS, group, window, sinks)


def test_prompt_with_no_page_at_all():
    cache = make_cache(22, [100, 50], 1, 64, 16, F16)
    cache.page_table[0] = -1
    q = normal(5, (80, 4, 64), F16)
    lse = torch.zeros(80, 4, device="cuda")
    out = mbg.gemv_attn_prompt(cache, q, ints([0, 60, 80]), ints([100, 50]), lse=lse)
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    assert (out[:60] == 0).all() and (lse[:60] == -float("inf")).all()
    assert out[60:].isfinite().all() and lse[60:].isfinite().all()


@pytest.mark.parametrize("dim,group", [(64, 4), (128, 4), (256, 2)])
def test_long_prompt_cut_between_blocks(dim, group):
    """Holes in parts of blocks, far apart."""
    fresh, lengths = [300, 2], [4000, 9000]
    cache = make_cache(23, lengths, 2, dim, 16, BF16)
    prompt_without(cache, [(0, 3, -1), (0, 100, -7), (0, 101, -1), (1, 500, 1 << 30), (1, 9, -1)], fresh, lengths, group, 0, 0)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hk,group,dim,page,prefix", [(2, 4, 128, 16, 300), (1, 3, 64, 7, 300), (1, 2, 256, 32, 3000), (2, 1, 80, 24, 1000)])
def test_prefix_leaves_out_slots_without_a_page(hk, group, dim, page, prefix, dtype):
    """In the prefix, and behind it."""
    lengths = [prefix + 5, prefix + 100, prefix // 2, prefix + 260]
    cache = shared_cache(24, lengths, prefix, hk, dim, page, dtype)
    q = normal(6, (4, hk * group, dim), dtype, 1.5)
    lost = [2, 100 // page, prefix // page - 1]
    own = (prefix + 150) // page
    want = []
    for b, n in enumerate(lengths):
        k, v = rows_of(cache, 0, list(range(min(n, prefix))))
        if n > prefix:
            k, v = (torch.cat(x) for x in zip((k, v), rows_of(cache, b, list(range(prefix, n)))))
        hid = hidden_of([n], n, 0, 0)
        for e in lost + [own] * (b == 3):
            hid[:, e * page:(e + 1) * page] = True
        want.append(attend(q[b:b + 1], k, v, hid, dim ** -0.5, dtype))
    for e in lost:
        cache.page_table[0, e] = -1
    cache.page_table[3, own] = 1 << 24
    lse = torch.full((4, hk * group), 7.0, device="cuda")
    out = mbg.gemv_attn_shared(cache, q, ints(lengths), ints([prefix]), lse=lse)
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    for b, (ref, tol, rl, lt) in enumerate(want):
        close(out[b:b + 1], ref, tol, f"out of {b}")
        close(lse[b:b + 1], rl, lt, f"lse of {b}")


def test_holes_and_infinities_together():
    """A row computed again alone leaves out the same slots."""
    cache = make_cache(25, [700], 1, 128, 16, F16)
    q = normal(7, (100, 2, 128), F16)
    k, v = rows_of(cache, 0, list(range(700)))
    hid = hidden_of(torch.arange(601, 701, device="cuda"), 700, 0, 0)
    hid[:, 160:176] = True
    ref, tol, rl, lt = attend(q, k, v, hid, 128 ** -0.5, F16)
    cache.v[int(cache.page_table[0, 699 // 16]), 699 % 16] = float("inf")  # the last token's own
    cache.page_table[0, 10] = -1
    lse = torch.full((100, 2), 7.0, device="cuda")
    out = mbg.gemv_attn_prompt(cache, q, ints([0, 100]), ints([700]), lse=lse)
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    close(out[:-1], ref[:-1], tol[:-1])
    close(lse, rl, lt)
    assert (out[-1] == float("inf")).all()
