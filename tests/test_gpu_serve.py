"""Page tables and slot maps, normed rotary append, and attention of single tokens with sinks, against plain
definitions in 64 bits.  Tolerances as in test_gpu_decode.

Norms of heads: the squares' sum is off by at most 20 roundings, half of which
the root leaves; the root itself is off by 2 ulp and each of the three products by half a step: below
2^-20 of the normed magnitude together, beside the turn's own 2^-20.
"""

import math

import numpy as np
import pytest

import memory_bound_gemv_gb300 as mbg
from test_gpu_decode import (BF16, F16, F32, HALF_STEP, TINY, attn_reference, close, make_cache, no_device_error,  # noqa: F401
                             normal, rope_reference, rows_of)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# --------------------------------------------------------------------------- pages and slots

def assign_reference(lengths, fresh, table, ring, state, page, room, shared=None):
    """The definition, request by request; lists in, lists out (table and ring are changed)."""
    front, count = state
    size, width = len(ring), len(table[0]) if table else 0
    returned, tokens, out = [], [], list(lengths)
    starts, dry, full, wanted, left = [0], False, False, 0, count
    for b, (n, f) in enumerate(zip(lengths, fresh)):
        have = -(-n // page)
        if f < 0:
            returned += table[b][(shared[b] // page if shared else 0):have]
            out[b] = 0
        elif n + f <= width * page:
            need = -(-(n + f) // page) - have
            if need:
                left -= need
                dry = dry or left < 0
            f = 0 if need and dry else f
            wanted += f
            full = full or wanted > room
            if f and not full:
                for i in range(need):
                    table[b][have + i] = ring[front % size]
                    front, count = front + 1, count - 1
                tokens += [(n + i, b) for i in range(f)]
                out[b] = n + f
        starts.append(len(tokens))
    end = front + count
    for i, p in enumerate(returned):
        ring[(end + i) % size] = p
    tokens += [(-1, 0)] * (room - len(tokens))
    return starts, [t[0] for t in tokens], [t[1] for t in tokens], out, [front % size if size else 0, count + len(returned)]


def check_assign(lengths, fresh, page, width, free, front, room, shared=None, spare=3, in_place=False, seed=0):
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lengths]
    total = sum(need) + free + spare
    order = rng.permutation(total).tolist()
    table = [[-1] * width for _ in lengths]
    for b, n in enumerate(need):
        table[b][:n] = [order.pop() for _ in range(n)]
    ring = [-1] * total
    for i in range(free):
        ring[(front + i) % total] = order.pop()
    kv = torch.zeros(total, page, 1, 1, dtype=F16, device="cuda")
    shape = (len(lengths), width)
    cache = mbg.PagedKV(kv, kv, ints(table).view(shape))
    pool = mbg.PagePool(ring=ints(ring), state=ints([front, free]))
    n, f = ints(lengths), ints(fresh)
    extra = {} if in_place else dict(lengths_out=torch.full_like(n, 77), state_out=ints([5, 5]))
    got = mbg.gemv_kv_assign(cache, pool, n, f, starts=torch.full((len(lengths) + 1,), 9, dtype=torch.int32, device="cuda"),
                             slots=torch.full((room,), 9, dtype=torch.int32, device="cuda"),
                             seq=torch.full((room,), 9, dtype=torch.int32, device="cuda"),
                             shared=None if shared is None else ints(shared), **extra)
    starts, slots, seq, out, state = assign_reference(lengths, fresh, table, ring, [front, free], page, room, shared)
    assert [x.tolist() for x in got] == [starts, slots, seq]
    assert cache.page_table.tolist() == table and pool.ring.tolist() == ring
    assert extra.get("lengths_out", n).tolist() == out
    assert extra.get("state_out", pool.state).tolist() == state
    if not in_place:
        assert n.tolist() == lengths and pool.state.tolist() == [front, free]
    return starts


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [1, 7, 16])
def test_assign_a_step(page, in_place):
    rng = np.random.default_rng(page)
    for batch in (1, 31, 32, 33, 300):
        lengths = rng.integers(0, 100, batch).tolist()
        fresh = rng.choice([-1, 0, 1, 1, 1], batch).tolist()
        check_assign(lengths, fresh, page, 110 // page + 2, 400, 123, batch + 5, in_place=in_place, seed=batch)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,longest,page,room", [(1, 0, 16, 20000), (3, 9000, 16, 30011), (700, 90, 5, 70000),
                                                     (1024, 30, 16, 40000), (1025, 30, 16, 40000), (2500, 12, 3, 33000)])
def test_assign_prompts(batch, longest, page, room, in_place):
    """Slot maps long enough for several blocks, more requests than one has threads, shared pages."""
    rng = np.random.default_rng(batch)
    lengths = rng.integers(0, longest + 1, batch).tolist()
    fresh = np.where(rng.random(batch) < 0.3, -1, rng.integers(0, max(2, 24000 // batch), batch)).tolist()
    shared = rng.integers(0, longest + 1, batch).tolist()
    width = (longest + 24000 // batch) // page + 2
    check_assign(lengths, fresh, page, width, 26000 // page + batch, 11, room, shared, in_place=in_place)


def test_assign_nothing_left():
    """Requests that need pages wait once they are gone; those that need none go on; so do those that are over."""
    check_assign([16, 15, 16, 0, 3, 32], [1, 1, 1, 40, 1, -1], 16, 4, 1, 0, 50)
    check_assign([16, 15, 16, 0, 3, 32], [1, 1, 1, 40, 1, -1], 16, 4, 0, 0, 50, spare=0)
    check_assign([16, 16, 16, 16], [1, 17, 1, 0], 16, 4, 3, 2, 50)
    # the slot map is full: the request that does not fit waits, and those behind it
    assert check_assign([5, 6, 7, 40], [3, 4, 1, -1], 16, 4, 9, 2, 6) == [0, 3, 3, 3, 3]
    assert check_assign([5, 6, 7], [3, 3, 0], 16, 4, 9, 2, 6) == [0, 3, 6, 6]
    check_assign([5] * 1500, [2] * 1500, 8, 3, 100, 0, 2100)


def test_assign_empty():
    check_assign([0], [0], 16, 1, 0, 0, 0)
    check_assign([16, 0], [-5, -1], 16, 2, 0, 0, 3, spare=0)
    cache = mbg.PagedKV(torch.zeros(1, 16, 1, 1, dtype=F16, device="cuda"), torch.zeros(1, 16, 1, 1, dtype=F16, device="cuda"),
                        torch.zeros(0, 4, dtype=torch.int32, device="cuda"))
    pool = mbg.PagePool(3)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    starts, slots, seq = mbg.gemv_kv_assign(cache, pool, none, none, tokens=5)
    assert starts.tolist() == [0] and slots.tolist() == [-1] * 5 and seq.tolist() == [0] * 5
    assert pool.state.tolist() == [0, 3]


def test_assign_reports_what_is_out_of_range():
    def call(lengths, fresh, state, ring, room=8, width=2):
        kv = torch.zeros(6, 4, 1, 1, dtype=F16, device="cuda")
        cache = mbg.PagedKV(kv, kv, torch.full((len(lengths), width), 5, dtype=torch.int32, device="cuda"))
        pool = mbg.PagePool(ring=ints(ring), state=ints(state))
        n = ints(lengths)
        starts, slots, seq = mbg.gemv_kv_assign(cache, pool, n, ints(fresh), tokens=room)
        assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
        return starts.tolist(), n.tolist(), pool.state.tolist(), cache.page_table.tolist(), pool.ring.tolist()

    starts, n, state, _, _ = call([-1, 3, 9, 4], [1, 1, 1, 5], [0, 4], [0, 1, 2, 3])  # below 0, and beyond the capacity of 8
    assert starts == [0, 0, 1, 1, 1] and n == [0, 4, 8, 4] and state == [0, 4]
    starts, n, state, table, _ = call([4, 0], [1, 1], [0, 2], [7, -3])  # pages that do not exist
    assert starts == [0, 1, 2] and table == [[5, -1], [-1, 5]]
    for state in ([-1, 2], [4, 1], [0, 5], [0, -1]):
        starts, n, after, _, ring = call([4, 3, 4], [1, 1, -1], state, [0, 1, 2, 3])
        assert starts == [0, 0, 1, 1] and n == [4, 4, 0] and after == state and ring == [0, 1, 2, 3]
    # more pages come back than the ring has places for
    _, _, state, _, ring = call([8, 8], [-1, -1], [1, 1], [0, 1, 2])
    assert state == [1, 3] and ring == [5, 1, 5]


def test_assign_in_a_graph_on_another_stream():
    """A captured call goes on from step to step: lengths, pages and the pool's state change in place."""
    kv = torch.zeros(40, 4, 1, 1, dtype=F16, device="cuda")
    table = torch.full((3, 10), -1, dtype=torch.int32, device="cuda")
    cache, pool = mbg.PagedKV(kv, kv, table), mbg.PagePool(40)
    n, f = ints([0, 0, 0]), ints([5, 1, 0])
    slots, seq, starts = (torch.empty(k, dtype=torch.int32, device="cuda") for k in (16, 16, 4))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            mbg.gemv_kv_assign(cache, pool, n, f, starts, slots, seq)
        t, r, state, ln = table.tolist(), list(range(40)), [0, 40], [0, 0, 0]
        for step in ([5, 1, 0], [1, 1, 9], [1, -1, 1], [4, 2, -1], [-1, 1, 3], [1, 16, -1]):
            f.copy_(ints(step))
            g.replay()
            want = assign_reference(ln, step, t, r, state, 4, 16)
            ln, state = want[3], want[4]
            assert [starts.tolist(), slots.tolist(), seq.tolist(), n.tolist(), pool.state.tolist()] == list(want)
            assert table.tolist() == t and pool.ring.tolist() == r


# --------------------------------------------------------------------------- norms of heads with the rotation

@pytest.mark.parametrize("src", [F32, F16, BF16])
@pytest.mark.parametrize("dst,weights,unit", [(F16, F16, False), (BF16, F32, True), (BF16, None, False)])
@pytest.mark.parametrize("dim,sections,pairs,page,shift", [
    (128, [64], False, 16, 0), (128, [16, 24, 24], True, 16, 0), (64, [16], False, 24, 0), (80, [40], False, 7, 0),
    (256, [64], True, 16, 0), (256, [1], False, 16, 0), (77, [5, 6], True, 5, 0), (10, [0, 5], False, 16, 0),
    (1, [0], False, 16, 0), (128, [64], False, 16, 1)])
def test_norm_rope_append(src, dst, weights, unit, dim, sections, pairs, page, shift):
    hq, hk, counts = 5, 2, [3, 0, 40, 1]
    starts = [0, 2, 17, 63]
    lengths = [a + n for a, n in zip(starts, counts)]
    T = sum(counts)
    cache = make_cache(31, lengths, hk, dim, page, dst, shift=shift, fill=0.0)
    qkv = normal(32, (T, hq + 2 * hk, dim), src, 3.0)
    qkv[4] = 0                 # heads of zeros stay zeros
    qkv[5] *= 2.0 ** -9        # eps counts
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    seq = torch.repeat_interleave(torch.arange(4), torch.tensor(counts)).to(torch.int32).cuda()
    slots = torch.cat([torch.arange(a, a + n) for a, n in zip(starts, counts)]).to(torch.int32).cuda()
    slots[1] = -1
    positions = torch.randint(-1000, 2000000, (len(sections), T), device="cuda", dtype=torch.int32)
    w = [None, None] if weights is None else [normal(7 + i, (dim,), weights, 0.5) for i in range(2)]
    rope = mbg.RopeTable(2 * sum(sections), sections=sections, pairs=pairs)
    old = [cache.k.clone(), cache.v.clone()]
    out = mbg.gemv_rope_append(cache, q, k, v, positions, slots, rope, seq=seq, norm=True, q_weight=w[0], k_weight=w[1],
                               unit_offset=unit, eps=1e-5)
    args = (2 * sum(sections), sections, pairs)

    def reference(x, weight):
        x = x.double()
        x = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        if weight is not None:
            x = x * (weight.double() + (1.0 if unit else 0.0))
        ref, mag = rope_reference(x, positions, args)
        plain = torch.maximum(mag, x.abs())  # elements that are not turned are normed all the same
        return ref, plain * 2.0 ** -19 + ref.abs() * HALF_STEP[dst] + TINY[dst]

    close(out, *reference(q, w[0]), "q")
    put = [i for i in range(T) if int(slots[i]) >= 0]
    pages = cache.page_table[seq[put].long(), slots[put].long() // page].long()
    offs = slots[put].long() % page
    ref, tol = reference(k, w[1])
    close(cache.k[pages, offs], ref[put], tol[put], "k")
    assert torch.equal(cache.v[pages, offs], v[put].float().to(dst))
    for now, was in zip((cache.k, cache.v), old):  # nothing else has changed
        was[pages, offs] = now[pages, offs]
        assert torch.equal(now, was)
    # the same through the quick form of the checks
    again = mbg.gemv_rope_append(cache, q, k, v, positions, slots, rope, seq=seq, norm=True, q_weight=w[0], k_weight=w[1],
                                 unit_offset=unit, eps=1e-5, q_out=torch.zeros_like(out))
    assert torch.equal(again, out)


def test_norm_rope_nan_and_infinities_stay_in_their_heads():
    cache = make_cache(3, [4, 4], 2, 128, 16, F16, fill=0.0)
    x = normal(4, (2, 6, 128), F32)
    q, k, v = x[:, :2], x[:, 2:4], x[:, 4:]
    slots, rope = ints([3, 3]), mbg.RopeTable(128)
    pos = ints([[3, 9]])
    clean = mbg.gemv_rope_append(cache, q, k, v, pos, slots, rope, norm=True)
    keys = cache.k.clone()
    x[0, 0, 7], x[1, 3, 100] = math.nan, math.inf
    got = mbg.gemv_rope_append(cache, q, k, v, pos, slots, rope, norm=True)
    assert got[0, 0].isnan().all() and torch.equal(got[0, 1], clean[0, 1]) and torch.equal(got[1], clean[1])
    p = cache.page_table[1, 0].long()
    assert cache.k[p, 3, 1].isnan().any()
    keys[p, 3, 1] = cache.k[p, 3, 1]
    assert torch.equal(keys.nan_to_num(5), cache.k.nan_to_num(5))


def test_norm_rope_checks_its_arguments():
    cache = make_cache(3, [4, 4], 2, 64, 16, F16, fill=0.0)
    x = normal(4, (2, 6, 64), F32)
    args = (cache, x[:, :2], x[:, 2:4], x[:, 4:], ints([[3, 9]]), ints([3, 3]), mbg.RopeTable(64))
    for bad in (dict(q_weight=x[0, 0]), dict(unit_offset=True), dict(norm=True, q_weight=x[0, 0, :63]),
                dict(norm=True, k_weight=x[0, :1]), dict(norm=True, k_weight=torch.ones(64))):
        for out in (None, torch.empty(2, 2, 64, dtype=F16, device="cuda")):
            with pytest.raises(ValueError):
                mbg.gemv_rope_append(*args, q_out=out, **bad)
    with pytest.raises(TypeError):
        mbg.gemv_rope_append(*args, norm=True, q_weight=torch.ones(64, dtype=torch.float64, device="cuda"))


def test_assign_checks_its_arguments():
    cache = make_cache(5, [4, 4], 2, 64, 16, F16, fill=0.0)
    pool, n, fresh = mbg.PagePool(6), ints([4, 4]), ints([1, 1])
    held = dict(starts=ints([0] * 3), slots=ints([0] * 9), seq=ints([0] * 9))
    for bad in (dict(tokens=5), dict(seq=held["seq"][:8]), dict(starts=ints([0, 0])), dict(slots=held["slots"][:, None]),
                dict(shared=ints([0])), dict(lengths_out=ints([0])), dict(state_out=ints([0])), dict(seq=held["seq"].cpu()),
                dict(slots=torch.zeros(18, dtype=torch.int32, device="cuda")[::2])):
        with pytest.raises(ValueError):
            mbg.gemv_kv_assign(cache, pool, n, fresh, **{**held, **bad})
    with pytest.raises(TypeError):
        mbg.gemv_kv_assign(cache, pool, n, fresh.long(), **held)
    with pytest.raises(ValueError):
        mbg.gemv_kv_assign(cache, pool, n, fresh)  # neither slots nor tokens
    assert n.tolist() == [4, 4] and pool.state.tolist() == [0, 6]  # nothing ran
    mbg.gemv_kv_assign(cache, pool, n, fresh, tokens=9, **held)
    assert n.tolist() == [5, 5] and held["slots"].tolist() == [4, 4] + [-1] * 7


# --------------------------------------------------------------------------- single tokens with sinks

def sinks_reference(cache, q, lengths, scale, window, sinks):
    """attn_reference over copies of the sequences in which only the visible slots are left."""
    out = [torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    hk, cap = cache.kv_heads, cache.capacity
    w = [torch.zeros(len(lengths), hk, cap, dtype=torch.float64, device="cuda") for _ in range(2)]
    lse = [torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda") for _ in range(2)]
    seen = torch.zeros(len(lengths), cap, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lengths):
        at = [t for t in range(n) if not window or t >= n - window or t < sinks]
        if not at:
            continue
        k, v = rows_of(cache, b, at)
        small = mbg.PagedKV(k.contiguous()[None], v.contiguous()[None], torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
        got = attn_reference(small, q[b:b + 1], [len(at)], scale, 0)
        for i in range(2):
            out[i][b] = got[i][0]
            w[i][b][:, at] = got[2 + i][0]
            lse[i][b] = got[4 + i][0]
        seen[b, at] = True
    return out, w, lse, seen


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hk,group,dim,page,window,sinks", [
    (2, 4, 128, 16, 64, 4), (2, 1, 80, 24, 33, 1), (1, 12, 64, 8, 100, 37), (1, 20, 128, 1, 50, 16), (2, 2, 256, 16, 1, 64),
    (1, 3, 33, 5, 40, 3), (2, 4, 64, 16, 16, 200), (2, 4, 64, 64, 250, 49), (2, 4, 128, 16, 0, 4), (2, 4, 192, 16, 100, 2 ** 31 - 1)])
def test_attn_sinks(dtype, hk, group, dim, page, window, sinks):
    """Windows whose first tile is the sinks' last, sinks that reach into the window, weights of both parts."""
    lengths = [0, 1, 15, 17, 65, 66, 300, 100, 101, 116, 317]
    cache = make_cache(41, lengths, hk, dim, page, dtype, history=True)
    q = normal(42, (len(lengths), hk * group, dim), dtype, 1.5)
    scale = dim ** -0.5
    out, w, lse, seen = sinks_reference(cache, q, lengths, scale, window, sinks)
    got_lse = torch.full(q.shape[:2], 7.0, device="cuda")
    got = mbg.gemv_attn_paged(cache, q, ints(lengths), window=window, sinks=sinks, lse=got_lse)
    close(got, *out, "out")
    close(got_lse, *lse, "lse")
    sums = torch.full_like(cache.scores, -5.0)
    again = mbg.gemv_attn_paged(cache, q, ints(lengths), window=window, sinks=sinks, accumulate=True, scores_out=sums)
    assert torch.equal(again, got)
    live = seen[:, None].expand_as(sums)
    ref = torch.where(live, cache.scores.double() + w[0], -5.0)
    close(sums, ref, torch.where(live, w[1] + ref.abs() * 2.0 ** -24 * (1 + group) + w[0] * group * 2.0 ** -24, 0.0), "scores")


def test_attn_sinks_of_long_rows():
    """Rows cut over many blocks, sinks and window in one tile and far apart."""
    lengths = [30011, 3, 9000, 5001]
    cache = make_cache(43, lengths, 2, 128, 64, BF16, fill=0.0)
    q = normal(44, (4, 8, 128), BF16, 2.0)
    for window, sinks in ((20000, 4), (4990, 8), (8000, 900), (100, 3000)):
        out, _, _, _ = sinks_reference(cache, q, lengths, 128 ** -0.5, window, sinks)
        close(mbg.gemv_attn_paged(cache, q, ints(lengths), window=window, sinks=sinks), *out)


def test_attn_sinks_hidden_slots_leave_no_trace():
    """What lies between the sinks and the window is not read: NaN there changes nothing."""
    lengths = [300, 40]
    cache = make_cache(45, lengths, 2, 64, 16, F16)
    q = normal(46, (2, 4, 64), F16)
    clean = mbg.gemv_attn_paged(cache, q, ints(lengths), window=20, sinks=5)
    for b, n in enumerate(lengths):
        t = torch.arange(5, n - 20, device="cuda")
        at = cache.page_table[b, t // 16].long(), t % 16
        cache.k[at], cache.v[at] = math.nan, math.inf
    assert torch.equal(mbg.gemv_attn_paged(cache, q, ints(lengths), window=20, sinks=5), clean)
    with pytest.raises(ValueError):
        mbg.gemv_attn_paged(cache, q, ints(lengths), window=20, sinks=-1)
    with pytest.raises(ValueError):
        mbg.gemv_attn_paged(cache, q, ints(lengths), window=20, sinks=2 ** 31)
