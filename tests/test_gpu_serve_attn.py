"""Attention of many tokens over the paged cache, prompts and shared prefixes, against its definition in 64 bits.

Tolerances.  Scores: a sum of D exact products in FP32, each addition off by at most one step of the running sum, so
|ds| <= (D + 8) 2^-23 A with A = scale sum |q_d k_d|; a weight is then off by 2 |ds| relative, plus 2^-20
for the exponential and the sums of weights.  Weights enter the value product in two 16-bit parts, off by 2^-16 (bf16) or
2^-21 relative and 2^-35 of the row's largest (f16).  The product is a sum of n / 8 parts in FP32, each addition off by
at most one step of it, and some 40 roundings join its pieces.  Output rounding: half a step.
"""

import math

import numpy as np
import pytest

import memory_bound_gemv_gb300 as mbg
from test_gpu_decode import (BF16, F16, HALF_STEP, TINY, close, make_cache, no_device_error, normal,  # noqa: F401
                             rows_of)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def attend(q, k, v, hidden, scale, dtype):
    """One sequence: q [m, Hq, D], k and v [n, Hkv, D], hidden [m, n]; out, its bound, lse, its bound."""
    m, hq, d = q.shape
    g = hq // k.shape[1]
    n = k.shape[0]
    outs = [torch.zeros(m, hq, d, dtype=torch.float64, device="cuda") for _ in range(2)]
    lses = [torch.full((m, hq), -math.inf, dtype=torch.float64, device="cuda") for _ in range(2)]
    if n == 0:
        lses[1].zero_()
        return *outs, *lses
    for h in range(hq):
        kh, vh, qh = k[:, h // g].double(), v[:, h // g].double(), q[:, h].double()
        for i in range(0, m, 256):
            hid = hidden[i:i + 256]
            s = (qh[i:i + 256] @ kh.T * scale).masked_fill(hid, -math.inf)
            ds = (d + 8) * 2.0 ** -23 * abs(scale) * (qh[i:i + 256].abs() @ kh.abs().nan_to_num(0, 0, 0).T).masked_fill(hid, 0.0).amax(-1)
            top = s.amax(-1, keepdim=True)
            dead = top == -math.inf
            e = torch.exp(s - torch.where(dead, 0.0, top))
            l = e.sum(-1, keepdim=True)
            p = torch.where(dead, 0.0, e / l)
            # a value that no row of the block sees must not be multiplied
            seen = vh.masked_fill(hid.all(0)[:, None], 0.0)
            outs[0][i:i + 256, h] = p @ seen
            mass, each = p @ seen.abs(), (~hid).double() @ seen.abs() / torch.where(dead, 1.0, l)
            err = 2 * ds + 2.0 ** -20 + (2.0 ** -16 if dtype == BF16 else 2.0 ** -21) + 2.0 ** -23 * (40 + n / 8)
            outs[1][i:i + 256, h] = mass * err[:, None] + outs[0][i:i + 256, h].abs() * HALF_STEP[dtype] + TINY[dtype]
            if dtype == F16:
                outs[1][i:i + 256, h] += 2.0 ** -35 * each
            lse = (top + l.log())[:, 0].masked_fill(dead[:, 0], -math.inf)
            lses[0][i:i + 256, h] = lse
            lses[1][i:i + 256, h] = ds + 2.0 ** -20 + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0) + 2.0 ** -24 * n / 8
    return *outs, *lses


def hidden_of(last, n, window, sinks):
    """[m, n]: what tokens with `last` slots up to and with their own do not see."""
    t = torch.arange(n, device="cuda")
    last = torch.as_tensor(last, device="cuda")[:, None]
    hid = t >= last
    return hid | ((t < last - window) & (t >= sinks)) if window else hid


def prompt_reference(cache, q, starts, lengths, scale, window, sinks):
    T, hq, d = q.shape
    got = [torch.zeros(T, hq, d, dtype=torch.float64, device="cuda") for _ in range(2)]
    got += [torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda"), torch.zeros(T, hq, dtype=torch.float64, device="cuda")]
    for b, n in enumerate(lengths):
        at = slice(starts[b], starts[b + 1])
        m = starts[b + 1] - starts[b]
        k, v = rows_of(cache, b, list(range(n)))
        last = torch.arange(n - m + 1, n + 1, device="cuda")
        for x, y in zip(got, attend(q[at], k, v, hidden_of(last, n, window, sinks), scale, cache.dtype)):
            x[at] = y
    return got


def check_prompt(cache, fresh, lengths, group, window=0, sinks=0, seed=3, extra=0, scale=None, q=None, **kw):
    starts = [0] + np.cumsum(fresh).tolist()
    T, hq = starts[-1] + extra, cache.kv_heads * group
    if q is None:
        q = normal(seed, (T, hq, cache.head_dim), cache.dtype, 1.5)
    scale = cache.head_dim ** -0.5 if scale is None else scale
    out = torch.full_like(q, 7.0)
    lse = torch.full((T, hq), 7.0, device="cuda")
    got = mbg.gemv_attn_prompt(cache, q, ints(starts), ints(lengths), window=window, sinks=sinks, lse=lse, out=out, scale=scale, **kw)
    ref, tol, rl, lt = prompt_reference(cache, q[:starts[-1]], starts, lengths, scale, window, sinks)
    close(got[:starts[-1]], ref, tol, "out")
    close(lse[:starts[-1]], rl, lt, "lse")
    assert (got[starts[-1]:] == 7).all() and (lse[starts[-1]:] == 7).all()  # rows behind the last sequence
    return got


FRESH = [3, 0, 1, 130, 64, 1, 17]
CACHED = [0, 0, 0, 5, 100, 299, 33]
LENGTHS = [a + b for a, b in zip(FRESH, CACHED)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hk,group,dim,page,window,sinks", [
    (2, 4, 128, 16, 0, 0), (2, 1, 80, 24, 50, 5), (1, 12, 64, 7, 100, 37), (1, 20, 128, 1, 1, 0), (2, 2, 256, 16, 64, 4),
    (1, 3, 192, 32, 0, 0), (2, 8, 8, 16, 20, 200), (1, 5, 96, 64, 130, 1), (3, 7, 72, 3, 0, 9), (1, 40, 24, 16, 33, 8),
    (1, 16, 128, 16, 0, 0), (2, 1, 64, 128, 128, 128), (1, 2, 136, 16, 40, 3), (1, 3, 200, 8, 0, 0)])
def test_prompt_shapes(dtype, hk, group, dim, page, window, sinks):
    """Single tokens, empty sequences, pages and windows that end inside a tile; unused slots hold NaN."""
    check_prompt(make_cache(51, LENGTHS, hk, dim, page, dtype), FRESH, LENGTHS, group, window, sinks, extra=2)


@pytest.mark.parametrize("dim,group", [(1, 1), (7, 2), (77, 3), (130, 1), (255, 2), (128, 10)])
def test_prompt_layouts_without_vector_loads(dim, group):
    check_prompt(make_cache(52, LENGTHS, 2, dim, 5, F16, shift=1), FRESH, LENGTHS, group, 70, 2)


def test_prompt_strides():
    """Pools by heads, q and out as parts of wider tensors."""
    cache = make_cache(53, LENGTHS, 2, 128, 16, BF16, layout="head")
    wide = normal(8, (sum(FRESH), 24, 128), BF16, 1.5)
    check_prompt(cache, FRESH, LENGTHS, 4, q=wide[:, 8:16])
    out = torch.zeros(sum(FRESH), 8, 256, dtype=BF16, device="cuda")
    starts = ints([0] + np.cumsum(FRESH).tolist())
    got = mbg.gemv_attn_prompt(cache, wide[:, 8:16], starts, ints(LENGTHS), out=out[:, :, 128:])
    assert torch.equal(got, mbg.gemv_attn_prompt(cache, wide[:, 8:16].contiguous(), starts, ints(LENGTHS)))
    assert (out[:, :, :128] == 0).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("fresh,cached,hk,group,dim,page,window,sinks", [
    ([1000], [0], 2, 4, 128, 16, 0, 0), ([1500, 700], [300, 0], 1, 8, 64, 64, 400, 6), ([40, 3], [9000, 20000], 2, 4, 128, 64, 0, 0),
    ([257], [5000], 1, 1, 128, 16, 3000, 100), ([129, 600], [70, 3], 2, 2, 256, 16, 0, 0), ([2100], [50], 3, 3, 80, 24, 1000, 900)])
def test_prompt_long(dtype, fresh, cached, hk, group, dim, page, window, sinks):
    """Rows of several blocks, blocks cut between several groups of tiles."""
    lengths = [a + b for a, b in zip(fresh, cached)]
    check_prompt(make_cache(54, lengths, hk, dim, page, dtype), fresh, lengths, group, window, sinks)


def test_prompt_many_sequences():
    """More sequences than a block has threads, some without tokens."""
    fresh = [(7 * i) % 5 for i in range(700)]
    lengths = [f + (13 * i) % 40 if f else 0 for i, f in enumerate(fresh)]
    check_prompt(make_cache(55, lengths, 1, 64, 16, BF16), fresh, lengths, 4)


def test_prompt_scale_of_either_sign_and_zero():
    cache = make_cache(56, LENGTHS, 1, 64, 16, F16)
    for scale in (-0.3, 0.0, 1.0):
        check_prompt(cache, FRESH, LENGTHS, 4, scale=scale)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lead", [10.0, 17.0])
def test_prompt_first_token_leads_and_adds_nothing(dtype, lead):
    """A sink of the largest weight by far and a value of zero: the others are all of the output."""
    fresh, lengths = [300, 2], [300, 900]
    cache = make_cache(57, lengths, 1, 128, 16, dtype)
    cache.k.zero_()
    for b, n in enumerate(lengths):
        t = torch.arange(n, device="cuda")
        at = cache.page_table[b, t // 16].long(), t % 16
        cache.k[at[0], at[1], 0, 0] = torch.rand(n, device="cuda").to(dtype)
        cache.v[at] = (256 * (1 + 0.1 * torch.randn(n, 1, 128, device="cuda"))).to(dtype)
        cache.k[at[0][0], 0, 0, 0], cache.v[at[0][0], 0] = lead, 0.0
    q = torch.zeros(302, 2, 128, dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    for window in (0, 200):
        check_prompt(cache, fresh, lengths, 2, window, 3, q=q, scale=1.0)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompt_scores_that_keep_growing(dtype):
    """The running maximum rises in every tile, by more than the weights' range in all."""
    n = 1500
    cache = make_cache(58, [n], 1, 64, 16, dtype)
    t = torch.arange(n, device="cuda")
    cache.k[cache.page_table[0, t // 16].long(), t % 16, 0] = (t / 20.0).to(dtype)[:, None] * torch.eye(1, 64, device="cuda").to(dtype)
    q = torch.zeros(n, 2, 64, dtype=dtype, device="cuda")
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    check_prompt(cache, [n], [n], 2, q=q, scale=1.0)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_hidden_infinities_leave_no_trace(dtype, dim):
    """What lies in a token's future or behind its window may be infinite or NaN; what it sees is as in the formula.

    Rows that share a tile with such a value are computed again, each for itself, so that the sums behind their outputs are
    made in another order: they need not have the bits of the call without it, but both calls are held to the
    same distance from the formula over what the row sees (the definition has no term for the rest)."""
    fresh, lengths = [200, 40], [260, 1000]
    cache = make_cache(59, lengths, 2, dim, 16, dtype)
    q = normal(60, (240, 4, dim), dtype, 1.0)
    starts, n = ints([0, 200, 240]), ints(lengths)
    ref, tol, _, _ = prompt_reference(cache, q, [0, 200, 240], lengths, dim ** -0.5, 150, 4)
    close(mbg.gemv_attn_prompt(cache, q, starts, n, window=150, sinks=4), ref, tol)

    def place(b, t):
        return int(cache.page_table[b, t // 16]), t % 16

    for b, t, what in ((0, 255, math.inf), (1, 999, math.nan), (1, 700, math.inf)):
        p, o = place(b, t)
        cache.k[p, o], cache.v[p, o] = math.nan if b else 2.0, what
    got = mbg.gemv_attn_prompt(cache, q, starts, n, window=150, sinks=4)
    close(got[:195], ref[:195], tol[:195])               # slot 255 is token 195's own
    assert (got[195:200] == math.inf).all()
    close(got[200:239], ref[200:239], tol[200:239])
    assert got[239].isnan().all()
    p, o = place(0, 255)                                 # infinities of both signs: NaN where both are seen
    p2, o2 = place(0, 257)
    cache.v[p, o, :, 3], cache.v[p2, o2, :, 3] = math.inf, -math.inf
    got = mbg.gemv_attn_prompt(cache, q, starts, n, window=150, sinks=4)
    close(got[:195], ref[:195], tol[:195])
    assert (got[195:197] == math.inf).all()
    assert got[197:200, :, 3].isnan().all()
    keep = [d for d in range(dim) if d != 3]
    assert (got[197:200][..., keep] == math.inf).all()


def test_prompt_keys_of_minus_infinity():
    """Weight 0; a row of nothing else gives zeros."""
    cache = make_cache(61, [40, 70], 1, 64, 16, BF16)
    q = torch.ones(60, 2, 64, dtype=BF16, device="cuda")
    for b, dead in ((0, range(0, 20)), (1, range(1, 70, 3))):
        t = torch.tensor(list(dead), device="cuda")
        cache.k[cache.page_table[b].long()[t // 16], t % 16] = -math.inf
    out = check_prompt(cache, [40, 20], [40, 70], 2, q=q)
    assert (out[:20] == 0).all() and (out[20:] != 0).any()


def test_prompt_same_bits_every_time_on_other_streams_and_in_graphs():
    fresh, lengths = [700, 5, 300], [900, 4000, 300]
    cache = make_cache(62, lengths, 2, 128, 16, BF16)
    q, starts, n = normal(1, (1005, 8, 128), BF16), ints([0, 700, 705, 1005]), ints(lengths)
    first = mbg.gemv_attn_prompt(cache, q, starts, n, window=600, sinks=2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [mbg.gemv_attn_prompt(cache, q, starts, n, window=600, sinks=2, stream=streams[i % 3]) for i in range(9)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    out, graphs = torch.empty_like(q), []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            mbg.gemv_attn_prompt(cache, q, starts, n, window=600, sinks=2, out=out)
    for g in graphs:
        out.zero_()
        g.replay()
        assert torch.equal(out, first)
    # the captured call takes other tokens and lengths; rows behind the last sequence stay
    starts.copy_(ints([0, 2, 2, 131]))
    n.copy_(ints([890, 77, 200]))
    out.fill_(3)
    graphs[0].replay()
    ref, tol, _, _ = prompt_reference(cache, q[:131], [0, 2, 2, 131], [890, 77, 200], 128 ** -0.5, 600, 2)
    close(out[:131], ref, tol)
    assert (out[131:] == 3).all()


def test_prompt_out_of_range_is_reported():
    cache = make_cache(63, [64, 64], 1, 64, 16, F16, fill=0.0)
    q = normal(2, (20, 2, 64), F16)

    def call(starts, lengths):
        out = torch.full_like(q, 7.0)
        mbg.gemv_attn_prompt(cache, q, ints(starts), ints(lengths), out=out)
        return out

    good = call([0, 10, 20], [64, 64])
    assert mbg.gemv_get_device_error() == mbg.OK
    for starts, left in (([0, 21, 20], slice(0, 20)), ([-1, 10, 20], slice(0, 10)), ([0, 10, 9], slice(10, 20)),
                         ([0, 10, 2 ** 31 - 1], slice(10, 20))):
        out = call(starts, [64, 64])
        assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
        assert (out[left] == 7).all()
    out = call([0, 10, 20], [7, 64])  # ten tokens, seven slots: three see nothing
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    assert (out[:3] == 0).all() and torch.equal(out[10:], good[10:]) and out[:10].isfinite().all()
    out = call([0, 10, 20], [-4, cache.capacity + 1])
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    assert (out[:10] == 0).all()
    for bad in (-1, 1 << 20):
        cache.page_table[1, 2] = bad
        out = call([0, 10, 20], [64, 64])
        assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
        assert torch.equal(out[:10], good[:10]) and out.isfinite().all()


def test_prompt_cache_beyond_32_bit_offsets():
    pages, page, hk, d = 131100, 64, 2, 128  # 2.15e9 elements, 4.3 GB each
    k = torch.zeros(pages, page, hk, d, dtype=F16, device="cuda")
    v = torch.zeros(pages, page, hk, d, dtype=F16, device="cuda")
    table = torch.tensor([[pages - 1, 0, pages - 2, 7]], dtype=torch.int32, device="cuda")
    for i, p in enumerate(table[0].tolist()):
        k[p], v[p] = normal(30 + i, (page, hk, d), F16), normal(40 + i, (page, hk, d), F16)
    cache = mbg.PagedKV(k, v, table)
    check_prompt(cache, [70], [250], 4)
    check_shared(cache, [250], 129, 4)


# --------------------------------------------------------------------------- a shared prefix

def shared_cache(seed, lengths, prefix, hk, dim, page, dtype, **kw):
    """A cache whose rows begin with the same pages; the page in which the prefix ends is copied."""
    whole = prefix // page
    own = [max(0, n - whole * page) for n in lengths]
    cache = make_cache(seed, [prefix] + own, hk, dim, page, dtype, **kw)
    width = max(whole + max(-(-n // page) for n in own) + 2, -(-prefix // page))
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
    last = prefix % page
    for b, n in enumerate(own):
        table[b, :whole] = cache.page_table[0, :whole]
        pages = cache.page_table[b + 1, :-(-n // page)]
        table[b, whole:whole + len(pages)] = pages
        if n and last:  # of what the sequence has of it
            c = min(last, n)
            cache.k[pages[0].long(), :c], cache.v[pages[0].long(), :c] = (x[cache.page_table[0, whole].long(), :c] for x in (cache.k, cache.v))
    if last and own[0] < last:  # the first row names the whole prefix
        table[0, whole] = cache.page_table[0, whole]
    return mbg.PagedKV(cache.k, cache.v, table)


def check_shared(cache, lengths, prefix, group, window=0, sinks=0, q=None, scale=None):
    hq, d = cache.kv_heads * group, cache.head_dim
    if q is None:
        q = normal(5, (len(lengths), hq, d), cache.dtype, 1.5)
    scale = d ** -0.5 if scale is None else scale
    lse = torch.full((len(lengths), hq), 7.0, device="cuda")
    out = mbg.gemv_attn_shared(cache, q, ints(lengths), ints([prefix]), window=window, sinks=sinks, lse=lse, scale=scale)
    for b, n in enumerate(lengths):
        k, v = rows_of(cache, 0, list(range(min(n, prefix))))
        if n > prefix:
            k, v = (torch.cat(x) for x in zip((k, v), rows_of(cache, b, list(range(prefix, n)))))
        ref, tol, rl, lt = attend(q[b:b + 1], k, v, hidden_of([n], n, window, sinks), scale, cache.dtype)
        close(out[b:b + 1], ref, tol, f"out of {b}")
        close(lse[b:b + 1], rl, lt, f"lse of {b}")
    return out


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hk,group,dim,page,prefix,window,sinks", [
    (2, 4, 128, 16, 160, 0, 0), (2, 1, 80, 24, 100, 0, 0), (1, 12, 64, 7, 33, 90, 5), (1, 20, 128, 1, 130, 0, 0),
    (2, 2, 256, 16, 127, 140, 129), (1, 3, 192, 32, 128, 0, 0), (2, 8, 8, 16, 1, 0, 0), (1, 5, 96, 64, 200, 60, 210),
    (3, 7, 72, 3, 0, 0, 0), (1, 40, 24, 16, 64, 1, 0), (1, 16, 128, 16, 300, 150, 4)])
def test_shared_shapes(dtype, hk, group, dim, page, prefix, window, sinks):
    """Sequences shorter than the prefix, empty ones, windows that end in the prefix or behind it."""
    lengths = [prefix + 5, 0, prefix, prefix + 300, 1, prefix // 2, prefix + 1, prefix + 64]
    check_shared(shared_cache(71, lengths, prefix, hk, dim, page, dtype), lengths, prefix, group, window, sinks)


def test_shared_first_sequence_empty():
    """The first row of the table names the prefix's pages though its sequence has ended."""
    lengths = [0, 100, 150]
    cache = shared_cache(72, lengths, 70, 2, 64, 16, BF16)
    out = check_shared(cache, lengths, 70, 4)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("dim,group", [(7, 2), (77, 3), (128, 10)])
def test_shared_layouts_without_vector_loads(dim, group):
    lengths = [70, 64, 200]
    check_shared(shared_cache(73, lengths, 65, 2, dim, 5, F16, shift=1), lengths, 65, group)


@pytest.mark.parametrize("batch,prefix,hk,group,dim,window", [
    (70, 5000, 2, 4, 128, 0), (33, 20011, 1, 8, 64, 0), (3, 9000, 2, 2, 128, 0), (300, 700, 1, 1, 80, 0), (40, 3000, 2, 8, 256, 0),
    (40, 4000, 1, 4, 128, 1000)])
def test_shared_long(batch, prefix, hk, group, dim, window):
    lengths = [prefix + (37 * i) % 200 for i in range(batch)]
    check_shared(shared_cache(74, lengths, prefix, hk, dim, 16, BF16), lengths, prefix, group, window, 6)


def test_shared_is_the_paged_attention():
    """Where every sequence has the prefix's pages the two calls compute the same."""
    lengths = [300, 256, 999]
    cache = shared_cache(75, lengths, 256, 2, 128, 16, F16)
    q = normal(6, (3, 8, 128), F16)
    a = mbg.gemv_attn_shared(cache, q, ints(lengths), ints([256]))
    b = mbg.gemv_attn_paged(cache, q, ints(lengths))
    close(a, b, b.double().abs() * 2.0 ** -10 + 2.0 ** -10, "shared against paged")


def test_shared_same_bits_every_time_and_in_graphs():
    lengths = [3100, 3000, 0, 3999]
    cache = shared_cache(76, lengths, 3000, 2, 128, 16, BF16)
    q, n, pre = normal(7, (4, 8, 128), BF16), ints(lengths), ints([3000])
    first = mbg.gemv_attn_shared(cache, q, n, pre)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [mbg.gemv_attn_shared(cache, q, n, pre, stream=streams[i % 3]) for i in range(9)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    out, g = torch.empty_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mbg.gemv_attn_shared(cache, q, n, pre, out=out)
    g.replay()
    assert torch.equal(out, first)
    n.copy_(ints([3050, 3000, 2990, 5]))
    pre.copy_(ints([2000]))
    g.replay()
    fresh = mbg.gemv_attn_shared(cache, q, n, pre)
    assert torch.equal(out, fresh)


def test_shared_infinities_stay_where_they_are_seen():
    lengths, prefix = [100, 300, 129], 256
    cache = shared_cache(77, lengths, prefix, 1, 128, 16, BF16)
    q, n, pre = normal(8, (3, 4, 128), BF16), ints(lengths), ints([prefix])
    k, v = rows_of(cache, 0, list(range(100)))
    ref, tol, _, _ = attend(q[:1], k, v, hidden_of([100], 100, 0, 0), 128 ** -0.5, BF16)
    p = int(cache.page_table[0, 128 // 16])
    cache.v[p, 0] = math.inf  # slot 128: sequences 1 and 2 see it
    got = mbg.gemv_attn_shared(cache, q, n, pre)
    close(got[:1], ref, tol)  # computed again without the tile: as near to the formula, not the same bits
    assert (got[1:] == math.inf).all()
    own = int(cache.page_table[1, 290 // 16])
    cache.v[p, 0] = 0.0
    cache.k[own, 290 % 16] = math.nan
    got = mbg.gemv_attn_shared(cache, q, n, pre)
    assert got[1].isnan().all() and got[2].isfinite().all()
    close(got[:1], ref, tol)


def test_shared_out_of_range_is_reported():
    lengths = [100, 120]
    cache = shared_cache(78, lengths, 64, 1, 64, 16, F16, fill=0.0)
    q = normal(9, (2, 2, 64), F16)
    none = mbg.gemv_attn_paged(cache, q, ints(lengths))
    out = mbg.gemv_attn_shared(cache, q, ints(lengths), ints([-5]))
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX and torch.equal(out, none)
    out = mbg.gemv_attn_shared(cache, q, ints(lengths), ints([cache.capacity + 1]))
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX and torch.equal(out[0], mbg.gemv_attn_shared(cache, q, ints(lengths), ints([100]))[0])
    mbg.gemv_get_device_error()
    mbg.gemv_attn_shared(cache, q, ints([cache.capacity + 9, -1]), ints([64]))
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    with pytest.raises(ValueError):
        mbg.gemv_attn_shared(cache, q, ints(lengths), ints([3, 4]))
    with pytest.raises(ValueError):
        mbg.gemv_attn_shared(cache, q[:, :, :32], ints(lengths), ints([3]))


@pytest.mark.parametrize("dim", [8, 16, 128])
def test_infinities_next_to_cut_blocks(dim):
    """Rows that are joined from parts, and rows of a prefix, are computed again where a hidden value is infinite."""
    n, m = 3000, 200
    cache = make_cache(81, [n], 1, dim, 16, BF16)
    q = normal(82, (m, 4, dim), BF16)
    starts, lens = ints([0, m]), ints([n])
    ref, tol, _, _ = prompt_reference(cache, q, [0, m], [n], dim ** -0.5, 0, 0)
    last = int(cache.page_table[0, (n - 1) // 16])
    cache.v[last, (n - 1) % 16] = math.inf  # the last token's own
    got = mbg.gemv_attn_prompt(cache, q, starts, lens)
    close(got[:-1], ref[:-1], tol[:-1])
    assert (got[-1] == math.inf).all()
    lengths = [2600, 2990, 3000]
    shared = mbg.PagedKV(cache.k, cache.v, cache.page_table.expand(3, -1).contiguous())
    got = mbg.gemv_attn_shared(shared, q[:3], ints(lengths), ints([3000]))
    for b in (0, 1):
        k, v = rows_of(cache, 0, list(range(lengths[b])))
        ref, tol, _, _ = attend(q[b:b + 1], k, v, hidden_of([lengths[b]], lengths[b], 0, 0), dim ** -0.5, BF16)
        close(got[b:b + 1], ref, tol, f"sequence {b}")
    assert (got[2] == math.inf).all()


def test_prompt_arguments_are_checked():
    cache = make_cache(83, [20, 20], 2, 64, 16, F16, fill=0.0)
    q, starts, n = normal(1, (9, 4, 64), F16), ints([0, 4, 9]), ints([20, 20])
    for bad in (dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q[0]), dict(starts=ints([0, 9])), dict(lengths=ints([20])),
                dict(window=-1), dict(sinks=2 ** 31), dict(out=q[:5]), dict(lse=torch.zeros(9, 3, device="cuda")),
                dict(starts=starts.cpu()), dict(q=q.transpose(1, 2))):
        args = dict(q=q, starts=starts, lengths=n)
        args.update(bad)
        with pytest.raises(ValueError):
            mbg.gemv_attn_prompt(cache, args.pop("q"), args.pop("starts"), args.pop("lengths"), **args)
    for bad in (q.float(), q.bfloat16()):
        with pytest.raises(TypeError):
            mbg.gemv_attn_prompt(cache, bad, starts, n)
    with pytest.raises(TypeError):
        mbg.gemv_attn_shared(cache, q[:2], n, torch.zeros(1, device="cuda"))
    empty = mbg.gemv_attn_prompt(cache, q[:0], ints([0, 0, 0]), n)
    assert empty.shape == (0, 4, 64)


def test_two_threads_share_a_prefix_call_by_call():
    """Calls of two threads on one stream do not mix: a call is three launches over one workspace."""
    import threading

    lengths = [700, 640, 900]
    caches = [shared_cache(84 + i, lengths, 640, 2, 128, 16, F16) for i in range(2)]
    q, n, pre = normal(86, (3, 8, 128), F16), ints(lengths), ints([640])
    want = [mbg.gemv_attn_shared(c, q, n, pre) for c in caches]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        outs = [mbg.gemv_attn_shared(caches[i], q, n, pre) for _ in range(50)]
        torch.cuda.synchronize()
        bad.extend(i for o in outs if not torch.equal(o, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_prompt_blocks_that_take_seconds():
    """A call's waits are bounded, not its length: 2^28 - 5 slots (one page, named again and again) for each of
    152 heads.  Keys of 0 weigh every slot alike and the values are powers of two, so that sums of a tile's weights
    and of 32768 slots' values are exact; the last ones' rounding is 2^-24 of them."""
    page, pages, hk, dim = 512, 2 ** 19, 152, 64
    n = page * pages - 5
    v = torch.tensor([2.0 ** (d % 4) * (1 - d % 2 * 2) for d in range(dim)], dtype=BF16, device="cuda")
    cache = mbg.PagedKV(torch.zeros(1, page, hk, dim, dtype=BF16, device="cuda"), v.expand(1, page, hk, dim).contiguous(),
                        torch.zeros(1, pages, dtype=torch.int32, device="cuda"))
    lse = torch.empty(1, hk, dtype=torch.float32, device="cuda")
    got = mbg.gemv_attn_prompt(cache, normal(91, (1, hk, dim), BF16), ints([0, 1]), ints([n]), lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(got, v.expand(1, hk, dim))
    assert (lse.double() - math.log(n)).abs().max() <= 2.0 ** -18  # half a step of 19.4, of its 13.4 / ln 2 and of log2


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim,m", [(64, 1), (128, 1), (128, 70), (192, 1)])
def test_prompt_and_prefix_sums_of_many_slots(dtype, dim, m):
    """2^20 slots of like weights and positive values (two pages named again and again), 200 heads, so that some
    blocks of rows are whole and some are cut.  A sum that keeps 24 bits loses up to 2^-23 of itself with each
    product, half of that on average, and is half of the whole on average: 2^-25 N = 2^-10 of N = 2^15 slots, which the
    kernel does not exceed; what joins the sums is FP32's rounding, far below."""
    page, hk, n = 256, 200, 2 ** 20
    torch.manual_seed(94)
    v = (0.5 + torch.rand(2, page, hk, dim, device="cuda") / 2).to(dtype)
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None] % 2
    cache = mbg.PagedKV(torch.zeros_like(v), v, table)
    want = v.double().mean((0, 1))[None, :, None]  # the last tokens' missing slots: m / n of it
    q = normal(95, (m, 4 * hk, dim), dtype)
    got = mbg.gemv_attn_prompt(cache, q, ints([0, m]), ints([n])).view(m, hk, 4, dim)
    tol = (2.0 ** -10 + HALF_STEP[dtype] + m / n) * want
    assert ((got.double() - want).abs() <= tol).all()
    both = mbg.PagedKV(cache.k, v, table.expand(m, -1).contiguous())
    got = mbg.gemv_attn_shared(both, q, ints([n] * m), ints([n - 7])).view(m, hk, 4, dim)
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("axis", [1, 2])
def test_prompt_and_prefix_over_broadcast_pools(axis):
    """Pools that are broadcast along their tokens or heads (a stride of 0)."""
    base = make_cache(92, [100, 77], 4, 64, 16, F16)
    k, v = (x.narrow(axis, 1, 1).expand_as(x) for x in (base.k, base.v))
    cache, dense = mbg.PagedKV(k, v, base.page_table), mbg.PagedKV(k.contiguous(), v.contiguous(), base.page_table)
    q, starts, lens = normal(93, (60, 8, 64), F16), ints([0, 40, 60]), ints([100, 77])
    assert torch.equal(mbg.gemv_attn_prompt(cache, q, starts, lens), mbg.gemv_attn_prompt(dense, q, starts, lens))
    a, b = (mbg.PagedKV(c.k, c.v, c.page_table[:1].expand(2, -1).contiguous()) for c in (cache, dense))
    assert torch.equal(mbg.gemv_attn_shared(a, q[:2], lens, ints([64])), mbg.gemv_attn_shared(b, q[:2], lens, ints([64])))
