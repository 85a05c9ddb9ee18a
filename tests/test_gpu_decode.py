"""The decode-step operators against their definitions in 64 bits.

Tolerances.  Output rounding: half a step of the type, eps / 2 relative (and
the smallest subnormal of binary16, 2^-25).  Scores: an FP32 sum of D exact
products, each addition off by at most one step of the running sum (the MMA
unit truncates), so |ds| <= (D + 8) 2^-23 A with A = scale sum |q_d k_d|; a
weight is then off by 2 |ds| relative, plus 2^-20 for the exponential and the
sums of weights.  P enters the V product as two 16-bit parts, off by 2^-16
(bf16) or 2^-21 relative and 2^-25 absolute (f16).  Angles: 2^-33 turns and
the FP32 rounding and 2 ulp of sincospi, 2^-21 in all.  Norms: FP32 sums of at
most 64 dependent additions, 2^-18 relative to the magnitudes summed.
"""

import math

import numpy as np
import pytest

import memory_bound_gemv_gb300 as mbg

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
HALF_STEP = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {F16: 2.0 ** -25, BF16: 0.0, F32: 0.0}


@pytest.fixture(autouse=True)
def no_device_error():
    assert mbg.gemv_get_device_error() in (mbg.OK, mbg.ERR_BAD_INDEX)
    yield
    assert mbg.gemv_get_device_error() == mbg.OK


def normal(seed, shape, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(0, scale, generator=g).to(dtype)


def close(got, ref, tol, what=""):
    got, ref, tol = got.double(), ref.double(), tol.double()
    same = (got == ref) | (got.isnan() & ref.isnan())
    bad = ~(same | ((got - ref).abs() <= tol))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((got - ref).abs() / tol)[bad].max():.3g} times the bound"


def make_cache(seed, lengths, heads, dim, page, dtype, layout="token", shift=0, spare=2, history=False, fill=float("nan")):
    """A cache whose unused slots and pages hold `fill`; shift moves the pools off 16-byte alignment."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lengths]
    width, total = max(need, default=0) + spare, sum(need) + 3
    order = rng.permutation(total)
    table = np.full((len(lengths), width), -1, np.int32)
    i = 0
    for b, n in enumerate(need):
        table[b, :n] = order[i:i + n]
        i += n
    pools = []
    used = torch.zeros(total, page, dtype=torch.bool)
    for b, n in enumerate(lengths):
        t = np.arange(n)
        used[table[b, t // page], t % page] = True
    used = used.cuda()[:, :, None, None]
    for k in range(2):
        shape = (total, page, heads, dim) if layout == "token" else (total, heads, page, dim)
        flat = normal(seed + k, (int(np.prod(shape)) + shift,), dtype)
        pool = flat[shift:].view(shape)
        if layout != "token":
            pool = pool.transpose(1, 2)
        pool.copy_(torch.where(used, pool, torch.tensor(fill, dtype=dtype, device="cuda")))
        pools.append(pool)
    extra = {}
    if history:
        shape = (len(lengths), heads, width * page)
        extra["scores"] = normal(seed + 5, shape).abs()
        extra["stamps"] = torch.from_numpy(rng.permuted(np.broadcast_to(np.arange(shape[2], dtype=np.int32), shape), axis=-1)).cuda().contiguous()
    return mbg.PagedKV(pools[0], pools[1], torch.from_numpy(table).cuda(), **extra)


def rows_of(cache, b, slots):
    """K and V of slots of sequence b, [n, heads, dim]."""
    slots = torch.as_tensor(slots, device="cuda").long()
    p = cache.page_table[b].long()[slots // cache.page_size]
    return cache.k[p, slots % cache.page_size], cache.v[p, slots % cache.page_size]


def attn_reference(cache, q, lengths, scale, window):
    """out, its bound, weights [B, Hkv, cap], their bound, lse, its bound."""
    B, hq, d = q.shape
    hk = cache.kv_heads
    g = hq // hk
    out, tol = torch.zeros(B, hq, d, dtype=torch.float64, device="cuda"), torch.zeros(B, hq, d, dtype=torch.float64, device="cuda")
    w = torch.zeros(B, hk, cache.capacity, dtype=torch.float64, device="cuda")
    wt = torch.zeros_like(w)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device="cuda")
    lt = torch.zeros_like(lse)
    split = 2.0 ** -16 if cache.dtype == BF16 else 2.0 ** -21
    for b, n in enumerate(lengths):
        lo = max(0, n - window) if window else 0
        if n == lo:
            continue
        k, v = rows_of(cache, b, list(range(lo, n)))
        k, v = (x.double().transpose(0, 1).repeat_interleave(g, 0) for x in (k, v))  # [hq, n, d]
        qq = q[b].double()[:, None]
        s = (qq * k).sum(-1) * scale
        ds = (d + 8) * 2.0 ** -23 * ((qq * k).abs().nan_to_num(0, 0, 0).sum(-1) * abs(scale)).amax(-1)
        m = s.amax(-1, keepdim=True)
        dead = (m == -math.inf)
        e = torch.exp(s - torch.where(dead, 0.0, m))
        l = e.sum(-1, keepdim=True)
        p = torch.where(dead, 0.0, e / l)
        out[b] = torch.einsum("hn,hnd->hd", p, v)
        mass = torch.einsum("hn,hnd->hd", p, v.abs())
        err = 2 * ds + 2.0 ** -20 + split + 2.0 ** -24 * (32 + (n - lo) / 16)
        tol[b] = mass * err[:, None] + out[b].abs() * HALF_STEP[cache.dtype] + TINY[cache.dtype]
        if cache.dtype == F16:
            tol[b] += 2.0 ** -25 * v.abs().sum(1) / torch.where(dead, 1.0, l)
        w[b, :, lo:n] = p.view(hk, g, -1).sum(1)
        wt[b, :, lo:n] = (p * err[:, None]).view(hk, g, -1).sum(1) + 2.0 ** -126
        lse[b] = torch.where(dead, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"), m + l.log())[:, 0]
        lt[b] = ds + 2.0 ** -20 + 2.0 ** -22 * lse[b].abs().nan_to_num(0, 0, 0)
    return out, tol, w, wt, lse, lt


def check_attn(cache, q, lengths, scale=None, window=0, **kw):
    scale = cache.head_dim ** -0.5 if scale is None else scale
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = mbg.gemv_attn_paged(cache, q, lens, scale=scale, window=window, lse=lse, **kw)
    ref, tol, _, _, rl, lt = attn_reference(cache, q, lengths, scale, window)
    close(out, ref, tol, "out")
    close(lse, rl, lt, "lse")
    return out


LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 300]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hk,group,dim,page", [
    (2, 1, 128, 16), (3, 2, 64, 16), (1, 3, 80, 24), (2, 5, 96, 1), (2, 7, 128, 3), (8, 4, 128, 16), (1, 8, 256, 64),
    (2, 9, 128, 16), (1, 12, 64, 7), (2, 16, 80, 16), (1, 20, 128, 32), (1, 17, 192, 16), (2, 4, 8, 16), (1, 40, 24, 16)])
def test_attn_shapes(dtype, hk, group, dim, page):
    """Head sizes, groups and pages that end inside a tile; unused slots hold NaN."""
    cache = make_cache(11, LENGTHS, hk, dim, page, dtype)
    q = normal(5, (len(LENGTHS), hk * group, dim), dtype, 1.5)
    check_attn(cache, q, LENGTHS)


@pytest.mark.parametrize("dim,group", [(1, 1), (7, 2), (77, 3), (100, 9), (130, 1), (255, 2), (128, 10)])
def test_attn_layouts_without_vector_loads(dim, group):
    """Odd head sizes and pools off 16-byte alignment take the element-wise loads."""
    cache = make_cache(12, LENGTHS, 2, dim, 5, F16, shift=1)
    q = normal(6, (len(LENGTHS), 2 * group, dim), F16, 1.5)
    check_attn(cache, q, LENGTHS)


@pytest.mark.parametrize("window", [1, 5, 16, 100, 250, 1000])
def test_attn_window(window):
    cache = make_cache(13, LENGTHS, 2, 64, 16, BF16)
    check_attn(cache, normal(7, (len(LENGTHS), 4, 64), BF16, 1.5), LENGTHS, window=window)


def test_attn_strides_and_output():
    """Pools by heads, q and out as parts of wider tensors."""
    cache = make_cache(14, LENGTHS, 2, 128, 16, F16, layout="head")
    wide = normal(8, (len(LENGTHS), 24, 128), F16, 1.5)
    out = torch.zeros(len(LENGTHS), 8, 256, dtype=F16, device="cuda")
    got = check_attn(cache, wide[:, 8:16], LENGTHS, out=out[:, :, 128:])
    assert got.data_ptr() == out[:, :, 128:].data_ptr()
    assert (out[:, :, :128] == 0).all()
    check_attn(cache, wide.transpose(1, 2).contiguous().transpose(1, 2)[:, 8:16].contiguous(), LENGTHS)


def test_attn_long_rows_split_over_many_blocks():
    lengths = [20011, 3, 70000]
    cache = make_cache(15, lengths, 2, 128, 64, F16, fill=0.0)
    check_attn(cache, normal(9, (3, 16, 128), F16, 2.0), lengths)


def test_attn_many_sequences():
    """More sequences than a block has threads, many of them empty."""
    lengths = [(37 * i) % 50 if i % 3 else 0 for i in range(301)]
    cache = make_cache(16, lengths, 1, 64, 16, BF16)
    check_attn(cache, normal(10, (301, 4, 64), BF16, 1.5), lengths)
    check_attn(cache, normal(10, (301, 4, 64), BF16, 1.5), [0] * 301)


def test_attn_infinite_scores():
    """Keys of -inf leave weight 0; a sequence of nothing else gives zeros."""
    lengths = [40, 40, 40]
    cache = make_cache(17, lengths, 1, 64, 16, BF16)
    q = torch.ones(3, 2, 64, dtype=BF16, device="cuda")
    for b, dead in ((0, range(0, 40, 3)), (1, range(40)), (2, [39])):
        s = torch.tensor(list(dead), device="cuda")
        cache.k[cache.page_table[b].long()[s // 16], s % 16] = -math.inf
    out = check_attn(cache, q, lengths)
    assert (out[1] == 0).all() and out.isfinite().all()


def test_attn_nan_stays_in_its_row():
    lengths = [40, 40, 40]
    cache = make_cache(18, lengths, 2, 64, 16, F16)
    clean = mbg.gemv_attn_paged(cache, normal(3, (3, 4, 64), F16), torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    p = cache.page_table[1].long()
    cache.k[p[1], 3, 1] = math.nan
    got = mbg.gemv_attn_paged(cache, normal(3, (3, 4, 64), F16), torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    assert got[1, 2:].isnan().all()
    got[1, 2:] = clean[1, 2:]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("group,dim,page,window", [(1, 128, 16, 0), (4, 128, 16, 0), (5, 80, 24, 33), (9, 64, 16, 0),
                                                   (20, 128, 8, 100), (3, 33, 16, 0)])
def test_attn_weights(group, dim, page, window):
    cache = make_cache(19, LENGTHS, 2, dim, page, F16, history=True)
    q = normal(4, (len(LENGTHS), 2 * group, dim), F16, 1.5)
    lens = torch.tensor(LENGTHS, dtype=torch.int32, device="cuda")
    before = cache.scores.clone()
    sums = torch.full_like(before, -5.0)
    mbg.gemv_attn_paged(cache, q, lens, window=window, accumulate=True, scores_out=sums)
    assert torch.equal(cache.scores, before)
    _, _, w, wt, _, _ = attn_reference(cache, q, LENGTHS, dim ** -0.5, window)
    slot = torch.arange(cache.capacity, device="cuda")
    n = lens[:, None, None]
    live = ((slot < n) & (slot >= ((n - window).clamp(min=0) if window else 0))).expand_as(before)
    ref = torch.where(live, before.double() + w, -5.0)
    close(sums, ref, torch.where(live, wt + ref.abs() * 2.0 ** -24 * 2 + w * group * 2.0 ** -24, 0.0), "scores")
    mbg.gemv_attn_paged(cache, q, lens, window=window, accumulate=True)  # in place
    assert torch.equal(cache.scores, torch.where(live, sums, before))


def test_attn_same_bits_every_time_and_on_other_streams():
    lengths = [5000, 100, 0, 2777]
    cache = make_cache(20, lengths, 2, 128, 16, BF16)
    q = normal(1, (4, 16, 128), BF16)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    first = mbg.gemv_attn_paged(cache, q, lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(12):
        outs.append(mbg.gemv_attn_paged(cache, q, lens, stream=streams[i % 3]))
    with torch.cuda.stream(streams[0]):
        outs.append(mbg.gemv_attn_paged(cache, q, lens))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)


def test_attn_in_a_graph_takes_new_lengths():
    lengths = [400, 0, 33]
    cache = make_cache(21, lengths, 2, 64, 16, F16, history=True)
    q = normal(2, (3, 8, 64), F16)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, sums = torch.empty_like(q), torch.zeros_like(cache.scores)
    mbg.gemv_attn_paged(cache, q, lens, out=out, accumulate=True, scores_out=sums)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mbg.gemv_attn_paged(cache, q, lens, out=out, accumulate=True, scores_out=sums)
    for new in ([400, 0, 33], [17, 0, 1], [399, 0, 20]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        got = out.clone()
        assert torch.equal(got, mbg.gemv_attn_paged(cache, q, lens))
        ref, tol, _, _, _, _ = attn_reference(cache, q, new, 0.125, 0)
        close(got, ref, tol)


def test_attn_bad_pages_and_lengths_are_reported_and_skipped():
    lengths = [64, 64, 64]
    cache = make_cache(22, lengths, 1, 64, 16, F16)
    q = normal(2, (3, 2, 64), F16)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    good = mbg.gemv_attn_paged(cache, q, lens)
    assert mbg.gemv_get_device_error() == mbg.OK
    cache.page_table[1, 2] = 1 << 20
    bad = mbg.gemv_attn_paged(cache, q, lens)
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    assert torch.equal(bad[0], good[0]) and torch.equal(bad[2], good[2]) and bad.isfinite().all()
    cache.page_table[1, 2] = -1
    mbg.gemv_attn_paged(cache, q, lens)
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    lens[1] = -3
    out = mbg.gemv_attn_paged(cache, q, lens)
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    assert (out[1] == 0).all() and torch.equal(out[0], good[0])
    lens[1] = cache.capacity + 1
    out = mbg.gemv_attn_paged(cache, q, lens)
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    assert torch.equal(out[2], good[2])
    mbg.gemv_attn_paged(cache, q, torch.tensor([64, 0, 64], dtype=torch.int32, device="cuda"))
    assert mbg.gemv_get_device_error() == mbg.OK


def test_attn_cache_beyond_32_bit_offsets():
    """Pools of more than 2^31 elements: the far pages are read where they are."""
    pages, page, hk, d = 131100, 64, 2, 128  # 2.15e9 elements, 4.3 GB each
    k = torch.zeros(pages, page, hk, d, dtype=F16, device="cuda")
    v = torch.zeros(pages, page, hk, d, dtype=F16, device="cuda")
    table = torch.tensor([[pages - 1, 0, pages - 2, 7]], dtype=torch.int32, device="cuda")
    for i, p in enumerate(table[0].tolist()):
        k[p], v[p] = normal(30 + i, (page, hk, d), F16), normal(40 + i, (page, hk, d), F16)
    cache = mbg.PagedKV(k, v, table)
    check_attn(cache, normal(3, (1, 8, d), F16), [250])


# --------------------------------------------------------------------------- rotary positions

def rope_reference(x, positions, table_args, theta=10000.0):
    rot, sections, pairs = table_args
    half = rot // 2
    axis = np.repeat(np.arange(len(sections)), sections)
    f = theta ** (-2.0 * np.arange(half) / max(rot, 1))
    ang = positions.cpu().numpy().astype(np.float64)[axis].T * f
    c, s = torch.from_numpy(np.cos(ang)).cuda()[:, None], torch.from_numpy(np.sin(ang)).cuda()[:, None]
    x = x.double()
    y = x.clone()
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    mag = torch.zeros_like(x)
    mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


@pytest.mark.parametrize("src", [F32, F16, BF16])
@pytest.mark.parametrize("dst", [F16, BF16])
@pytest.mark.parametrize("dim,sections,pairs,page,shift", [
    (128, [64], False, 16, 0), (128, [16, 24, 24], False, 16, 0), (128, [16, 24, 24], True, 16, 0),
    (64, [16], False, 24, 0), (64, [8], True, 16, 0), (80, [13, 14, 13], False, 7, 0), (256, [40, 44, 44], False, 16, 0),
    (77, [5, 6], True, 5, 0), (10, [0, 5], False, 16, 0), (12, [0], False, 16, 0), (128, [64], False, 16, 1)])
def test_rope_append(src, dst, dim, sections, pairs, page, shift):
    hq, hk, counts = 5, 2, [3, 0, 40, 1]
    starts = [0, 2, 17, 63]
    lengths = [a + n for a, n in zip(starts, counts)]
    T = sum(counts)
    cache = make_cache(31, lengths, hk, dim, page, dst, shift=shift, fill=0.0, history=True)
    qkv = normal(32, (T, hq + 2 * hk, dim), src, 1.3)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    seq = torch.repeat_interleave(torch.arange(4), torch.tensor(counts)).to(torch.int32).cuda()
    slots = torch.cat([torch.arange(a, a + n) for a, n in zip(starts, counts)]).to(torch.int32).cuda()
    slots[1] = -1  # padding
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    positions = torch.randint(-1000, 2000000, (len(sections), T), generator=g, device="cuda", dtype=torch.int32)
    positions[:, 2] = 2 ** 31 - 1
    stamps = torch.arange(900, 900 + T, dtype=torch.int32, device="cuda")
    old = [cache.k.clone(), cache.v.clone(), cache.scores.clone(), cache.stamps.clone()]
    rope = mbg.RopeTable(2 * sum(sections), sections=sections, pairs=pairs)
    out = mbg.gemv_rope_append(cache, q, k, v, positions, slots, rope, seq=seq, stamps=stamps)
    args = (2 * sum(sections), sections, pairs)
    # 2^31 radians in 64 bits are themselves off by 2^-22; sines and the table add 2^-21
    for got, x in ((out, q),):
        ref, mag = rope_reference(x, positions, args)
        close(got, ref, mag * 2.0 ** -20 + ref.abs() * HALF_STEP[dst] + TINY[dst], "q")
    put = [i for i in range(T) if int(slots[i]) >= 0]
    pages = cache.page_table[seq[put].long(), slots[put].long() // page].long()
    offs = slots[put].long() % page
    ref, mag = rope_reference(k, positions, args)
    close(cache.k[pages, offs], ref[put], mag[put] * 2.0 ** -20 + ref[put].abs() * HALF_STEP[dst] + TINY[dst], "k")
    assert torch.equal(cache.v[pages, offs], v[put].float().to(dst))
    for now, was in zip((cache.k, cache.v), old):  # nothing else has changed
        was[pages, offs] = now[pages, offs]
        assert torch.equal(now, was)
    b, s = seq[put].long(), slots[put].long()
    old[2][b, :, s] = 0.0
    old[3][b, :, s] = stamps[put][:, None]
    assert torch.equal(cache.scores, old[2]) and torch.equal(cache.stamps, old[3])


def test_rope_defaults_single_tokens_and_bad_slots():
    cache = make_cache(33, [20, 20], 1, 64, 16, F16, fill=0.0, history=True)
    q, k, v = normal(1, (2, 2, 64)), normal(2, (2, 1, 64)), normal(3, (2, 1, 64))
    rope = mbg.RopeTable(64)
    pos = torch.tensor([[19, 4]], dtype=torch.int32, device="cuda")
    slots = torch.tensor([19, 4], dtype=torch.int32, device="cuda")
    mbg.gemv_rope_append(cache, q, k, v, pos, slots, rope)
    assert mbg.gemv_get_device_error() == mbg.OK
    assert cache.stamps[0, 0, 19] == 19 and cache.stamps[1, 0, 4] == 4 and cache.scores[1, 0, 4] == 0
    kept = [cache.k.clone(), cache.v.clone(), cache.scores.clone(), cache.stamps.clone()]
    for bad, seq in ((cache.capacity, None), (2 ** 31 - 1, None), (40, None), (3, 2), (3, -1)):
        slots[0] = bad if seq is None else 3
        slots[1] = -1
        mbg.gemv_rope_append(cache, q, k, v, pos, slots, rope,
                             seq=None if seq is None else torch.tensor([seq, 1], dtype=torch.int32, device="cuda"))
        assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
        assert all(torch.equal(a, b) for a, b in zip(kept, (cache.k, cache.v, cache.scores, cache.stamps)))
    with pytest.raises(ValueError):
        mbg.gemv_rope_append(cache, normal(1, (3, 2, 64)), normal(1, (3, 1, 64)), normal(1, (3, 1, 64)),
                             torch.zeros(1, 3, dtype=torch.int32, device="cuda"),
                             torch.zeros(3, dtype=torch.int32, device="cuda"), rope)


# --------------------------------------------------------------------------- eviction

def evict_reference(scores, stamps, n, keep, sinks, recent):
    """Moves of one row: the definition, by sorting."""
    s = np.where(np.isnan(scores[:n]), -np.inf, scores[:n]).astype(np.float64)
    if n <= keep:
        return []
    newest = int(stamps[:n].max())
    safe = (stamps[:n] < sinks) | (stamps[:n].astype(np.int64) > newest - recent)
    order = np.lexsort((np.arange(n), -s, ~safe))
    stays = np.zeros(n, bool)
    stays[order[:keep]] = True
    holes = np.flatnonzero(~stays[:keep])
    movers = keep + np.flatnonzero(stays[keep:])
    assert len(holes) == len(movers)
    return list(zip(movers.tolist(), holes.tolist()))


def same_bits(a, b):
    t = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.view(t), b.view(t))


def check_evict(cache, lengths, keep, sinks, recent):
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    k, v, sc, st = cache.k.clone(), cache.v.clone(), cache.scores.clone(), cache.stamps.clone()
    moves, counts = mbg.gemv_kv_evict_plan(cache, lens, keep, sinks=sinks, recent=recent)
    assert same_bits(cache.k, k) and torch.equal(lens, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    moves, counts, scn, stn = moves.cpu().numpy(), counts.cpu().numpy(), sc.cpu().numpy(), st.cpu().numpy()
    for b, n in enumerate(lengths):
        for h in range(cache.kv_heads):
            want = evict_reference(scn[b, h], stn[b, h], n, keep, sinks, recent)
            got = [tuple(m) for m in moves[b, h, :counts[b, h]].tolist()]
            assert got == want, (b, h, n, len(got), len(want))
            for src, dst in want:
                ps, pd = (int(cache.page_table[b, x // cache.page_size]) for x in (src, dst))
                for pool in (k, v):
                    pool[pd, dst % cache.page_size, h] = pool[ps, src % cache.page_size, h]
                sc[b, h, dst], st[b, h, dst] = sc[b, h, src], st[b, h, src]
    for _ in range(2):  # a plan may be carried out again
        mbg.gemv_kv_evict_apply(cache, torch.from_numpy(moves).cuda(), torch.from_numpy(counts).cuda(), lens, keep)
        for a, b in ((cache.k, k), (cache.v, v), (cache.scores, sc)):
            assert same_bits(a, b)
        assert torch.equal(cache.stamps, st)
        assert lens.tolist() == [min(n, keep) for n in lengths]


@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (7, 2, 3), (64, 4, 16), (64, 100, 100), (64, 0, 1000),
                                               (100, 0, 0), (299, 4, 10), (300, 0, 0), (1000, 0, 0)])
def test_evict_budgets(keep, sinks, recent):
    lengths = [0, 1, 8, 64, 65, 300, 299]
    check_evict(make_cache(51, lengths, 2, 64, 16, F16, history=True), lengths, keep, sinks, recent)


@pytest.mark.parametrize("dim,page,shift,layout", [(80, 24, 0, "token"), (77, 5, 0, "token"), (128, 16, 1, "token"),
                                                   (256, 64, 0, "head"), (8, 1, 0, "token")])
def test_evict_layouts(dim, page, shift, layout):
    lengths = [130, 77]
    cache = make_cache(52, lengths, 3, dim, page, BF16, shift=shift, layout=layout, history=True)
    check_evict(cache, lengths, 50, 2, 10)


@pytest.mark.parametrize("kind", ["equal", "signs", "special", "fine"])
def test_evict_ties_and_special_scores(kind):
    lengths = [2500, 1025, 1024]
    cache = make_cache(53, lengths, 2, 8, 16, F16, history=True)
    shape = cache.scores.shape
    if kind == "equal":
        cache.scores.fill_(0.5)
    elif kind == "signs":  # -0 and 0 are equal
        cache.scores.copy_(torch.where(torch.rand(shape, device="cuda") < 0.5, -0.0, 0.0))
    elif kind == "special":
        pick = torch.randint(0, 7, shape, device="cuda")
        values = torch.tensor([math.nan, -math.inf, math.inf, -1.0, 0.0, 1e-45, 3.0], device="cuda")
        cache.scores.copy_(values[pick])
    else:  # neighbours in the last bits
        cache.scores.copy_(1.0 + torch.randint(0, 50, shape, device="cuda") * 2.0 ** -23)
    check_evict(cache, lengths, 777, 4, 100)


def test_evict_long_rows():
    lengths = [70001, 20000]
    cache = make_cache(54, lengths, 1, 16, 64, F16, history=True)
    check_evict(cache, lengths, 4000, 4, 512)


def test_evict_stamps_at_the_ends_of_their_range():
    cache = make_cache(55, [100], 1, 8, 16, F16, history=True)
    cache.stamps.copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, cache.stamps.shape, device="cuda").to(torch.int32))
    cache.stamps[0, 0, 5], cache.stamps[0, 0, 6] = 2 ** 31 - 1, -2 ** 31
    check_evict(cache, [100], 30, 0, 2 ** 31 - 1)


def test_evict_bad_lengths_and_moves_are_reported():
    cache = make_cache(56, [60, 60], 1, 8, 16, F16, history=True)
    lens = torch.tensor([60, cache.capacity + 5], dtype=torch.int32, device="cuda")
    mbg.gemv_kv_evict_plan(cache, lens, 20)
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    before = cache.k.clone()
    moves = torch.tensor([[[[1 << 20, 3]]], [[[cache.capacity - 1, 2]]]], dtype=torch.int32, device="cuda")
    counts = torch.tensor([[1], [1]], dtype=torch.int32, device="cuda")
    mbg.gemv_kv_evict_apply(cache, moves, counts, None, 20)  # a slot outside, and one without a page
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    assert same_bits(cache.k, before)
    with pytest.raises(ValueError):
        mbg.gemv_kv_evict_plan(cache, lens, 20, moves=torch.zeros(2, 1, 3, 2, dtype=torch.int32, device="cuda"))


# --------------------------------------------------------------------------- norms

def norm_reference(y, x, a):
    f = lambda t: t.double()  # noqa: E731
    eps = a.get("eps", 1e-6)

    def norm(v, dv):
        mean = v.mean(-1, keepdim=True) if a.get("kind") == "layer" else torch.zeros_like(v[:, :1])
        c = v - mean
        r = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
        # the mean's and the square sum's errors, and those that came in
        scale = v.abs() + v.abs().mean(-1, keepdim=True)
        dc = 2.0 ** -18 * scale + dv + (dv.mean(-1, keepdim=True) if a.get("kind") == "layer" else 0)
        dr = 2.0 ** -18 + (c.abs() * dc).mean(-1, keepdim=True) * r * r
        return c * r, dc * r + (c * r).abs() * dr

    u, du = f(y), torch.zeros_like(f(y))
    if a.get("post"):
        u, du = norm(u, du)
        if a.get("post_weight") is not None:
            u, du = u * f(a["post_weight"]), du * f(a["post_weight"]).abs()
    if a.get("gate") is not None:
        u, du = u * f(a["gate"]), du * f(a["gate"]).abs()
    s = f(x) + a.get("alpha", 1.0) * u
    ds = abs(a.get("alpha", 1.0)) * (du + u.abs() * 2.0 ** -22) + s.abs() * 2.0 ** -23 + f(x).abs() * 2.0 ** -24
    h, dh = norm(s, ds)
    w = f(a["pre_weight"]) if a.get("pre_weight") is not None else torch.ones_like(s)
    if a.get("unit_offset"):
        w = 1 + w
    h, dh = h * w, dh * w.abs() + (h * w).abs() * 2.0 ** -22
    if a.get("pre_bias") is not None:
        h = h + f(a["pre_bias"])
        dh = dh + h.abs() * 2.0 ** -23 + f(a["pre_bias"]).abs() * 2.0 ** -24
    return s, ds, h, dh


def check_norm(y, x, h_dtype=F16, **a):
    out, h = mbg.gemv_norm_residual(y, x, h_dtype=h_dtype, **a)
    s, ds, rh, dh = norm_reference(y, x, a)
    assert out.dtype == x.dtype and h.dtype == h_dtype
    close(out, s, ds + s.abs() * HALF_STEP[x.dtype] + TINY[x.dtype], "out")
    close(h, rh, dh + rh.abs() * HALF_STEP[h_dtype] + TINY[h_dtype], "h")
    return out, h


@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (2, 8), (5, 100), (1, 255), (4, 1024), (1, 4096), (3, 4104),
                                        (2, 8192), (2, 14336), (1, 16384), (2, 16392), (1, 40001)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_widths(rows, width, kind):
    for yt, xt, ht in ((F32, F32, F16), (BF16, BF16, BF16), (F16, F32, F32)):
        y, x = normal(61, (rows, width), yt, 1.7), normal(62, (rows, width), xt, 3.0)
        w = lambda i: 1 + normal(i, (width,), F32, 0.2)  # noqa: E731
        check_norm(y, x, ht, kind=kind, post=True, post_weight=w(1).to(xt), gate=normal(3, (width,), xt, 0.5), alpha=0.7,
                   pre_weight=w(2).to(xt), eps=1e-5)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_operands_left_out_and_by_row(kind):
    y, x = normal(63, (6, 520), F32, 1.7), normal(64, (6, 520), F16, 3.0)
    row = lambda i, t=BF16: normal(i, (6, 520), t, 0.3)  # noqa: E731
    check_norm(y, x, kind=kind)
    check_norm(y, x, kind=kind, post=True)
    check_norm(y, x, BF16, kind=kind, gate=row(1), pre_weight=row(2), pre_bias=row(3), unit_offset=True)
    check_norm(y, x, F32, kind=kind, gate=row(1, F16), pre_weight=row(2, F32), pre_bias=row(3, F32)[0], alpha=-2.0)
    out, h = mbg.gemv_norm_residual(y, x, kind=kind, pre=False)
    assert h is None
    close(out, x.double() + y.double(), (x.double().abs() + y.double().abs()) * 2.0 ** -23
          + (x.double() + y.double()).abs() * HALF_STEP[F16])


def test_norm_strides_in_place_and_offsets():
    wide = normal(65, (5, 1100), F32, 1.5)
    x = normal(66, (5, 700), F32)
    s, ds, rh, dh = norm_reference(wide[:, 3:603], x[:, :600], {})
    out, h = mbg.gemv_norm_residual(wide[:, 3:603], x[:, :600], out=x[:, :600], h_dtype=F32)  # unaligned rows, in place
    assert out.data_ptr() == x.data_ptr()
    close(out, s, ds + s.abs() * 2.0 ** -24)
    close(h, rh, dh + rh.abs() * 2.0 ** -24)
    for width in (512, 20000):  # the long rows read their inputs several times
        y, x = normal(67, (2, width)), normal(68, (2, width))
        s, ds, rh, dh = norm_reference(y, x, {"post": True})
        out, h = mbg.gemv_norm_residual(y, x, post=True, out=x, h=y)
        close(out, s, ds + s.abs() * 2.0 ** -24)
        close(h, rh, dh + rh.abs() * 2.0 ** -24)


def test_norm_large_mean_keeps_the_variance():
    """A LayerNorm of values around 1000 with a spread of 0.1."""
    x = (1000 + normal(69, (3, 4096), F32, 0.1))
    y = torch.zeros_like(x)
    check_norm(y, x, F32, kind="layer", eps=1e-12)


def test_norm_zero_rows_and_nan():
    y, x = torch.zeros(3, 64, device="cuda"), torch.zeros(3, 64, device="cuda")
    x[1, 5] = math.nan
    x[2] = 2.0
    out, h = mbg.gemv_norm_residual(y, x)
    assert (h[0] == 0).all() and h[1].isnan().all() and torch.equal(h[2], torch.ones(64, dtype=F16, device="cuda"))
    assert mbg.gemv_norm_residual(y[:0], x[:0])[0].shape == (0, 64)


def test_norm_refusals_of_the_binding():
    y, x = torch.zeros(2, 8, device="cuda"), torch.zeros(2, 8, device="cuda")
    for bad in (dict(gate=torch.zeros(3, 8, device="cuda")), dict(pre_weight=torch.zeros(9, device="cuda")),
                dict(out=torch.zeros(2, 9, device="cuda")), dict(pre=False, pre_weight=torch.zeros(8, device="cuda")),
                dict(h=torch.zeros(8, 2, device="cuda").t())):
        with pytest.raises(ValueError):
            mbg.gemv_norm_residual(y, x, **bad)
    for bad in (dict(out=torch.zeros(2, 8, dtype=F16, device="cuda")), dict(gate=torch.zeros(8, dtype=torch.int32, device="cuda"))):
        with pytest.raises(TypeError):
            mbg.gemv_norm_residual(y, x, **bad)
    with pytest.raises(mbg.GemvError):
        mbg.gemv_norm_residual(y, x, out=torch.zeros(8, device="cuda").expand(2, 8))


def test_binding_refusals():
    cache = make_cache(71, [20, 20], 2, 64, 16, F16)
    lens = torch.tensor([20, 20], dtype=torch.int32, device="cuda")
    q = normal(1, (2, 4, 64), F16)
    for bad in (dict(q=q[:1]), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(lengths=lens[:1]), dict(window=-1),
                dict(accumulate=True), dict(scores_out=torch.zeros(1, device="cuda")),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(lse=torch.zeros(2, 3, device="cuda"))):
        with pytest.raises(ValueError):
            mbg.gemv_attn_paged(cache, **{**dict(q=q, lengths=lens), **bad})
    for bad in (dict(q=q.bfloat16()), dict(lengths=lens.long()), dict(out=q.float())):
        with pytest.raises(TypeError):
            mbg.gemv_attn_paged(cache, **{**dict(q=q, lengths=lens), **bad})
    with pytest.raises(ValueError):
        mbg.gemv_kv_evict_plan(cache, lens, 4)  # no scores
    with pytest.raises(ValueError):
        mbg.PagedKV(cache.k, cache.v, cache.page_table, scores=torch.zeros(2, 2, 5, device="cuda"))


@pytest.mark.parametrize("kind", ["normal", "equal", "few values"])
@pytest.mark.parametrize("keep,sinks,recent", [(2000, 4, 100), (50, 0, 0), (50, 3, 60), (5000, 2, 5000), (4990, 0, 4992)])
def test_evict_a_few_slots_over_the_budget(keep, sinks, recent, kind):
    """One to six slots too many, as in decode steps; rows where every slot is protected among them."""
    lengths = [keep + k for k in (1, 2, 3, 4, 5, 6, 0)]
    cache = make_cache(57, lengths, 2, 8, 16, F16, history=True)
    if kind == "equal":
        cache.scores.fill_(2.0)
    elif kind == "few values":
        cache.scores.copy_(torch.randint(0, 3, cache.scores.shape, device="cuda").float())
    check_evict(cache, lengths, keep, sinks, recent)


def test_the_compiled_checks_take_the_common_calls_and_leave_the_others():
    from memory_bound_gemv_gb300 import decode

    cache = make_cache(72, [20, 20], 2, 64, 16, F16, fill=0.0, history=True)
    lens = torch.tensor([20, 20], dtype=torch.int32, device="cuda")
    q, out = normal(1, (2, 4, 64), F16), torch.empty(2, 4, 64, dtype=F16, device="cuda")
    ws = cache._workspace(4, False, mbg._stream_ptr(None), None)

    def attn(q=q, lens=lens, out=out, lse=None, window=0):
        return decode._quick.attn(cache._at, 0, q, lens, out, lse, 0, ws[0], ws[1], 0.125, window, None)

    assert attn() == 0 and attn(q=normal(1, (2, 8, 64), F16)[:, ::2]) == 0
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q.cpu()), dict(q=3),
                dict(lens=lens.long()), dict(lens=lens[:1]), dict(out=None), dict(out=out[0]), dict(window=-1),
                dict(window=1 << 40), dict(window="2"), dict(lse=out), dict(lens=torch.stack((lens, lens), 1)[:, 0])):
        assert attn(**bad) == -1, bad
    y = normal(2, (3, 32))
    assert decode._quick.norm(y, y, None, None, None, None, y.clone(), None, 1.0, 1e-6, 0, None) == 0
    for bad in ((y, y, None, None, None, None, y.half(), None), (y, y[:2], None, None, None, None, y, None),
                (y, y, y[0][:31], None, None, None, y, None), (y.int(), y, None, None, None, None, y, None),
                (y, y, None, None, None, None, y, y[0]), (y, None, None, None, None, None, y, None)):
        assert decode._quick.norm(*bad, 1.0, 1e-6, 0, None) == -1
    with pytest.raises(mbg.GemvError):  # a refusal of the library comes through the Python form
        mbg.gemv_norm_residual(y, y.clone(), out=torch.zeros(1, 32, device="cuda").expand(3, 32), pre=False)
    moves = torch.empty(2, 2, 16, 2, dtype=torch.int32, device="cuda")
    counts = torch.empty(2, 2, dtype=torch.int32, device="cuda")
    assert decode._quick.plan(cache._at, 0, lens, 16, 0, 0, moves, counts, None) == 0
    assert decode._quick.apply(cache._at, 0, moves, counts, None, 16, None) == 0
    assert decode._quick.plan(cache._at, 0, lens, 0, 0, 0, moves, counts, None) == -1
    assert decode._quick.plan(cache._at, 0, lens, 16, 0, 0, moves[:, :, :3], counts, None) == -1
    assert decode._quick.apply(cache._at, 0, moves.float(), counts, None, 16, None) == -1


@pytest.mark.parametrize("width", [2, 9, 17, 250, 1001, 4001, 8191, 16383, 20001])
@pytest.mark.parametrize("yt,xt,ht", [(F32, F32, F16), (BF16, BF16, BF16), (F32, F16, F32)])
def test_norm_rows_that_begin_anywhere(width, yt, xt, ht):
    """Nine rows of an odd width begin at every place between two 16-byte borders."""
    y, x = normal(81, (9, width), yt, 1.7), normal(82, (9, width), xt, 3.0)
    args = dict(kind="layer", post=True, post_weight=normal(83, (width,), xt), gate=normal(84, (9, width), xt),
                pre_weight=normal(85, (width,), F32), pre_bias=normal(86, (9, width), ht), alpha=0.5)
    s, ds, rh, dh = norm_reference(y, x, args)
    out, h = check_norm(y, x, ht, **args)
    guard = torch.full((9 * width + 64,), -3.0, dtype=xt, device="cuda")  # in place, between guards
    inside = guard[32:32 + 9 * width].view(9, width)
    inside.copy_(x)
    again, h2 = mbg.gemv_norm_residual(y, inside, out=inside, h_dtype=ht, **args)
    assert torch.equal(inside, out) and torch.equal(h2, h)
    assert (guard[:32] == -3).all() and (guard[32 + 9 * width:] == -3).all()
    wide = torch.full((9, width + 5), -3.0, dtype=ht, device="cuda")  # rows of another stride than x's
    _, h3 = mbg.gemv_norm_residual(y, x, out=torch.empty_like(x), h=wide[:, 3:3 + width], **args)
    assert torch.equal(h3, h) and (wide[:, :3] == -3).all() and (wide[:, 3 + width:] == -3).all()


def test_attn_calls_with_wide_and_narrow_loads_share_a_workspace():
    # many rows, one tile of 16 query heads for the wide loads, two of eight for the narrow ones; long enough to be cut
    lengths = [300 + 97 * (b % 31) for b in range(512)]
    pools = [normal(3 + i, (4096, 16, 8, 64), F16) for i in range(2)]
    per = -(-max(lengths) // 16)
    table = torch.from_numpy(np.random.default_rng(9).integers(0, 4096, (512, per)).astype(np.int32)).cuda()
    cache = mbg.PagedKV(*pools, table)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    flat = normal(8, (512 * 128 * 64 + 1,), F16)
    narrow, wide = flat[1:].view(512, 128, 64), flat[1:].clone().view(512, 128, 64)
    first = mbg.gemv_attn_paged(cache, narrow, n, out=torch.full_like(wide, math.nan))
    for _ in range(3):
        mbg.gemv_attn_paged(cache, wide, n, out=torch.full_like(wide, math.nan))
        again = mbg.gemv_attn_paged(cache, narrow, n, out=torch.full_like(wide, math.nan))
        assert same_bits(first, again)


@pytest.mark.parametrize("width,pad", [(333, 0), (1001, 0), (4001, 0), (777, 3), (9001, 0), (11908, 0)])
@pytest.mark.parametrize("yt,xt", [(BF16, BF16), (F32, F16), (F32, F32)])
def test_norm_nan_stays_in_its_row_at_odd_widths(yt, xt, width, pad):
    rows = 1400  # several rows per block, neighbours in other blocks
    y = normal(1, (rows, width + pad), yt)[:, :width]
    x = normal(2, (rows, width + pad), xt)[:, :width]
    w, g = normal(3, (width,), F16), normal(4, (width,), BF16)
    # rows laid out like x: where a row begins settles how its sums are grouped
    call = dict(post=True, post_weight=w, gate=g, pre_weight=w, kind="layer", h_dtype=F16)
    call["out"] = torch.empty(rows, width + pad, dtype=xt, device="cuda")[:, :width]
    out, h = mbg.gemv_norm_residual(y, x, **call)
    y[1::3] = math.nan
    x[2::3] = math.inf
    call["out"] = torch.empty_strided(out.shape, out.stride(), dtype=xt, device="cuda")
    bad_out, bad_h = mbg.gemv_norm_residual(y, x, **call)
    assert same_bits(out[::3].contiguous(), bad_out[::3].contiguous())
    assert same_bits(h[::3].contiguous(), bad_h[::3].contiguous())
    assert bad_out[1::3].isnan().all() and bad_h[1::3].isnan().all() and bad_h[2::3].isnan().all()
    # in place: the neighbours' elements are being written meanwhile
    y, x = normal(1, (rows, width + pad), yt)[:, :width], normal(2, (rows, width + pad), xt)[:, :width]
    mbg.gemv_norm_residual(y, x, **{**call, "out": x, "h": y, "h_dtype": None})
    assert same_bits(x.contiguous(), out.contiguous())


@pytest.mark.parametrize("batch,longest,spread,window", [
    (57, 400, 0, 0), (57, 400, 3, 0), (57, 400, 60, 0), (24, 900, 0, 0), (24, 900, 17, 0), (48, 300, 200, 256), (64, 700, 1, 0)])
def test_attn_rows_of_about_one_length(batch, longest, spread, window):
    # uncut, cut and ragged rows, by lanes (up to 32 sequences) and by blocks
    lengths = [longest - (7 * b) % (spread + 1) for b in range(batch)]
    cache = make_cache(batch, lengths, 8, 64, 16, BF16)
    check_attn(cache, normal(batch + 1, (batch, 16, 64), BF16), lengths, window=window)
