"""Serving a batch over a paged cache: page tables and slot maps built on the GPU, the append of normed and
turned queries and keys, attention with a sliding window and first tokens that stay visible (of one new
token per sequence and of whole prompts), and attention of a batch that shares a long prefix.

Each case is one call as a serving program makes it.  The plain forms below are elementary torch operations
in 32 bits; with ``own`` the calls go to ``memory_bound_gemv_gb300``.
"""

import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a decode step's bookkeeping: one token for each of a batch's requests, some of them over, pages of 16
        dict(name="tables_step", op="tables", batch=64, longest=6000, fresh="step", page=16, prefix=0, pad=0),
        # a call that admits prompts: ragged ones beside requests that go on, a slot map padded to a fixed size
        dict(name="tables_prompts", op="tables", batch=307, longest=1500, fresh="prompts", page=16, prefix=512, pad=999),
        # one decode step: the FP32 output of the QKV product, normed for each head, rotated and appended
        dict(name="norm_rope_step", op="rope", type="f16", source="f32", tokens=1, batch=1, q_heads=32, kv_heads=8,
             dim=128, sections="64", pairs=False, page=16, far=4000, unit=False),
        # a prompt of three sequences in one call
        dict(name="norm_rope_prompt", op="rope", type="bf16", source="bf16", tokens=7001, batch=3, q_heads=32,
             kv_heads=8, dim=128, sections="64", pairs=False, page=32, far=9000, unit=True),
        # a serving batch whose layer sees a window and four first tokens
        dict(name="sinks_step_batch", op="attn", type="bf16", batch=48, q_heads=32, kv_heads=8, dim=128, longest=6000,
             page=16, window=1024, sinks=4, weights=False),
        # no shared heads, heads of 80, pages of 24 that end inside a tile, an empty row, weights kept for eviction
        dict(name="sinks_step_odd", op="attn", type="f16", batch=11, q_heads=14, kv_heads=14, dim=80, longest=5003,
             page=24, window=777, sinks=37, weights=True),
        # a whole prompt through such a layer
        dict(name="prompt_window_sinks", op="prompt", type="f16", batch=1, q_heads=32, kv_heads=8, dim=128, fresh=9001,
             cached=0, page=16, window=2048, sinks=4),
        # parts of long prompts, each behind what its sequence has cached already, no window
        dict(name="prompt_parts", op="prompt", type="bf16", batch=6, q_heads=32, kv_heads=8, dim=128, fresh=2000,
             cached=12000, page=64, window=0, sinks=0),
        # a few short ones: heads of 80, pages of 24, single tokens and empty sequences among them
        dict(name="prompt_short_odd", op="prompt", type="bf16", batch=5, q_heads=14, kv_heads=14, dim=80, fresh=130,
             cached=300, page=24, window=100, sinks=5),
        # a few users behind a system prompt
        dict(name="shared_few", op="shared", type="f16", batch=4, q_heads=32, kv_heads=8, dim=128, prefix=1000,
             longest=300, page=16, window=0, sinks=0),
        # a batch of answers to questions about one long document
        dict(name="shared_document", op="shared", type="bf16", batch=64, q_heads=32, kv_heads=8, dim=128, prefix=32768,
             longest=900, page=16, window=0, sinks=0),
        # samples of one prompt whose end lies inside a page, heads of 80 in pages of 24, one row of them empty
        dict(name="shared_odd", op="shared", type="bf16", batch=23, q_heads=14, kv_heads=14, dim=80, prefix=7001,
             longest=500, page=24, window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "attn", "prompt", "prompt", "shared", "shared"])
    most_bytes = max(work(c)["bytes"] for c in listed())
    most_flops = max(work(c)["flops"] for c in listed())
    while True:
        hk = rng.choice([1, 2, 4, 5, 8, 14])
        heads = dict(type=rng.choice(["f16", "bf16"]), q_heads=hk * rng.choice([1, 2, 4, 5, 7, 8, 12, 16]), kv_heads=hk,
                     dim=rng.choice([64, 80, 96, 128, 128, 192, 256]), page=rng.choice([1, 8, 16, 16, 24, 64, 128]))
        seen = dict(window=rng.choice([0, _log(rng, 1, 8192)]), sinks=rng.choice([0, rng.randint(1, 8), _log(rng, 1, 300)]))
        if op == "tables":
            c = dict(op=op, batch=_log(rng, 1, 2000), longest=_log(rng, 1, 8000), fresh=rng.choice(["step", "prompts"]),
                     page=rng.choice([1, 8, 16, 24, 64]), prefix=0, pad=rng.choice([0, rng.randint(1, 3000)]))
            c["prefix"] = rng.choice([0, rng.randint(0, c["longest"])])
        elif op == "rope":
            dim = rng.choice([64, 80, 96, 128, 128, 256])
            half = dim // 2
            a = rng.randint(1, half - 2)
            b = rng.randint(1, half - a - 1)
            tokens = _log(rng, 1, 8000)
            c = dict(op=op, type=rng.choice(["f16", "bf16"]), source=rng.choice(["f32", "f16", "bf16"]),
                     tokens=tokens, batch=rng.randint(1, min(tokens, 64)), q_heads=8 * rng.choice([1, 4, 5]),
                     kv_heads=rng.choice([1, 4, 8]), dim=dim,
                     sections=rng.choice(["%d" % half, "%d" % max(1, half // 2), "%d,%d,%d" % (a, b, half - a - b)]),
                     pairs=rng.random() < 0.5, page=rng.choice([8, 16, 24, 64]), far=_log(rng, 100, 2000000),
                     unit=rng.random() < 0.5)
        elif op == "attn":
            c = dict(op=op, batch=_log(rng, 1, 96), longest=_log(rng, 1, 131072), weights=rng.random() < 0.3, **heads, **seen)
            c["window"] = c["window"] or _log(rng, 1, 8192)
        elif op == "prompt":
            c = dict(op=op, batch=rng.randint(1, 12), fresh=_log(rng, 1, 9000), cached=rng.choice([0, _log(rng, 1, 30000)]),
                     **heads, **seen)
        else:
            c = dict(op=op, batch=_log(rng, 2, 128), prefix=_log(rng, 16, 60000), longest=_log(rng, 1, 1500), **heads,
                     window=0, sinks=0)
            if rng.random() < 0.2:
                c.update(seen)
        w = work(c)
        if op in ("tables", "rope"):
            pool = 0
        else:
            pool = sum(_spans(c)[1]) * c["kv_heads"] * c["dim"] * 4
            pool += c.get("prefix", 0) * c["kv_heads"] * c["dim"] * 4
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops and pool <= 5.3e8:
            return c


def _spans(c):
    """(new tokens, slots in use with them) of each sequence, in order; shared: slots behind the prefix."""
    n = c["batch"]
    if c["op"] == "attn":
        got = [max(1, c["longest"] * (n - i) // n) for i in range(n)]
        if n > 1:
            got[-1] = 0
        return [1 if g else 0 for g in got], got
    if c["op"] == "prompt":  # longest first; the one before the last a single token, the last empty (of more than two)
        fresh = [max(1, c["fresh"] * (n - i) // n) for i in range(n)]
        cached = [c["cached"] * (i + 1) // n for i in range(n)]
        if n > 2:
            fresh[-2] = 1
            fresh[-1] = cached[-1] = 0
        return fresh, [a + b for a, b in zip(fresh, cached)]
    got = [c["longest"] * (n - i) // n for i in range(n)]
    return [1] * n, got


def _seen(c, n):
    """Slots that a token with n slots before and with it attends to."""
    if not c["window"] or n <= c["window"]:
        return n
    return min(n, c["window"] + min(c["sinks"], n - c["window"]))


def _empty(c):
    """The row of a shared batch that is empty (its sequence has ended)."""
    return c["batch"] - 1 if c["batch"] > 8 else None


def work(case):
    c = case
    if c["op"] == "tables":
        p = _plan(c)
        return {"bytes": 16 * c["batch"] + 8 * p["tokens"] + 8 * (p["pages"] + p["freed"]), "flops": 4 * c["batch"] + p["tokens"]}
    if c["op"] == "rope":
        n = c["tokens"] * (c["q_heads"] + 2 * c["kv_heads"]) * c["dim"]
        axes = c["sections"].count(",") + 1
        return {"bytes": n * (SIZE[c["source"]] + 2) + 4 * c["tokens"] * (axes + 2) + 4 * c["dim"],
                "flops": 7.0 * c["tokens"] * (c["q_heads"] + c["kv_heads"]) * c["dim"]}
    slot, vector = c["kv_heads"] * c["dim"] * 4, 4 * c["q_heads"] * c["dim"]  # K and V of a slot; q and out of a token
    fresh, lengths = _spans(c)
    if c["op"] == "attn":
        seen = sum(_seen(c, n) for n in lengths)
        return {"bytes": seen * slot + c["batch"] * vector + (8 * seen * c["kv_heads"] if c["weights"] else 0),
                "flops": 4.0 * seen * c["q_heads"] * c["dim"]}
    if c["op"] == "prompt":
        b = f = 0
        for m, n in zip(fresh, lengths):
            b += min(n, _seen(c, n - m + 1) + m - 1) * slot + m * vector
            # each token sees one slot more than the one before until its window is full
            most = n if not c["window"] else _seen(c, 10 ** 9)
            first = n - m + 1
            grow = min(m, max(0, most - first + 1))
            f += grow * (2 * first + grow - 1) / 2 + (m - grow) * most
        return {"bytes": b, "flops": 4.0 * f * c["q_heads"] * c["dim"]}
    pre, gone = c["prefix"], _empty(c)
    tails = [0 if i == gone else n for i, n in enumerate(lengths)]
    whole = [0 if i == gone else n + pre for i, n in enumerate(lengths)]
    rows = sum(_seen(c, n) for n in whole)
    tail = sum(min(t, _seen(c, n)) for t, n in zip(tails, whole))
    # of the prefix: what any of the rows sees
    past = max([_seen(c, n) - min(t, _seen(c, n)) for t, n in zip(tails, whole)] + [0])
    return {"bytes": (past + tail) * slot + c["batch"] * vector, "flops": 4.0 * rows * c["q_heads"] * c["dim"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, scale, generator=g).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _pages(need, width, rng, first=()):
    """A page table over a pool in which the sequences' pages lie scattered behind the pages that all begin with;
    -1 where a sequence has none."""
    total = sum(need) + len(first) + 7
    order = list(range(total))
    rng.shuffle(order)
    first = [order.pop() for _ in first]
    table = torch.full((len(need), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :len(first) + n] = torch.tensor(first + order[at:at + n], dtype=torch.int32)
        at += n
    return table.cuda(), total


def _plan(c, order=None):
    """A scheduler's step: slots in use and new tokens (-1: over) of each request, and what that asks for."""
    p, n, hi, rng = c["page"], c["batch"], c["longest"], random.Random(c["batch"])
    lengths, fresh = [], []
    for _ in range(n):
        k = rng.randint(min(hi, c["prefix"] + 1), hi)
        if c["fresh"] == "step":
            lengths.append(k)
            fresh.append(-1 if rng.random() < 0.05 else 1)
        else:
            new = rng.random()
            lengths.append(min(k, c["prefix"]) // p * p if new < 0.4 else k)
            fresh.append(rng.randint(1, max(1, hi // 3)) if new < 0.4 else -1 if new < 0.5 else 1)
    if order is not None:  # the same requests in another order
        mixed = list(zip(lengths, fresh))
        order.shuffle(mixed)
        lengths, fresh = zip(*mixed)
    have = [-(-k // p) for k in lengths]
    pages = sum(-(-(k + f) // p) - h for k, f, h in zip(lengths, fresh, have) if f > 0)
    freed = sum(max(0, h - c["prefix"] // p) for f, h in zip(fresh, have) if f < 0)
    return dict(lengths=lengths, fresh=fresh, have=have, pages=pages, freed=freed, tokens=sum(max(0, f) for f in fresh))


def _tables(s, seed):
    c, rng = s, random.Random(seed)
    plan, p = _plan(c, rng), c["page"]
    held = [max(0, h - c["prefix"] // p) for h in plan["have"]]
    width = -(-(c["longest"] + c["longest"] // 3 + 2) // p) + 1
    table, total = _pages(held, width, rng, first=range(c["prefix"] // p))
    spare = plan["pages"] + 50
    s["total"] = total + spare
    # the ring of free pages, whose next one lies anywhere in it
    ring, at = [-1] * s["total"], rng.randrange(s["total"])
    free = list(range(total, total + spare))
    rng.shuffle(free)
    for i, page in enumerate(free):
        ring[(at + i) % s["total"]] = page
    s["table"], s["ring"], s["ring_at"] = table, _ints(ring), _ints([at, spare])
    s["lengths"], s["fresh_of"] = _ints(plan["lengths"]), _ints(plan["fresh"])
    s["shared"] = _ints([c["prefix"]] * c["batch"])
    room = c["pad"] + max(c["batch"], -(-plan["tokens"] // 256) * 256)
    s["slots"], s["seq"] = torch.empty(room, dtype=torch.int32, device="cuda"), torch.empty(room, dtype=torch.int32, device="cuda")
    s["starts"] = torch.empty(c["batch"] + 1, dtype=torch.int32, device="cuda")
    s["lengths_after"], s["ring_at_after"] = torch.empty_like(s["lengths"]), torch.empty_like(s["ring_at"])


def prepare(case, seed):
    c, g, rng = case, _gen(seed), random.Random(seed)
    s = dict(case)
    if own:
        import memory_bound_gemv_gb300 as mbg

        s["mbg"] = mbg
    if c["op"] == "tables":
        _tables(s, seed)
        if own:
            # the pools themselves are not touched by this call: a token's K and V of one element stand for them
            kv = torch.empty(s["total"], c["page"], 1, 1, dtype=torch.float16, device="cuda")
            s["cache"] = mbg.PagedKV(kv, kv, s["table"])
            s["pool"] = mbg.PagePool(ring=s["ring"], state=s["ring_at"])
        return s
    dt, hk, hq, d, page = DT[c["type"]], c["kv_heads"], c["q_heads"], c["dim"], c["page"]
    if c["op"] == "rope":
        t, n = c["tokens"], c["batch"]
        counts = [t // n + (1 if i < t % n else 0) for i in range(n)]
        starts = [(37 * i + 11) % 200 for i in range(n)]
        lengths = [a + b for a, b in zip(starts, counts)]
        s["seq"] = torch.repeat_interleave(torch.arange(n), torch.tensor(counts)).to(torch.int32).cuda()
        s["slots"] = torch.cat([torch.arange(a, a + b) for a, b in zip(starts, counts)]).to(torch.int32).cuda()
        axes = c["sections"].count(",") + 1
        s["positions"] = torch.randint(0, c["far"], (axes, t), generator=g, device="cuda", dtype=torch.int32)
        # the QKV product's output, seen as three parts; a few channels are much larger than the others
        qkv = _normal(g, (t, (hq + 2 * hk), d), torch.float32, 1.3)
        qkv[..., rng.sample(range(d), 3)] *= 9.0
        qkv = qkv.to(DT[c["source"]])
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        shift = 0.0 if c["unit"] else 1.0
        s["q_weight"], s["k_weight"] = (shift + _normal(g, (2, d), torch.float32, 0.2)).to(dt)
        parts = [int(x) for x in c["sections"].split(",")]
        rot = 2 * sum(parts)
        s["rot"] = rot
        s["freq"] = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
        s["axis"] = torch.repeat_interleave(torch.arange(len(parts)), torch.tensor(parts)).cuda()
        s["q_out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")
        s["table"], total = _pages([-(-n // page) for n in lengths], max(lengths) // page + 4, rng)
        if own:
            s["rope"] = mbg.RopeTable(rot, sections=parts, theta=10000.0, pairs=c["pairs"])
    else:
        fresh, lengths = _spans(c)
        order = list(range(c["batch"]))
        rng.shuffle(order)
        fresh, lengths = [fresh[i] for i in order], [lengths[i] for i in order]
        pre = c["prefix"] if c["op"] == "shared" else 0
        # pages of the prefix that all have; the one in which it ends is each sequence's own copy
        own_slots = [n + pre - pre // page * page for n in lengths]
        if pre and _empty(c) is not None:
            lengths[order.index(_empty(c))] = -pre
        s["spans"] = [(m, n + pre) for m, n in zip(fresh, lengths)]
        s["lengths"] = _ints([n + pre for n in lengths])
        need = [-(-n // page) for n in own_slots]
        s["table"], total = _pages(need, pre // page + max(need) + 3, rng, first=range(pre // page))
        tokens = sum(fresh) if c["op"] == "prompt" else c["batch"]
        s["qv"] = _normal(g, (tokens, hq, d), dt, 1.6)
        s["out"] = torch.empty_like(s["qv"])
        s["scale"] = d ** -0.5
        if c["op"] == "prompt":
            at = [0]
            for m in fresh:
                at.append(at[-1] + m)
            s["starts"] = _ints(at)
    s["kp"] = _normal(g, (total, page, hk, d), dt)
    s["vp"] = _normal(g, (total, page, hk, d), dt)
    if c["op"] == "attn" and c["weights"]:
        cap = s["table"].shape[1] * page
        s["scores"] = torch.empty((c["batch"], hk, cap), device="cuda").exponential_(1.0, generator=g).pow_(3)
        s["scores_out"] = torch.zeros_like(s["scores"])
    if c["op"] == "shared":
        s["prefix_dev"] = _ints([c["prefix"]])
        if c["prefix"] % page:  # the copies of the page in which the prefix ends
            at = s["table"][:, c["prefix"] // page].long()
            for pool in (s["kp"], s["vp"]):
                pool[at, :c["prefix"] % page] = pool[at[0], :c["prefix"] % page]
    if own:  # the handle that a program makes once for its cache and keeps
        s["cache"] = mbg.PagedKV(s["kp"], s["vp"], s["table"], scores=s.get("scores"))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return {"tables": _assign, "rope": _rope, "attn": _attn, "prompt": _prompt, "shared": _shared}[state["op"]](state)


def _assign(s):
    if own:
        s["mbg"].gemv_kv_assign(s["cache"], s["pool"], s["lengths"], s["fresh_of"], s["starts"], s["slots"], s["seq"],
                                shared=s["shared"], lengths_out=s["lengths_after"], state_out=s["ring_at_after"])
    else:
        n, f, p = s["lengths"].long(), s["fresh_of"].long(), s["page"]
        ring, (at, count), size = s["ring"].long(), s["ring_at"].long(), s["total"]
        width, room = s["table"].shape[1], s["slots"].shape[0]
        over = f < 0
        f = torch.where(n + f <= width * p, f.clamp(min=0), 0)
        have = (n + p - 1) // p
        need = (n + f + p - 1) // p - have
        ends = need.cumsum(0)
        f = torch.where((need == 0) | (ends <= count), f, 0)
        f = torch.where(f.cumsum(0) <= room, f, 0)
        need = torch.where(f > 0, need, 0)
        # pages from the ring into the table, behind those that are there
        first = need.cumsum(0) - need
        col = torch.arange(width, device="cuda") - have[:, None]
        new = (col >= 0) & (col < need[:, None])
        from_ring = ring[(at + first[:, None] + torch.where(new, col, 0)) % size]
        s["table"].copy_(torch.where(new, from_ring, s["table"].long()))
        # pages of those that are over, back to the ring's end
        keep = s["shared"].long() // p
        gone = torch.where(over, (have - keep).clamp(min=0), 0)
        gone_ends = gone.cumsum(0)
        place = (torch.arange(size, device="cuda") - at - count) % size
        b = torch.searchsorted(gone_ends, place, right=True).clamp(max=len(n) - 1)
        page = s["table"][b, (keep[b] + place - gone_ends[b] + gone[b]).clamp(0, width - 1)]
        s["ring"].copy_(torch.where(place < gone_ends[-1], page, s["ring"]))
        # each token's sequence and slot
        token_ends = f.cumsum(0)
        t = torch.arange(room, device="cuda")
        b = torch.searchsorted(token_ends, t, right=True).clamp(max=len(n) - 1)
        live = t < token_ends[-1]
        s["slots"].copy_(torch.where(live, n[b] + t - token_ends[b] + f[b], -1))
        s["seq"].copy_(torch.where(live, b, 0))
        s["starts"][:1] = 0
        s["starts"][1:] = token_ends
        s["lengths_after"].copy_(torch.where(over, 0, n + f))
        taken = need.sum()
        s["ring_at_after"].copy_(torch.stack(((at + taken) % size, count - taken + gone_ends[-1])))
    return {"table": s["table"], "starts": s["starts"], "slots": s["slots"], "seq": s["seq"],
            "lengths": s["lengths_after"], "ring": s["ring"], "ring_at": s["ring_at_after"]}


def _rope(s):
    if own:
        s["mbg"].gemv_rope_append(s["cache"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"],
                                  q_out=s["q_out"], seq=s["seq"], norm=True, q_weight=s["q_weight"],
                                  k_weight=s["k_weight"], unit_offset=s["unit"], eps=1e-5)
    else:
        angle = s["positions"].double()[s["axis"]].T * s["freq"]               # [T, rot/2]: far positions need 64 bits
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        rot = s["rot"]

        def turn(x, weight):
            x = x.float()
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5) * (weight.float() + (1.0 if s["unit"] else 0.0))
            if s["pairs"]:
                a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            else:
                a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            first, second = a * cos - b * sin, a * sin + b * cos
            both = torch.stack((first, second), -1).flatten(-2) if s["pairs"] else torch.cat((first, second), -1)
            return torch.cat((both, x[..., rot:]), -1)

        s["q_out"].copy_(turn(s["q"], s["q_weight"]))
        slot = s["slots"].long()
        page = s["table"][s["seq"].long(), slot // s["page"]].long()
        s["kp"][page, slot % s["page"]] = turn(s["k"], s["k_weight"]).to(s["kp"].dtype)
        s["vp"][page, slot % s["page"]] = s["v"].float().to(s["vp"].dtype)
    return {"q": s["q_out"], "k": s["kp"], "v": s["vp"]}


def _visible(s, slot, n):
    """Which slots a token sees that is the last of n."""
    ok = slot < n
    return ok & ((slot >= n - s["window"]) | (slot < s["sinks"])) if s["window"] else ok


def _softmax(x, ok):
    x = torch.where(ok, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = x.sum(-1, keepdim=True)
    return x / torch.where(total == 0, 1.0, total)


def _attn(s):
    if own:
        s["mbg"].gemv_attn_paged(s["cache"], s["qv"], s["lengths"], out=s["out"], scale=s["scale"], window=s["window"],
                                 sinks=s["sinks"], accumulate=s["weights"], scores_out=s.get("scores_out"))
    else:
        b, hq, d = s["qv"].shape
        hk, page = s["kv_heads"], s["page"]
        at = s["table"].clamp(min=0).long()
        cap = at.shape[1] * page
        ok = _visible(s, torch.arange(cap, device="cuda"), s["lengths"].long()[:, None])[:, None, None]  # [B, 1, 1, cap]
        k = s["kp"][at].reshape(b, cap, hk, d).permute(0, 2, 3, 1).float()      # [B, Hkv, D, cap]
        p = _softmax(torch.matmul(s["qv"].float().reshape(b, hk, hq // hk, d) * s["scale"], k), ok)
        del k
        v = s["vp"][at].reshape(b, cap, hk, d).permute(0, 2, 1, 3).float()
        v = torch.where(ok.reshape(b, 1, cap, 1), v, 0.0)
        s["out"].copy_(torch.matmul(p, v).reshape(b, hq, d))
        if s["weights"]:
            live = ok[:, :, 0].expand(b, hk, cap)
            s["scores_out"].copy_(torch.where(live, s["scores"] + p.sum(2), s["scores_out"]))
    return {"out": s["out"], "scores": s.get("scores_out")}


def _cached(s, b, n, dtype):
    """K and V of sequence b's first n slots, [Hkv, n, D]."""
    t = torch.arange(n, device="cuda")
    page = s["table"][b, t // s["page"]].long()
    return (pool[page, t % s["page"]].to(dtype).transpose(0, 1) for pool in (s["kp"], s["vp"]))


def _prompt(s):
    if own:
        s["mbg"].gemv_attn_prompt(s["cache"], s["qv"], s["starts"], s["lengths"], out=s["out"], scale=s["scale"],
                                  window=s["window"], sinks=s["sinks"])
    else:
        hk, group = s["kv_heads"], s["q_heads"] // s["kv_heads"]
        done = 0
        for b, (m, n) in enumerate(s["spans"]):
            if m == 0:
                continue
            k, v = _cached(s, b, n, torch.float32)
            slot = torch.arange(n, device="cuda")
            step = max(1, min(m, 250_000_000 // (n * s["q_heads"])))  # tokens whose scores take 1 GB
            for i in range(0, m, step):
                c = min(step, m - i)
                q = s["qv"][done + i:done + i + c].float().reshape(c, hk, group, -1).permute(1, 0, 2, 3) * s["scale"]
                x = torch.matmul(q.reshape(hk, c * group, -1), k.transpose(1, 2)).reshape(hk, c, group, n)
                last = torch.arange(n - m + i + 1, n - m + i + c + 1, device="cuda")
                p = _softmax(x, _visible(s, slot, last[:, None])[None, :, None])
                o = torch.matmul(p.reshape(hk, c * group, n), v).reshape(hk, c, group, -1)
                s["out"][done + i:done + i + c] = o.permute(1, 0, 2, 3).reshape(c, hk * group, -1).to(s["out"].dtype)
            done += m
    return {"out": s["out"]}


def _shared(s):
    if own:
        s["mbg"].gemv_attn_shared(s["cache"], s["qv"], s["lengths"], s["prefix_dev"], out=s["out"], scale=s["scale"],
                                  window=s["window"], sinks=s["sinks"])
    else:
        b, hq, d = s["qv"].shape
        hk, page, pre = s["kv_heads"], s["page"], s["prefix"]
        group = hq // hk
        q = s["qv"].float().reshape(b, hk, group, d) * s["scale"]
        # the prefix once for all: scores [Hkv, B * group, prefix]
        k1, v1 = _cached(s, 0, pre, torch.float32)
        x1 = torch.matmul(q.transpose(0, 1).reshape(hk, b * group, d), k1.transpose(1, 2))
        x1 = x1.reshape(hk, b, group, pre).transpose(0, 1)
        # each sequence's own slots
        at = s["table"][:, pre // page:].clamp(min=0).long()
        own_slots = at.shape[1] * page
        k2 = s["kp"][at].reshape(b, own_slots, hk, d).permute(0, 2, 3, 1).float()
        x2 = torch.matmul(q, k2)
        slot = torch.cat((torch.arange(pre, device="cuda"), pre // page * page + torch.arange(own_slots, device="cuda")))
        n = s["lengths"].long()[:, None]
        ok = _visible(s, slot, n)
        ok[:, pre:] &= slot[pre:] >= pre
        p = _softmax(torch.cat((x1, x2), -1), ok[:, None, None])
        v2 = s["vp"][at].reshape(b, own_slots, hk, d).permute(0, 2, 1, 3).float()
        v2 = torch.where(ok[:, None, pre:, None], v2, 0.0)
        o = torch.matmul(p[..., :pre].transpose(0, 1).reshape(hk, b * group, pre), v1).reshape(hk, b, group, d)
        s["out"].copy_((o.transpose(0, 1) + torch.matmul(p[..., pre:], v2)).reshape(b, hq, d))
    return {"out": s["out"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers: nothing is computed that could be off
    if case["op"] == "prompt" and work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    return {"attn": _attn64, "rope": _rope64, "prompt": _prompt64, "shared": _shared64}[case["op"]](s)


def _row64(s, q, b, n):
    """Attention of one token's query heads [Hq, D], sequence b's last of n slots: out, weights, their slots."""
    hk = s["kv_heads"]
    lo = max(0, n - s["window"]) if s["window"] else 0
    at = torch.cat((torch.arange(min(lo, s["sinks"])), torch.arange(lo, n))).cuda()
    page = s["table"][b, at // s["page"]].long()
    k, v = (pool[page, at % s["page"]].double() for pool in (s["kp"], s["vp"]))
    x = torch.einsum("hgd,nhd->hgn", q.double().reshape(hk, -1, q.shape[-1]), k) * s["scale"]
    p = torch.softmax(x, -1)
    return torch.einsum("hgn,nhd->hgd", p, v).reshape(q.shape), p, at


def _attn64(s):
    out = torch.zeros(s["qv"].shape, dtype=torch.float64, device="cuda")
    sums = s["scores_out"].double() if s["weights"] else None
    for i, (_, n) in enumerate(s["spans"]):
        if n == 0:
            continue
        out[i], p, at = _row64(s, s["qv"][i], i, n)
        if sums is not None:
            sums[i][:, at] = s["scores"][i][:, at].double() + p.sum(1)
    return {"out": out, "scores": sums}


def _shared64(s):
    out = torch.zeros(s["qv"].shape, dtype=torch.float64, device="cuda")
    for i, (_, n) in enumerate(s["spans"]):
        if n > 0:
            out[i] = _row64(s, s["qv"][i], i, n)[0]
    return {"out": out}


def _prompt64(s):
    out = torch.zeros(s["qv"].shape, dtype=torch.float64, device="cuda")
    hk, group = s["kv_heads"], s["q_heads"] // s["kv_heads"]
    done = 0
    for b, (m, n) in enumerate(s["spans"]):
        if m == 0:
            continue
        k, v = _cached(s, b, n, torch.float64)
        for i in range(0, m, 512):
            c = min(512, m - i)
            last = n - m + i + c                       # slots that any of these tokens sees
            first = max(0, last - c - s["window"]) if s["window"] else 0
            at = torch.cat((torch.arange(min(first, s["sinks"])), torch.arange(first, last))).cuda()
            mine = torch.arange(last - c, last, device="cuda")[:, None]
            gap = mine - at
            hidden = gap < 0
            if s["window"]:
                hidden |= (gap >= s["window"]) & (at >= s["sinks"])
            for h in range(hk):
                q = s["qv"][done + i:done + i + c, h * group:(h + 1) * group].double()
                x = torch.einsum("tgd,nd->gtn", q, k[h, at]) * s["scale"]
                p = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
                out[done + i:done + i + c, h * group:(h + 1) * group] = torch.einsum("gtn,nd->tgd", p, v[h, at])
        done += m
    return {"out": out}


def _rope64(s):
    rot, half = s["rot"], s["rot"] // 2
    first = torch.arange(half, device="cuda") * (2 if s["pairs"] else 1)
    second = first + (1 if s["pairs"] else half)
    turns = torch.stack([s["positions"][int(a)].double() * f for a, f in zip(s["axis"].tolist(), s["freq"])], -1)
    spin = torch.polar(torch.ones_like(turns), turns)[:, None]

    def turn(x, weight):
        x = x.double()
        w = weight.double() + 1.0 if s["unit"] else weight.double()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w
        z = torch.complex(x[..., first], x[..., second]) * spin
        x[..., first], x[..., second] = z.real, z.imag
        return x

    kp, vp = s["kp"].double(), s["vp"].double()
    slot = s["slots"].long()
    page = s["table"][s["seq"].long(), slot // s["page"]].long()
    kp[page, slot % s["page"]] = turn(s["k"], s["k_weight"])
    vp[page, slot % s["page"]] = s["v"].double()
    return {"q": turn(s["q"], s["q_weight"]), "k": kp, "v": vp}
