"""The decode-step operators: attention of one new token over a paged cache, eviction from that cache
by accumulated attention weight, rotary positions with the append to the cache, and the norms around a
block with its gate and residual.

Each case is one call (eviction: the plan and its moves) as a decode or prefill program makes it.  The
plain forms below are elementary torch operations in 32 bits; with ``own`` the calls go to
``memory_bound_gemv_gb300``.
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
        # one user's first tokens: 32 query heads over 8 cached heads of 128 (the 4096-wide shapes)
        dict(name="attn_first_tokens", op="attn", type="f16", batch=1, q_heads=32, kv_heads=8, dim=128,
             longest=77, page=16, window=0, weights=False),
        # a serving batch of ragged lengths that also keeps the weights eviction goes by
        dict(name="attn_batch_weights", op="attn", type="bf16", batch=48, q_heads=32, kv_heads=8, dim=128,
             longest=6000, page=16, window=0, weights=True),
        # one user with a very long context: the work of a single row has to be split over the GPU
        dict(name="attn_long", op="attn", type="f16", batch=1, q_heads=32, kv_heads=8, dim=128,
             longest=131001, page=64, window=0, weights=False),
        # no shared heads, a head of 80, pages of 24 that end inside a tile, a sliding window, an empty row
        dict(name="attn_window_odd", op="attn", type="bf16", batch=11, q_heads=14, kv_heads=14, dim=80,
             longest=5003, page=24, window=1000, weights=False),
        # one decode step: the FP32 output of the QKV product, rotated and appended
        dict(name="rope_step", op="rope", type="f16", source="f32", tokens=1, batch=1, q_heads=32, kv_heads=8,
             dim=128, sections="64", pairs=False, page=16, far=4000),
        # a step of a batch at far positions, with text, height and width axes
        dict(name="rope_batch_far", op="rope", type="bf16", source="f32", tokens=64, batch=64, q_heads=32,
             kv_heads=8, dim=128, sections="16,24,24", pairs=False, page=16, far=1000000),
        # a video prompt: time, height and width positions, three sequences in one call
        dict(name="rope_video_prompt", op="rope", type="bf16", source="bf16", tokens=7001, batch=3, q_heads=32,
             kv_heads=8, dim=128, sections="16,24,24", pairs=True, page=32, far=9000),
        # a decode step of a batch at its budget: one token more than may stay
        dict(name="evict_step", op="evict", type="f16", batch=16, kv_heads=8, dim=128, longest=2049, shortest=2049,
             keep=2048, sinks=4, recent=256, page=16),
        # prompts just read, cut to the budget at once
        dict(name="evict_prompt", op="evict", type="bf16", batch=4, kv_heads=8, dim=128, longest=30011, shortest=1000,
             keep=4096, sinks=4, recent=512, page=64),
        # the step between two products of one user: 4096 wide, FP32 in, the next product's binary16 out
        dict(name="norm_step", op="norm", y="f32", x="f32", h="f16", rows=1, width=4096, kind="rms", post=True,
             gate="none"),
        # adaptive norms: gate, scale and shift of each row, LayerNorm, 14336 wide
        dict(name="norm_adaptive", op="norm", y="f16", x="f16", h="f16", rows=331, width=14336, kind="layer",
             post=False, gate="row"),
        # a prompt through a block with a norm before and after and one learned gate
        dict(name="norm_prompt", op="norm", y="bf16", x="bf16", h="bf16", rows=8192, width=4096, kind="rms",
             post=True, gate="shared"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "evict", "norm"])
    while True:
        if op == "attn":
            hk = rng.choice([1, 2, 4, 5, 8, 14])
            c = dict(op=op, type=rng.choice(["f16", "bf16"]), batch=_log(rng, 1, 96),
                     q_heads=hk * rng.choice([1, 2, 4, 5, 7, 8, 12, 16]), kv_heads=hk,
                     dim=rng.choice([64, 80, 96, 128, 128, 192, 256]), longest=_log(rng, 1, 131072),
                     page=rng.choice([1, 8, 16, 16, 24, 64, 128]), window=rng.choice([0, 0, _log(rng, 1, 8192)]),
                     weights=rng.random() < 0.4)
        elif op == "rope":
            dim = rng.choice([64, 96, 128, 128, 256])
            half = dim // 2
            a = rng.randint(1, half - 2)
            b = rng.randint(1, half - a - 1)
            tokens = _log(rng, 1, 8000)
            c = dict(op=op, type=rng.choice(["f16", "bf16"]), source=rng.choice(["f32", "f16", "bf16"]),
                     tokens=tokens, batch=rng.randint(1, min(tokens, 64)), q_heads=8 * rng.choice([1, 4, 5]),
                     kv_heads=rng.choice([1, 4, 8]), dim=dim,
                     sections=rng.choice(["%d" % half, "%d" % max(1, half // 2), "%d,%d,%d" % (a, b, half - a - b)]),
                     pairs=rng.random() < 0.5, page=rng.choice([8, 16, 24, 64]), far=_log(rng, 100, 2000000))
        elif op == "evict":
            longest = _log(rng, 40, 131072)
            keep = max(8, int(longest * rng.choice([rng.uniform(0.02, 0.5), rng.uniform(0.9, 0.999)])))
            c = dict(op=op, type=rng.choice(["f16", "bf16"]), batch=_log(rng, 1, 48), kv_heads=rng.choice([1, 2, 8]),
                     dim=rng.choice([64, 80, 128, 256]), longest=longest,
                     shortest=rng.choice([longest, rng.randint(1, longest)]), keep=keep,
                     sinks=rng.randint(0, 4), recent=rng.randint(1, max(1, keep // 4)), page=rng.choice([8, 16, 24, 64]))
        else:
            c = dict(op=op, y=rng.choice(["f32", "f16", "bf16"]), x=rng.choice(["f32", "f16", "bf16"]),
                     h=rng.choice(["f16", "bf16", "f32"]), rows=_log(rng, 1, 8192), width=_log(rng, 64, 16384),
                     kind=rng.choice(["rms", "layer"]), post=rng.random() < 0.6,
                     gate=rng.choice(["none", "shared", "row"]))
        pool = c["batch"] * c["longest"] * c["kv_heads"] * c["dim"] * 4 if op in ("attn", "evict") else 0
        if work(c)["bytes"] <= 5.0e8 and pool <= 5.3e8:
            return c


def _lengths(c):
    """The case's ragged lengths, in order: from the longest down in equal steps; with a window the last row is empty."""
    if c["op"] == "evict":
        lo, hi, n = c["shortest"], c["longest"], c["batch"]
        return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]
    got = [max(1, c["longest"] * (c["batch"] - i) // c["batch"]) for i in range(c["batch"])]
    if c["window"] and c["batch"] > 1:
        got[-1] = 0
    return got


def work(case):
    c = case
    if c["op"] == "attn":
        seen = sum(min(n, c["window"] or n) for n in _lengths(c))
        pages = sum(-(-min(n, c["window"] or n) // c["page"]) for n in _lengths(c))
        b = seen * c["kv_heads"] * c["dim"] * 4 + 4 * c["batch"] * c["q_heads"] * c["dim"] + 4 * (pages + c["batch"])
        if c["weights"]:
            b += 8 * seen * c["kv_heads"]
        return {"bytes": b, "flops": 4.0 * seen * c["q_heads"] * c["dim"]}
    if c["op"] == "rope":
        n = c["tokens"] * (c["q_heads"] + 2 * c["kv_heads"]) * c["dim"]
        axes = c["sections"].count(",") + 1
        return {"bytes": n * (SIZE[c["source"]] + 2) + 4 * c["tokens"] * (axes + 2),
                "flops": 3.0 * c["tokens"] * (c["q_heads"] + c["kv_heads"]) * c["dim"]}
    if c["op"] == "evict":
        b = f = 0
        for n in _lengths(c):
            over = max(0, n - c["keep"])
            # about this many kept tokens lie behind the budget's end: the recent ones, and an even share of the others
            moves = 0 if not over else min(over, c["recent"]) + max(0, c["keep"] - c["recent"]) * max(0, over - c["recent"]) // n
            b += c["kv_heads"] * (8 * n + moves * (8 * c["dim"] + 16 + 8))
            f += c["kv_heads"] * n
        return {"bytes": b + 8 * c["batch"], "flops": f}
    n = c["rows"] * c["width"]
    b = n * (SIZE[c["y"]] + 2 * SIZE[c["x"]] + SIZE[c["h"]])
    if c["gate"] == "row":
        b += 3 * n * SIZE[c["x"]]  # gate, scale and shift of each row
    return {"bytes": b, "flops": 12.0 * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, scale, generator=g).to(dtype)


def _pages(c, lengths, rng, spare=3):
    """A page table over a pool in which the sequences' pages lie scattered; -1 where a sequence has none."""
    need = [-(-n // c["page"]) for n in lengths]
    width = max(need) + spare
    total = sum(need) + 7
    order = list(range(total))
    rng.shuffle(order)
    table = torch.full((len(lengths), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table.cuda(), total, width * c["page"]


def prepare(case, seed):
    c, g, rng = case, _gen(seed), random.Random(seed)
    s = dict(case)
    if own:
        import memory_bound_gemv_gb300 as mbg

        s["mbg"] = mbg
    if c["op"] == "norm":
        m, n, xt = c["rows"], c["width"], DT[c["x"]]
        s["yv"] = _normal(g, (m, n), DT[c["y"]], 1.7)
        s["residual"] = _normal(g, (m, n), xt, 3.0)
        s["post_weight"] = (1.0 + _normal(g, (n,), torch.float32, 0.2)).to(xt) if c["post"] else None
        if c["gate"] == "row":
            s["gate_v"] = _normal(g, (m, n), xt, 0.5)
            s["pre_weight"] = _normal(g, (m, n), xt, 0.2)  # 1 + scale
            s["pre_bias"] = _normal(g, (m, n), xt, 0.3)
        else:
            s["gate_v"] = _normal(g, (n,), xt, 0.5) if c["gate"] == "shared" else None
            s["pre_weight"] = (1.0 + _normal(g, (n,), torch.float32, 0.2)).to(xt)
            s["pre_bias"] = None
        s["alpha"] = 0.7
        s["out"] = torch.empty((m, n), dtype=xt, device="cuda")
        s["hv"] = torch.empty((m, n), dtype=DT[c["h"]], device="cuda")
        return s
    dt, hk, d = DT[c["type"]], c["kv_heads"], c["dim"]
    if c["op"] == "rope":
        t, n, hq = c["tokens"], c["batch"], c["q_heads"]
        counts = [t // n + (1 if i < t % n else 0) for i in range(n)]
        starts = [(37 * i + 11) % 200 for i in range(n)]
        lengths = [a + b for a, b in zip(starts, counts)]
        s["seq"] = torch.repeat_interleave(torch.arange(n), torch.tensor(counts)).to(torch.int32).cuda()
        s["slots"] = torch.cat([torch.arange(a, a + b) for a, b in zip(starts, counts)]).to(torch.int32).cuda()
        axes = c["sections"].count(",") + 1
        s["positions"] = torch.randint(0, c["far"], (axes, t), generator=g, device="cuda", dtype=torch.int32)
        qkv = _normal(g, (t, (hq + 2 * hk), d), DT[c["source"]], 1.3)  # the QKV product's output, seen as three parts
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        parts = [int(x) for x in c["sections"].split(",")]
        rot = 2 * sum(parts)
        s["rot"] = rot
        s["freq"] = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
        s["axis"] = torch.repeat_interleave(torch.arange(len(parts)), torch.tensor(parts)).cuda()
        s["q_out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")
    else:
        lengths = _lengths(c)
        rng.shuffle(lengths)
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    s["table"], total, cap = _pages(c, lengths, rng)
    s["kp"] = _normal(g, (total, c["page"], hk, d), dt)
    s["vp"] = _normal(g, (total, c["page"], hk, d), dt)
    if c["op"] == "attn":
        s["qv"] = _normal(g, (c["batch"], c["q_heads"], d), dt, 1.6)
        s["out"] = torch.empty_like(s["qv"])
        s["scale"] = d ** -0.5
        if c["weights"]:
            s["scores"] = torch.empty((c["batch"], hk, cap), device="cuda").exponential_(1.0, generator=g).pow_(3)
            s["scores_out"] = torch.zeros_like(s["scores"])
    if c["op"] == "evict":
        # what earlier steps have summed up: a few tokens with much, most with little, many equal zeros
        sc = torch.empty((c["batch"], hk, cap), device="cuda").exponential_(1.0, generator=g).pow_(4)
        s["scores"] = torch.where(torch.rand(sc.shape, generator=g, device="cuda") < 0.1, 0.0, sc)
        # numbers of the tokens in the slots: earlier evictions have mixed their order within a few places
        near = torch.arange(cap, device="cuda") + 9.0 * torch.rand(sc.shape, generator=g, device="cuda")
        s["stamps"] = near.argsort(dim=-1).to(torch.int32)
        s["scores_kept"], s["stamps_kept"] = s["scores"].clone(), s["stamps"].clone()
        s["lengths_kept"] = s["lengths"].clone()
        most = max(1, min(c["keep"], cap - c["keep"]))
        s["moves"] = torch.full((c["batch"], hk, most, 2), -1, dtype=torch.int32, device="cuda")
        s["counts"] = torch.zeros((c["batch"], hk), dtype=torch.int32, device="cuda")
    if own:  # the handle that a program makes once for its cache and keeps
        s["cache"] = mbg.PagedKV(s["kp"], s["vp"], s["table"], scores=s.get("scores"), stamps=s.get("stamps"))
        if c["op"] == "evict":
            s["kept"] = mbg.PagedKV(s["kp"], s["vp"], s["table"], scores=s["scores_kept"], stamps=s["stamps_kept"])
        if c["op"] == "rope":
            s["rope"] = mbg.RopeTable(rot, sections=parts, theta=10000.0, pairs=c["pairs"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return {"attn": _attn, "rope": _rope, "evict": _evict, "norm": _norm}[state["op"]](state)


def _attn(s):
    if own:
        s["mbg"].gemv_attn_paged(s["cache"], s["qv"], s["lengths"], out=s["out"], scale=s["scale"], window=s["window"],
                                 accumulate=s["weights"], scores_out=s.get("scores_out"))
    else:
        b, hq, d = s["qv"].shape
        hk, page = s["kv_heads"], s["page"]
        at = s["table"].clamp(min=0).long()
        cap = at.shape[1] * page
        slot = torch.arange(cap, device="cuda")
        n = s["lengths"].long()[:, None]
        first = (n - s["window"]).clamp(min=0) if s["window"] else torch.zeros_like(n)
        ok = ((slot < n) & (slot >= first))[:, None, None]                      # [B, 1, 1, cap]
        k = s["kp"][at].reshape(b, cap, hk, d).permute(0, 2, 3, 1).float()      # [B, Hkv, D, cap]
        x = torch.matmul(s["qv"].float().reshape(b, hk, hq // hk, d) * s["scale"], k)
        del k
        x = torch.where(ok, x, -math.inf)
        top = x.amax(-1, keepdim=True)
        x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        total = x.sum(-1, keepdim=True)
        p = x / torch.where(total == 0, 1.0, total)
        del x
        v = s["vp"][at].reshape(b, cap, hk, d).permute(0, 2, 1, 3).float()
        v = torch.where(ok.reshape(b, 1, cap, 1), v, 0.0)
        s["out"].copy_(torch.matmul(p, v).reshape(b, hq, d))
        if s["weights"]:
            live = ok[:, :, 0].expand(b, hk, cap)
            s["scores_out"].copy_(torch.where(live, s["scores"] + p.sum(2), s["scores_out"]))
    return {"out": s["out"], "scores": s.get("scores_out")}


def _rope(s):
    if own:
        s["mbg"].gemv_rope_append(s["cache"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"],
                                  q_out=s["q_out"], seq=s["seq"])
    else:
        angle = s["positions"].double()[s["axis"]].T * s["freq"]               # [T, rot/2]: far positions need 64 bits
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        rot = s["rot"]

        def turn(x):
            x = x.float()
            if s["pairs"]:
                a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            else:
                a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            first, second = a * cos - b * sin, a * sin + b * cos
            both = torch.stack((first, second), -1).flatten(-2) if s["pairs"] else torch.cat((first, second), -1)
            return torch.cat((both, x[..., rot:]), -1)

        s["q_out"].copy_(turn(s["q"]))
        slot = s["slots"].long()
        page = s["table"][s["seq"].long(), slot // s["page"]].long()
        s["kp"][page, slot % s["page"]] = turn(s["k"]).to(s["kp"].dtype)
        s["vp"][page, slot % s["page"]] = s["v"].float().to(s["vp"].dtype)
    return {"q": s["q_out"], "k": s["kp"], "v": s["vp"]}


def _evict(s):
    if own:
        s["mbg"].gemv_kv_evict_plan(s["cache"], s["lengths"], s["keep"], sinks=s["sinks"], recent=s["recent"],
                                    moves=s["moves"], counts=s["counts"])
        s["mbg"].gemv_kv_evict_apply(s["kept"], s["moves"], s["counts"], s["lengths_kept"], s["keep"])
    else:
        n, keep = s["lengths"].long()[:, None, None], s["keep"]
        score, stamp = s["scores"], s["stamps"]
        b, hk, cap = score.shape
        slot = torch.arange(cap, device="cuda")
        ok = (slot < n).expand(b, hk, cap)
        newest = torch.where(ok, stamp, -1).amax(-1, keepdim=True)
        safe = (stamp < s["sinks"]) | (stamp > newest - s["recent"])
        # order: protected ones, then the larger score, then the lower slot; slots past the length last
        by_score = torch.sort(score, dim=-1, descending=True, stable=True).indices
        klass = torch.where(ok, torch.where(safe, 2, 1), 0).gather(-1, by_score)
        order = by_score.gather(-1, torch.sort(klass, dim=-1, descending=True, stable=True).indices)
        rank = torch.empty_like(order).scatter_(-1, order, slot.expand(b, hk, cap))
        kept = ok & (rank < keep)
        hole, mover = ok & ~kept & (slot < keep), kept & (slot >= keep)
        s["counts"].copy_(mover.sum(-1))
        bi, hi, dst = hole.nonzero(as_tuple=True)     # both lists ascend in slot within a row, and are as long
        _, _, src = mover.nonzero(as_tuple=True)
        place = (hole.cumsum(-1) - 1)[bi, hi, dst]
        s["moves"][bi, hi, place] = torch.stack((src, dst), -1).to(torch.int32)
        page = s["page"]
        ps, pd = s["table"][bi, src // page].long(), s["table"][bi, dst // page].long()
        for pool in (s["kp"], s["vp"]):
            pool[pd, dst % page, hi] = pool[ps, src % page, hi]
        for kept_of, old in ((s["scores_kept"], score), (s["stamps_kept"], stamp)):
            kept_of[bi, hi, dst] = old[bi, hi, src]
        s["lengths_kept"].copy_(s["lengths"].clamp(max=keep))
    return {"moves": s["moves"], "counts": s["counts"], "lengths": s["lengths_kept"], "k": s["kp"], "v": s["vp"],
            "scores": s["scores_kept"], "stamps": s["stamps_kept"]}


def _norm(s):
    adaptive = s["gate"] == "row"
    if own:
        s["mbg"].gemv_norm_residual(s["yv"], s["residual"], post=s["post"], post_weight=s["post_weight"],
                                    gate=s["gate_v"], alpha=s["alpha"], pre_weight=s["pre_weight"],
                                    pre_bias=s["pre_bias"], kind=s["kind"], unit_offset=adaptive, eps=1e-5,
                                    out=s["out"], h=s["hv"])
    else:
        def norm(x):
            if s["kind"] == "layer":
                x = x - x.mean(-1, keepdim=True)
            return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)

        u = s["yv"].float()
        if s["post"]:
            u = norm(u) * s["post_weight"].float()
        if s["gate_v"] is not None:
            u = u * s["gate_v"].float()
        x = s["residual"].float() + s["alpha"] * u
        s["out"].copy_(x)
        h = norm(x) * (s["pre_weight"].float() + (1.0 if adaptive else 0.0))
        if s["pre_bias"] is not None:
            h = h + s["pre_bias"].float()
        s["hv"].copy_(h)
    return {"x": s["out"], "h": s["hv"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "evict":
        return None  # selections and copies: nothing is computed
    s = prepare(case, seed)
    return {"attn": _attn64, "rope": _rope64, "norm": _norm64}[case["op"]](s)


def _attn64(s):
    b, hq, d = s["qv"].shape
    hk, page, group = s["kv_heads"], s["page"], hq // s["kv_heads"]
    out = torch.zeros((b, hq, d), dtype=torch.float64, device="cuda")
    sums = s["scores_out"].double() if s["weights"] else None
    for i, n in enumerate(s["lengths"].tolist()):
        lo = max(0, n - s["window"]) if s["window"] else 0
        if n == lo:
            continue
        at = torch.arange(lo, n, device="cuda")
        pages = s["table"][i, at // page].long()
        for j in range(hk):
            k, v = s["kp"][pages, at % page, j].double(), s["vp"][pages, at % page, j].double()
            q = s["qv"][i, j * group:(j + 1) * group].double()
            p = torch.softmax(q @ k.T * s["scale"], -1)
            out[i, j * group:(j + 1) * group] = p @ v
            if sums is not None:
                sums[i, j, lo:n] = s["scores"][i, j, lo:n].double() + p.sum(0)
    return {"out": out, "scores": sums}


def _rope64(s):
    rot, half = s["rot"], s["rot"] // 2
    first = torch.arange(half, device="cuda") * (2 if s["pairs"] else 1)
    second = first + (1 if s["pairs"] else half)
    turns = torch.stack([s["positions"][int(a)].double() * f for a, f in zip(s["axis"].tolist(), s["freq"])], -1)
    spin = torch.polar(torch.ones_like(turns), turns)[:, None]

    def turn(x):
        x = x.double().clone()
        z = torch.complex(x[..., first], x[..., second]) * spin
        x[..., first], x[..., second] = z.real, z.imag
        return x

    kp, vp = s["kp"].double(), s["vp"].double()
    slot = s["slots"].long()
    page = s["table"][s["seq"].long(), slot // s["page"]].long()
    kp[page, slot % s["page"]] = turn(s["k"])
    vp[page, slot % s["page"]] = s["v"].double()
    return {"q": turn(s["q"]), "k": kp, "v": vp}


def _norm64(s):
    def norm(x):
        if s["kind"] == "layer":
            x = x - x.mean(-1, keepdim=True)
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)

    u = s["yv"].double()
    if s["post"]:
        u = norm(u) * s["post_weight"].double()
    if s["gate_v"] is not None:
        u *= s["gate_v"].double()
    x = s["residual"].double() + s["alpha"] * u
    w = s["pre_weight"].double() + (1.0 if s["gate"] == "row" else 0.0)
    h = norm(x) * w
    if s["pre_bias"] is not None:
        h += s["pre_bias"].double()
    return {"x": x, "h": h}
