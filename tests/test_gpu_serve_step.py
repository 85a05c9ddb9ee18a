"""The serving example: pages, normed append, prompt, windowed and shared attention together, against a plain model
in 64 bits.

Tolerance: per layer eight vectors are rounded to binary16 on the way (h, the product's q, k and v, the turned q and k, the
attention's output, the product's output), each off by at most 2^-11 relative (the library product's own sums are
finer), and a product of normalised vectors keeps that relative to the row's norm; the two layers' residual is
therefore within 2 * 8 * 2^-11 = 0.8 % of its norm.  Errors of earlier tokens enter through the cache, at most doubling it; a
step's input is the example's own output, so that steps do not add up.
"""

import math
import os
import sys

import pytest

import memory_bound_gemv_gb300 as mbg

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import serve_batch  # noqa: E402

BOUND = 2 * 2 * 8 * 2.0 ** -11


class Plain:
    """Each request by itself: all inputs so far through both layers in 64 bits."""

    def __init__(self, m):
        self.m = m
        half = m.dim // 2
        self.freq = 10000.0 ** (-2.0 * torch.arange(half, dtype=torch.float64, device="cuda") / m.dim)

    def norm(self, x, w):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()

    def turn(self, x):
        half = self.m.dim // 2
        ang = torch.arange(x.shape[0], device="cuda")[:, None, None] * self.freq
        a, b = x[..., :half], x[..., half:]
        return torch.cat((a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()), -1)

    def __call__(self, x):
        m, x, n = self.m, x.double(), x.shape[0]
        gap = torch.arange(n, device="cuda")[:, None] - torch.arange(n, device="cuda")
        for w in m.layers:
            qkv = (self.norm(x, w["norm"]) @ w["qkv"].double().T).view(n, -1, m.dim)
            q, k, v = qkv.split((m.q_heads, m.kv_heads, m.kv_heads), dim=1)
            q, k = self.turn(self.norm(q, w["q_norm"])), self.turn(self.norm(k, w["k_norm"]))
            k, v = (t.repeat_interleave(m.q_heads // m.kv_heads, 1) for t in (k, v))
            s = torch.einsum("thd,shd->hts", q, k) / math.sqrt(m.dim)
            hidden = gap < 0
            if w["window"]:
                hidden = hidden | ((gap >= w["window"]) & (torch.arange(n, device="cuda") >= m.sinks))
            o = torch.einsum("hts,shd->thd", torch.softmax(s.masked_fill(hidden, -math.inf), -1), v)
            x = x + o.reshape(n, -1) @ w["out"].double().T
        return x


@pytest.mark.parametrize("graph", [False, True])
def test_requests_behind_one_prompt_match_the_plain_model(graph):
    m = serve_batch.Server(requests=3, longest=160)
    plain = Plain(m)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)

    def normal(*shape):
        return torch.empty(shape, device="cuda").normal_(generator=g)

    def near(got, want, what):
        err = (got.double() - want).norm(dim=-1) / want.norm(dim=-1)
        assert float(err.max()) < BOUND, (what, float(err.max()))

    first = normal(48, 256)
    near(m.read_prefix(first), plain(first), "prefix")
    counts = [5, 1, 30]
    own = list(normal(sum(counts), 256).split(counts))
    out = m.read_prompts(torch.cat(own), counts).split(counts)
    for b, x in enumerate(own):
        near(out[b], plain(torch.cat((first, x)))[48:], f"prompt of {b}")
    run = m.step
    m.x.copy_(normal(3, 256))
    for step in range(24):
        own = [torch.cat((x, m.x[b:b + 1])) for b, x in enumerate(own)]
        if graph and step == 2:
            run = m.capture().replay
        run()
        if step % 6 in (0, 5):
            for b, x in enumerate(own):
                near(m.x[b], plain(torch.cat((first, x)))[-1], f"step {step} of {b}")
    assert m.lengths.tolist() == [48 + n + 24 for n in counts]
    used = [-(-n // 16) - 3 for n in m.lengths.tolist()]
    assert m.pool.state.tolist() == [3 + sum(used), 64 - 3 - sum(used)]
    pages = [p for row in m.table.tolist() for p in row[3:] if p >= 0]
    assert len(set(pages)) == len(pages) == sum(used)
    # one request is over: its own pages come back, the shared ones do not
    m.fresh.copy_(torch.tensor([0, -1, 0], dtype=torch.int32))
    mbg.gemv_kv_assign(m.layers[0]["cache"], m.pool, m.lengths, m.fresh, shared=m.shared, tokens=0)
    assert m.lengths.tolist()[1] == 0 and int(m.pool.state[1]) == 64 - 3 - used[0] - used[2]
    assert mbg.gemv_get_device_error() == mbg.OK


def test_the_command_runs():
    sys_argv, sys.argv = sys.argv, ["serve_batch.py", "--requests", "5", "--tokens", "20"]
    try:
        assert serve_batch.main() == 0
    finally:
        sys.argv = sys_argv
