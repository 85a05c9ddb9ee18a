"""The decode-step example: all operators and the INT4 GEMVs in one step, against a plain model in 64 bits.

Tolerance: per layer eight vectors are rounded to binary16 on the way (h twice
in, q, k, v, the attention's output, the MLP's inner vector, h of the next
block), each off by at most 2^-11 relative, and a product of normalised
vectors keeps that relative to the row's norm; the residual stream of two
layers is therefore within 2 * 8 * 2^-11 = 0.8 % of its norm, and errors of
earlier tokens enter through the cache, at most doubling it.
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
import decode_step  # noqa: E402

BOUND = 2 * 2 * 8 * 2.0 ** -11


class Plain:
    """The same model in 64 bits; which tokens stay is read from the example's stamps."""

    def __init__(self, m):
        self.m = m
        self.w = [{n: mbg.gemv_dequant_q4(*l[n]).double() for n in ("qkv", "out", "up", "down")} for l in m.layers]
        self.kv = [dict() for _ in m.layers]  # token number -> (k, v) [kv_heads, dim]
        half = m.dim // 2
        self.freq = 10000.0 ** (-2.0 * torch.arange(half, dtype=torch.float64, device="cuda") / m.dim)

    def norm(self, x, w):
        return x / torch.sqrt((x * x).mean() + 1e-6) * w.double()

    def turn(self, x, position):
        half = self.m.dim // 2
        ang = position[self.m.rope.axis.long()].double() * self.freq
        a, b = x[..., :half], x[..., half:]
        return torch.cat((a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()), -1)

    def step(self, x, position, token, kept):
        """kept[layer][head]: tokens in the cache besides this one."""
        m = self.m
        qd, kd, g = m.q_heads * m.dim, m.kv_heads * m.dim, m.q_heads // m.kv_heads
        h = self.norm(x, m.layers[0]["norms"][3])
        for i, w in enumerate(self.w):
            norms = m.layers[i]["norms"]
            q, k, v = (t.view(-1, m.dim) for t in (w["qkv"] @ h).split((qd, kd, kd)))
            q, k = self.turn(q, position), self.turn(k, position)
            self.kv[i][token] = (k, v)
            o = []
            for head in range(m.q_heads):
                seen = kept[i][head // g] + [token]
                ks = torch.stack([self.kv[i][t][0][head // g] for t in seen])
                vs = torch.stack([self.kv[i][t][1][head // g] for t in seen])
                o.append(torch.softmax(ks @ q[head] / math.sqrt(m.dim), 0) @ vs)
            x = x + self.norm(w["out"] @ torch.cat(o), norms[0])
            h = self.norm(x, norms[1])
            x = x + self.norm(w["down"] @ torch.relu(w["up"] @ h).square(), norms[2])
            h = self.norm(x, m.layers[(i + 1) % len(self.w)]["norms"][3])
        return x


@pytest.mark.parametrize("graph", [False, True])
def test_steps_match_the_plain_model_through_evictions(graph):
    m = decode_step.Decoder(layers=2, keep=24, sinks=1, recent=6)
    plain = Plain(m)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    run = m.step
    for token in range(40):
        x = torch.empty(1, m.hidden, device="cuda").normal_(generator=g)
        m.x.copy_(x)
        m.positions[1:].copy_(torch.tensor([[token % 7], [token // 7]], dtype=torch.int32))
        kept = [[l["cache"].stamps[0, h, :int(l["lengths"])].tolist() for h in range(m.kv_heads)] for l in m.layers]
        for tokens in (t for layer in kept for t in layer):
            assert len(set(tokens)) == len(tokens) == min(token, 24)  # no token twice, none lost
            if token > 24:
                assert 0 in tokens and set(range(token - 6, token)) <= set(tokens)  # the sink and the recent ones
        want = plain.step(x[0].double(), m.positions[:, 0].clone(), token, kept)
        if graph and token == 1:
            saved = [(l["cache"].k.clone(), l["cache"].v.clone(), l["cache"].scores.clone(), l["cache"].stamps.clone(),
                      l["lengths"].clone()) for l in m.layers]
            state = (m.token.clone(), m.positions.clone())
            captured = m.capture()
            for l, s in zip(m.layers, saved):  # a capture runs nothing, but leaves nothing to chance
                for t, old in zip((l["cache"].k, l["cache"].v, l["cache"].scores, l["cache"].stamps, l["lengths"]), s):
                    t.copy_(old)
            m.token.copy_(state[0]), m.positions.copy_(state[1])
            run = captured.replay
        run()
        assert float((m.x[0].double() - want).norm() / want.norm()) < BOUND, token
    assert mbg.gemv_get_device_error() == mbg.OK
    assert all(int(l["lengths"]) == 24 for l in m.layers)


def test_the_command_runs():
    sys_argv, sys.argv = sys.argv, ["decode_step.py", "--tokens", "90", "--keep", "40"]
    try:
        assert decode_step.main() == 0
    finally:
        sys.argv = sys_argv
