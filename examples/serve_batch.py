"""Serving a batch behind one system prompt, on this library's paged cache (products, and the MLP left out, are torch's).

Two layers with normed heads over one page table: one attends to everything, the other to a window and a few first
tokens.  Pages and slots come from the requests' lengths on the GPU; the system prompt is read once and its
pages are shared by all requests; then their own prompts, in one ragged call; then tokens one by one, as a CUDA
graph.  Weights are random.

    python examples/serve_batch.py --requests 8 --tokens 50
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_bound_gemv_gb300 as mbg  # noqa: E402


class Server:
    """Weights, caches and pages of `requests` requests."""

    def __init__(self, requests=3, q_heads=4, kv_heads=2, dim=64, hidden=256, page=16, pages=64, longest=256, windows=(0, 24),
                 sinks=3, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.empty(shape, device="cuda").normal_(0, scale, generator=g)

        self.requests, self.q_heads, self.kv_heads, self.dim, self.page, self.sinks = requests, q_heads, kv_heads, dim, page, sinks
        self.table = torch.full((requests, -(-longest // page)), -1, dtype=torch.int32, device="cuda")
        self.pool = mbg.PagePool(pages)
        self.layers = []
        for window in windows:
            shape = (pages, page, kv_heads, dim)
            cache = mbg.PagedKV(torch.zeros(shape, dtype=torch.float16, device="cuda"),
                                torch.zeros(shape, dtype=torch.float16, device="cuda"), self.table)
            self.layers.append({
                "cache": cache, "window": window,
                "qkv": normal((q_heads + 2 * kv_heads) * dim, hidden, scale=hidden ** -0.5).half(),
                "out": normal(hidden, q_heads * dim, scale=(q_heads * dim) ** -0.5).half(),
                "norm": 1 + normal(hidden, scale=0.1),
                "q_norm": 1 + normal(dim, scale=0.2), "k_norm": 1 + normal(dim, scale=0.2)})
        self.rope = mbg.RopeTable(dim)
        self.lengths = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.fresh = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.prefix = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.shared = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.x = torch.zeros(requests, hidden, device="cuda")  # the next tokens' inputs, and their outputs

    def forward(self, x, one_each):
        """self.fresh tokens of each request, x [tokens, hidden] in their order; returns the last residual."""
        starts, slots, seq = mbg.gemv_kv_assign(self.layers[0]["cache"], self.pool, self.lengths, self.fresh,
                                                shared=self.shared, tokens=x.shape[0])
        x = x.clone()
        for w in self.layers:
            cache = w["cache"]
            _, h = mbg.gemv_norm_residual(torch.zeros_like(x), x, pre_weight=w["norm"], out=x)
            qkv = (h @ w["qkv"].T).view(x.shape[0], -1, self.dim)
            q, k, v = qkv.split((self.q_heads, self.kv_heads, self.kv_heads), dim=1)
            q = mbg.gemv_rope_append(cache, q, k, v, slots[None], slots, self.rope, seq=seq, norm=True, q_weight=w["q_norm"],
                                     k_weight=w["k_norm"])
            if not one_each:
                o = mbg.gemv_attn_prompt(cache, q, starts, self.lengths, window=w["window"], sinks=self.sinks)
            elif w["window"]:
                o = mbg.gemv_attn_paged(cache, q, self.lengths, window=w["window"], sinks=self.sinks)
            else:
                o = mbg.gemv_attn_shared(cache, q, self.lengths, self.prefix)
            y = o.view(x.shape[0], -1) @ w["out"].T
            mbg.gemv_norm_residual(y, x, out=x, pre=False)
        return x

    def read_prefix(self, x):
        """A prompt that all requests begin with; its whole pages are shared."""
        self.fresh.zero_()
        self.fresh[0] = x.shape[0]
        out = self.forward(x, False)
        whole = x.shape[0] // self.page
        self.table[1:, :whole] = self.table[0, :whole]
        rest = x.shape[0] % self.page
        assert rest == 0, "the example shares whole pages"
        self.prefix.fill_(x.shape[0])
        self.shared.fill_(x.shape[0])
        self.lengths.fill_(x.shape[0])
        return out

    def read_prompts(self, x, counts):
        self.fresh.copy_(torch.tensor(counts, dtype=torch.int32))
        out = self.forward(x, False)
        self.fresh.fill_(1)
        return out

    def step(self):
        """One token for each request; its output is the next one's input."""
        self.x.copy_(self.forward(self.x, True))

    def capture(self):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=50)
    ap.add_argument("--prefix", type=int, default=160)
    a = ap.parse_args()
    longest = a.prefix + 40 + a.tokens + 2
    server = Server(requests=a.requests, longest=longest, pages=a.requests * (-(-longest // 16)) + 4)
    server.read_prefix(torch.randn(a.prefix // 16 * 16, 256, device="cuda"))
    counts = [3 + 5 * i % 37 for i in range(a.requests)]
    server.read_prompts(torch.randn(sum(counts), 256, device="cuda"), counts)
    server.x.normal_()
    server.step()
    graph = server.capture()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.tokens - 1):
        graph.replay()
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    status = mbg.gemv_get_device_error()
    print(f"{a.requests} requests, {a.tokens} tokens each: {t / max(1, a.tokens - 1) * 1e6:.1f} us per step, lengths "
          f"{server.lengths.tolist()}, {int(server.pool.state[1])} pages free, device status {mbg.STATUS[status]}")
    return 0 if status == mbg.OK and bool(server.x.isfinite().all()) else 1


if __name__ == "__main__":
    sys.exit(main())
