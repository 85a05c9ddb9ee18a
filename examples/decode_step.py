"""A decode step of a small transformer on this library's kernels (the MLP's activation and the counters are torch's).

Per layer: the QKV product (INT4 GEMV), rotary positions with three axes and
the append to the paged cache, attention of the new token with its weights
summed up, the output product, the norms around the block with the residual,
the MLP's two products, and the eviction of what the budget does not hold.
Every length, slot and position lives on the device, so a whole step is
captured into one CUDA graph and replayed; weights are random.

    python examples/decode_step.py --tokens 200 --keep 64
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_bound_gemv_gb300 as mbg  # noqa: E402


class Decoder:
    """Weights, caches and one token's state of `layers` layers for one sequence."""

    def __init__(self, layers=2, q_heads=8, kv_heads=2, dim=64, hidden=512, mlp=1024, page=16, keep=64, sinks=2,
                 recent=16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weights(rows, cols):
            w = torch.empty(rows, cols, device="cuda").normal_(0, cols ** -0.5, generator=g).half()
            return mbg.quantize(w, "q4")

        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        self.hidden, self.keep, self.sinks, self.recent = hidden, keep, sinks, recent
        self.layers = []
        pages = keep // page + 2  # one token more than the budget, before it is cut
        for _ in range(layers):
            shape = (pages, page, kv_heads, dim)
            slots = (1, kv_heads, pages * page)
            cache = mbg.PagedKV(torch.zeros(shape, dtype=torch.float16, device="cuda"),
                                torch.zeros(shape, dtype=torch.float16, device="cuda"),
                                torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None],
                                scores=torch.zeros(slots, device="cuda"),
                                stamps=torch.zeros(slots, dtype=torch.int32, device="cuda"))
            most = max(1, min(keep, cache.capacity - keep))
            self.layers.append({
                "qkv": weights((q_heads + 2 * kv_heads) * dim, hidden), "out": weights(hidden, q_heads * dim),
                "up": weights(mlp, hidden), "down": weights(hidden, mlp), "cache": cache,
                # norm after each block, and before the next one
                "norms": [1 + 0.1 * torch.empty(hidden, device="cuda").normal_(generator=g) for _ in range(4)],
                "lengths": torch.zeros(1, dtype=torch.int32, device="cuda"),
                "moves": torch.empty(1, kv_heads, most, 2, dtype=torch.int32, device="cuda"),
                "counts": torch.empty(1, kv_heads, dtype=torch.int32, device="cuda")})
        third = dim // 2 // 3
        self.rope = mbg.RopeTable(dim, sections=[dim // 2 - 2 * third, third, third])
        self.token = torch.zeros(1, dtype=torch.int32, device="cuda")         # its number
        self.positions = torch.zeros(3, 1, dtype=torch.int32, device="cuda")  # time, height, width
        self.x = torch.zeros(1, hidden, device="cuda")
        self.zero = torch.zeros(1, hidden, device="cuda")
        self.h = torch.zeros(1, hidden, dtype=torch.float16, device="cuda")

    def step(self):
        """One token: self.x (the residual) goes through all layers; positions and lengths move on."""
        qd, kd = self.q_heads * self.dim, self.kv_heads * self.dim
        # the first block's input: its norm of the residual as it is
        mbg.gemv_norm_residual(self.zero, self.x, pre_weight=self.layers[0]["norms"][3], out=self.x, h=self.h)
        for i, w in enumerate(self.layers):
            qkv = mbg.gemv_q4(w["qkv"][0], self.h[0], w["qkv"][1])  # FP32
            q, k, v = (t.view(1, -1, self.dim) for t in qkv.split((qd, kd, kd)))
            q = mbg.gemv_rope_append(w["cache"], q, k, v, self.positions, w["lengths"], self.rope, stamps=self.token)
            w["lengths"].add_(1)
            o = mbg.gemv_attn_paged(w["cache"], q, w["lengths"], accumulate=True)
            y = mbg.gemv_q4(w["out"][0], o.view(-1), w["out"][1])
            mbg.gemv_norm_residual(y[None], self.x, post=True, post_weight=w["norms"][0], pre_weight=w["norms"][1],
                                   out=self.x, h=self.h)
            up = mbg.gemv_q4(w["up"][0], self.h[0], w["up"][1])
            y = mbg.gemv_q4(w["down"][0], torch.relu(up).square().half(), w["down"][1])
            after = self.layers[(i + 1) % len(self.layers)]["norms"][3]
            mbg.gemv_norm_residual(y[None], self.x, post=True, post_weight=w["norms"][2], pre_weight=after, out=self.x,
                                   h=self.h)
            mbg.gemv_kv_evict(w["cache"], w["lengths"], self.keep, sinks=self.sinks, recent=self.recent,
                              moves=w["moves"], counts=w["counts"])
        self.token.add_(1)
        self.positions[0].add_(1)

    def capture(self):
        """The step as a CUDA graph (run a step before: it sets up what is kept)."""
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--keep", type=int, default=64)
    ap.add_argument("--layers", type=int, default=2)
    a = ap.parse_args()
    model = Decoder(layers=a.layers, keep=a.keep)
    model.x.normal_()
    model.step()
    graph = model.capture()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.tokens - 1):
        graph.replay()
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    status = mbg.gemv_get_device_error()
    print(f"{a.tokens} tokens, {a.layers} layers: {t / max(1, a.tokens - 1) * 1e6:.1f} us per token, cache holds "
          f"{int(model.layers[0]['lengths'])} of them, device status {mbg.STATUS[status]}")
    return 0 if status == mbg.OK and bool(model.x.isfinite().all()) else 1


if __name__ == "__main__":
    sys.exit(main())
