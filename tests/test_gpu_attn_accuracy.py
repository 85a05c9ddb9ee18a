"""Paged attention where the softmax's weights differ widely, against its definition in 64 bits.

Keys are multiples of one axis and queries its unit vector, so that every
score is a product of two stored numbers and exact but for the two roundings
of scale * log2 e and of the product: |ds| <= 2^-23 |s|.  A weight is then off
by 2 ds, by 2^-22 (two ulp of the exponential) and by its own rounding: 2^-21
relative and 2^-38 of the warp's largest weight in binary16 (two parts of 11
bits over that floor), none in bfloat16 (24 bits in three parts).  Each sum
adds at most 2^-23 of its magnitude per addition.
"""

import math

import numpy as np
import pytest

import memory_bound_gemv_gb300 as mbg

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

F16, BF16 = torch.float16, torch.bfloat16
OWN = {F16: 2.0 ** -21, BF16: 0.0}
FLOOR = {F16: 2.0 ** -38, BF16: 2.0 ** -126}
HALF_STEP = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F16: 2.0 ** -25, BF16: 0.0}


def cache_of(scores, values, dim, page=16):
    """One cached head per sequence; scores: lists of numbers, values: [tokens, dim] each."""
    dtype = values[0].dtype
    need = [-(-len(s) // page) for s in scores]
    table = torch.full((len(scores), max(need) + 1), -1, dtype=torch.int32)
    k, v = (torch.zeros(sum(need), page, 1, dim, dtype=dtype) for _ in range(2))
    order, at = np.random.default_rng(1).permutation(sum(need)), 0
    for b, (s, val) in enumerate(zip(scores, values)):
        pages = torch.from_numpy(order[at:at + need[b]])
        at += need[b]
        table[b, :need[b]] = pages.to(torch.int32)
        t = torch.arange(len(s))
        k[pages[t // page], t % page, 0, 0] = torch.as_tensor(s, dtype=torch.float64).to(dtype)
        v[pages[t // page], t % page, 0] = val
    return mbg.PagedKV(k.cuda(), v.cuda(), table.cuda())


def run(cache, lengths, heads):
    q = torch.zeros(len(lengths), heads, cache.head_dim, dtype=cache.dtype, device="cuda")
    q[..., 0] = 1.0
    out = mbg.gemv_attn_paged(cache, q, torch.tensor(lengths, dtype=torch.int32, device="cuda"), scale=1.0)
    return out.double().cpu()


def exact(scores, values):
    """out, sum p |v| and sum |v| / l of one sequence."""
    s, v = torch.as_tensor(scores, dtype=torch.float64), values.double()
    e = torch.exp(s - s.max())
    return (e @ v) / e.sum(), (e @ v.abs()) / e.sum(), v.abs().sum(0) / e.sum()


def stored(x, dtype):
    return torch.as_tensor(x, dtype=torch.float64).to(dtype).double().tolist()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim", [8, 128, 256])
def test_attn_values_that_cancel(dtype, dim):
    """The output is what is left of two large terms: an error of a weight shows undiminished by the output's rounding."""
    rng = np.random.default_rng(2)
    scores, values = [], []
    for x in stored(-rng.uniform(0.05, 8.0, 120), dtype):
        p = math.exp(x)
        v = [1.0, stored([-1.0 / p], dtype)[0]]
        for _ in range(3):  # and the residuals of rounding that
            v.append(stored([-(v[0] + p * v[1] + sum(v[2:]))], dtype)[0])
        scores.append([0.0, x, 0.0, 0.0, 0.0])
        values.append(torch.tensor(v, dtype=torch.float64).to(dtype)[:, None].expand(5, dim))
    got = run(cache_of(scores, values, dim), [5] * len(scores), 2)
    for b, (s, v) in enumerate(zip(scores, values)):
        ref, mass, each = exact(s, v)
        # five products at most the size of one, and the join of four warps
        tol = mass * (2 * 2.0 ** -23 * abs(s[1]) + 2.0 ** -22 + OWN[dtype] + 10 * 2.0 ** -23) + FLOOR[dtype] * each
        tol = tol + ref.abs() * HALF_STEP[dtype] + TINY[dtype]
        assert ((got[b] - ref).abs() <= tol).all(), (b, s[1], float(((got[b] - ref).abs() / tol).max()))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads,dim", [(1, 64), (4, 128), (12, 128), (2, 256), (3, 33)])
@pytest.mark.parametrize("lead", [10.0, 14.0, 17.5, 20.0])
def test_attn_first_token_leads_and_adds_nothing(dtype, heads, dim, lead):
    """A sink: the largest weight by far, of a token whose value is zero; the others are all of the output."""
    rng = np.random.default_rng(3)
    lengths = [40, 1, 700, 5000]
    scores, values = [], []
    for n in lengths:
        scores.append(stored([lead] + (rng.random(n - 1) * 2 - 1).tolist(), dtype))
        v = 256.0 * (1.0 + 0.1 * rng.standard_normal((n, dim)))
        v[0] = 0.0
        values.append(torch.from_numpy(v).to(dtype))
    got = run(cache_of(scores, values, dim), lengths, heads)
    for b, n in enumerate(lengths):
        ref, mass, each = exact(scores[b], values[b])
        # a warp takes a quarter of the tokens at most; 16 products in up to three parts per tile; the joins
        adds = 48 * (n // 64 + 1) + 200
        tol = mass * (2 * 2.0 ** -23 * lead + 2.0 ** -22 + OWN[dtype] + adds * 2.0 ** -23) + FLOOR[dtype] * each
        tol = tol + ref.abs() * HALF_STEP[dtype] + TINY[dtype]
        assert ((got[b] - ref).abs() <= tol).all(), (n, float(((got[b] - ref).abs() / tol).max()))
