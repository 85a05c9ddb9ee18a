"""Infinite and NaN values in paged attention go where the weighted sum takes them."""

import math

import pytest

import memory_bound_gemv_gb300 as mbg

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,dim,length", [(1, 64, 40), (4, 128, 16), (4, 128, 3000), (12, 64, 300), (2, 256, 77), (2, 33, 50)])
def test_attn_infinite_values(dtype, heads, dim, length):
    g = torch.Generator(device="cuda")
    g.manual_seed(length)
    pages = -(-length // 16)
    k, v = (torch.empty(pages, 16, 1, dim, device="cuda").normal_(generator=g).to(dtype) for _ in range(2))
    q = torch.empty(1, heads, dim, device="cuda").normal_(generator=g).to(dtype)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    n = torch.tensor([length], dtype=torch.int32, device="cuda")
    cache = mbg.PagedKV(k, v, table)
    clean = mbg.gemv_attn_paged(cache, q, n)

    def put(token, d, value):
        v[table[0, token // 16].long(), token % 16, 0, d] = value

    put(1, 3, math.inf), put(length - 1, 5, -math.inf)
    put(0, 6, math.inf), put(length // 2, 6, math.inf)
    put(2, 8, math.inf), put(length - 2, 8, -math.inf)  # a sum of both
    put(4, 9, math.nan)
    got = mbg.gemv_attn_paged(cache, q, n)
    assert (got[..., 3] == math.inf).all() and (got[..., 5] == -math.inf).all() and (got[..., 6] == math.inf).all()
    assert got[..., 8].isnan().all() and got[..., 9].isnan().all()
    other = [d for d in range(dim) if d not in (3, 5, 6, 8, 9)]
    assert torch.equal(got[..., other], clean[..., other])


def test_attn_a_key_of_minus_infinity_leaves_no_weight_to_a_large_value():
    """Weight 0 is exactly 0, whatever the value next to it."""
    for dtype, large in ((torch.float16, 6e4), (torch.bfloat16, 3e38)):
        k, v = torch.zeros(3, 16, 1, 64, dtype=dtype, device="cuda"), torch.ones(3, 16, 1, 64, dtype=dtype, device="cuda")
        k[1, 4], v[1, 4] = -math.inf, large
        q = torch.ones(1, 2, 64, dtype=dtype, device="cuda")
        table = torch.arange(3, dtype=torch.int32, device="cuda")[None]
        out = mbg.gemv_attn_paged(mbg.PagedKV(k, v, table), q, torch.tensor([40], dtype=torch.int32, device="cuda"))
        assert (out == 1).all()
