"""Rows of many slots that are computed one by one (a scale of 0, or a hidden infinity in their tile).

2^20 slots of like weights.  A warp has an eighth of them, in pieces of 1024: a sum of N positive terms, each addition
off by at most half a step of it, is off by at most N 2^-24 relative: 1024 terms and 128 pieces, 1152 2^-24 < 2^-13, the
weights' sum alike (of 32 at a time: less) and 2^-20 for the rest; half a step of the output."""

import pytest

import memory_bound_gemv_gb300 as mbg
from test_gpu_decode import BF16, F16, HALF_STEP, no_device_error, normal  # noqa: F401
from test_gpu_serve_attn import ints

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

N, PAGE = 2 ** 20, 256
TOL = 2.0 ** -13 + 2.0 ** -13 + 2.0 ** -20


def pools(value, dim, dtype):
    v = torch.full((2, PAGE, 1, dim), value, dtype=dtype, device="cuda")
    return torch.zeros_like(v), v


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("value", [0.7, 0.9, 1.0])
@pytest.mark.parametrize("dim", [64, 200])
def test_like_values_with_a_scale_of_zero(dtype, value, dim):
    k, v = pools(value, dim, dtype)
    table = torch.arange(N // PAGE, dtype=torch.int32, device="cuda")[None] % 2
    q = normal(95, (3, 2, dim), dtype)
    want = v[0, 0, 0].double()
    got = mbg.gemv_attn_prompt(mbg.PagedKV(k, v, table), q, ints([0, 3]), ints([N]), scale=0.0).double()
    assert ((got - want).abs() <= (TOL + HALF_STEP[dtype]) * want).all()
    got = mbg.gemv_attn_shared(mbg.PagedKV(k, v, table.expand(3, -1).contiguous()), q, ints([N] * 3), ints([N - 7]), scale=0.0).double()
    assert ((got - want).abs() <= (TOL + HALF_STEP[dtype]) * want).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_like_values_next_to_an_infinite_one(dtype):
    """The last token's own value, on a page of its own."""
    k, v = pools(0.7, 64, dtype)
    k, v = torch.cat([k, k[:1]]), torch.cat([v, v[:1]])
    v[2, PAGE - 1] = float("inf")
    table = torch.arange(N // PAGE, dtype=torch.int32, device="cuda")[None] % 2
    table[0, -1] = 2
    q = normal(96, (3, 2, 64), dtype)
    want = v[0, 0, 0].double()
    got = mbg.gemv_attn_prompt(mbg.PagedKV(k, v, table), q, ints([0, 3]), ints([N])).double()
    assert ((got[:2] - want).abs() <= (TOL + HALF_STEP[dtype]) * want).all()
    assert (got[2] == float("inf")).all()
