"""The waits of the attention of many tokens run out, are reported, and leave nothing behind: the hook withholds one tile of K,
so that every block gives up with copies, products and softmax under way.  Limit 2 ms, as for the other kernels."""

import pytest

import memory_bound_gemv_gb300 as mbg
from test_gpu_decode import BF16, F16, make_cache, no_device_error, normal  # noqa: F401
from test_gpu_serve_attn import check_prompt, check_shared, ints, shared_cache

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


HEADS = 152  # as many as SMs, so that every block has three tiles or more


def gives_up(run):
    assert mbg.gemv_get_device_error() == mbg.OK
    try:
        mbg.debug_set_wait_limit_ns(2_000_000)
        mbg.debug_skip_copies(mbg.SKIP_TILE)
        run()
        status = mbg.gemv_get_device_error()
    finally:
        mbg.debug_skip_copies(0)
        mbg.debug_set_wait_limit_ns(0)
    assert status == mbg.ERR_TIMEOUT, mbg.STATUS.get(status, status)  # and no copy left under way


# pages of 16 and 64 go by bulk copies, 7 piece by piece, shifted pools element by element; 1003 slots end inside a box
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim,page,shift", [(128, 16, 0), (64, 64, 0), (128, 7, 0), (192, 16, 0), (256, 7, 0), (128, 16, 1)])
@pytest.mark.parametrize("fresh", [300, 3])  # rows for both streams, for one tile of rows
def test_a_prompt_gives_up(dtype, dim, page, shift, fresh):
    cache = make_cache(41, [1003], HEADS, dim, page, dtype, shift=shift)
    q = normal(42, (fresh, HEADS, dim), dtype)
    out, lse = torch.empty_like(q), torch.empty(fresh, HEADS, device="cuda")
    gives_up(lambda: mbg.gemv_attn_prompt(cache, q, ints([0, fresh]), ints([1003]), out=out, lse=lse))
    check_prompt(cache, [fresh], [1003], 1)


@pytest.mark.parametrize("dim,page", [(128, 16), (64, 7)])
def test_a_prefix_gives_up(dim, page):
    lengths = [100003, 99000, 100100]
    cache = shared_cache(43, lengths, 100003, 1, dim, page, BF16)
    q, n, pre = normal(44, (3, 2, dim), BF16), ints(lengths), ints([100003])
    gives_up(lambda: mbg.gemv_attn_shared(cache, q, n, pre))
    check_shared(cache, lengths, 100003, 2)
