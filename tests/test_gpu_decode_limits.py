"""Arguments at and beyond the limits of the decode-step calls: refused, or right."""

import math

import pytest

import memory_bound_gemv_gb300 as mbg

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_decode import F16, make_cache, normal  # noqa: E402


def test_caches_without_heads_slots_or_elements_are_refused():
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for shape in ((4, 16, 0, 64), (4, 0, 2, 64), (4, 16, 2, 0)):
        with pytest.raises(ValueError):
            mbg.PagedKV(torch.zeros(shape, dtype=F16, device="cuda"), torch.zeros(shape, dtype=F16, device="cuda"), table)


@pytest.mark.parametrize("many", [2 ** 31, 2 ** 32 + 5, 2 ** 40])
def test_counts_beyond_32_bits_are_refused(many):
    cache = make_cache(131, [40, 40], 2, 8, 16, F16, history=True)
    n = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    moves = torch.empty(2, 2, 64, 2, dtype=torch.int32, device="cuda")
    counts = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mbg.gemv_kv_evict_apply(cache, moves, counts, n, many)  # lengths would become 5
    for bad in (dict(keep=many), dict(keep=8, sinks=many), dict(keep=8, recent=many)):
        for room in (dict(), dict(moves=moves, counts=counts)):
            with pytest.raises(ValueError):
                mbg.gemv_kv_evict_plan(cache, n, **bad, **room)
    with pytest.raises(ValueError):
        mbg.gemv_attn_paged(cache, normal(1, (2, 4, 8), F16), n, window=many)
    assert n.tolist() == [40, 40]


def test_attn_of_a_cache_without_slots():
    """Lengths beyond a capacity of 0 are reported, and the row is an empty one like any other."""
    k = torch.zeros(1, 16, 1, 64, dtype=F16, device="cuda")
    cache = mbg.PagedKV(k, k.clone(), torch.zeros(2, 0, dtype=torch.int32, device="cuda"))
    q, lse = normal(2, (2, 4, 64), F16), torch.zeros(2, 4, device="cuda")
    for lengths, status in (([0, 0], mbg.OK), ([0, 5], mbg.ERR_BAD_INDEX)):
        out = torch.full_like(q, 7.0)
        mbg.gemv_attn_paged(cache, q, torch.tensor(lengths, dtype=torch.int32, device="cuda"), out=out, lse=lse.zero_())
        assert mbg.gemv_get_device_error() == status
        assert (out == 0).all() and (lse == -math.inf).all()


def test_attn_weights_of_a_row_that_ends_close_to_2_to_the_31():
    """One page stands for all: 2^31 slots of equal keys, weights of 1 / n each."""
    page, pages = 65536, 32767
    n = page * pages
    k, v = torch.zeros(1, page, 1, 8, dtype=F16, device="cuda"), torch.ones(1, page, 1, 8, dtype=F16, device="cuda")
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    cache = mbg.PagedKV(k, v, table, scores=torch.zeros(1, 1, n, device="cuda"))
    q, lse = torch.ones(1, 1, 8, dtype=F16, device="cuda"), torch.zeros(1, 1, device="cuda")
    out = mbg.gemv_attn_paged(cache, q, torch.tensor([n - 3], dtype=torch.int32, device="cuda"), lse=lse, accumulate=True)
    # sums of some hundred parts in FP32
    assert (out == 1).all() and abs(float(lse) - math.log(n - 3)) < 2.0 ** -14
    got = cache.scores[0, 0]
    low, high = float(got[:n - 3].min()), float(got[:n - 3].max())
    assert (got[n - 3:] == 0).all()
    assert abs(low * (n - 3) - 1) < 2.0 ** -14 and abs(high * (n - 3) - 1) < 2.0 ** -14
