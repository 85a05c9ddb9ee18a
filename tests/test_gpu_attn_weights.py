"""Accumulated attention weights of rows that several blocks share, on both cache types, against 64 bits."""

import pytest

import memory_bound_gemv_gb300 as mbg

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_decode import BF16, F16, LENGTHS, attn_reference, close, make_cache, no_device_error, normal  # noqa: E402,F401


def check_weights(cache, lengths, group, window, seed):
    q = normal(seed, (len(lengths), cache.kv_heads * group, cache.head_dim), cache.dtype, 1.5)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    before, sums = cache.scores.clone(), torch.full_like(cache.scores, -5.0)
    out = mbg.gemv_attn_paged(cache, q, n, window=window, accumulate=True, scores_out=sums)
    ref, tol, w, wt, _, _ = attn_reference(cache, q, lengths, cache.head_dim ** -0.5, window)
    close(out, ref, tol, "out")
    slot = torch.arange(cache.capacity, device="cuda")
    end = n[:, None, None]
    live = ((slot < end) & (slot >= ((end - window).clamp(min=0) if window else 0))).expand_as(before)
    want = torch.where(live, before.double() + w, -5.0)
    # the sum with what was there, and the heads' sums in order
    close(sums, want, torch.where(live, wt + want.abs() * 2.0 ** -23 + w * group * 2.0 ** -24, 0.0), "scores")
    mbg.gemv_attn_paged(cache, q, n, window=window, accumulate=True)
    assert torch.equal(cache.scores, torch.where(live, sums, before))


@pytest.mark.parametrize("group,dim,page,window", [(1, 128, 16, 0), (4, 128, 16, 0), (5, 80, 24, 33), (9, 64, 16, 0),
                                                   (20, 128, 8, 100), (3, 33, 16, 0)])
def test_attn_weights_of_bfloat16_caches(group, dim, page, window):
    check_weights(make_cache(91, LENGTHS, 2, dim, page, BF16, history=True), LENGTHS, group, window, 92)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hk,group,dim,page,window", [(2, 4, 128, 16, 0), (1, 20, 64, 16, 0), (2, 4, 128, 24, 5000), (1, 3, 192, 64, 0),
                                                      (1, 12, 256, 16, 3000), (2, 1, 77, 5, 0), (3, 2, 80, 16, 1025)])
def test_attn_weights_of_rows_cut_over_blocks(dtype, hk, group, dim, page, window):
    lengths = [20011, 3, 5000, 0, 7001]
    check_weights(make_cache(93, lengths, hk, dim, page, dtype, history=True), lengths, group, window, 94)


def test_attn_weights_of_many_cut_rows():
    lengths = [4000 - 61 * (b % 40) for b in range(70)]
    check_weights(make_cache(95, lengths, 2, 64, 16, BF16, history=True), lengths, 2, 0, 96)
