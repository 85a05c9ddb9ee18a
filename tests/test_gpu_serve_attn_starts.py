"""Starts that do not ascend: no two sequences have the same tokens, whichever kernel computes them."""

import math

import pytest

import memory_bound_gemv_gb300 as mbg
from test_gpu_decode import BF16, F16, close, make_cache, no_device_error, normal  # noqa: F401
from test_gpu_serve_attn import ints, prompt_reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def expected(starts, tokens):
    """The definition: (sequence, its first token, its end) of those that have tokens."""
    kept, top = [], 0
    for b, (s0, s1) in enumerate(zip(starts, starts[1:])):
        if top <= s0 < s1 <= tokens:
            kept.append((b, s0, s1))
        top = max(top, s0)
    return kept


def check(starts, lengths, tokens, dtype, dim, scale, infinite=False, group=2):
    cache = make_cache(31, lengths, 1, dim, 16, dtype)
    q = normal(32, (tokens, group, dim), dtype)
    kept = expected(starts, tokens)
    want = []
    for b, s0, s1 in kept:
        one = mbg.PagedKV(cache.k, cache.v, cache.page_table[b:b + 1].contiguous())
        want.append(prompt_reference(one, q[s0:s1], [0, s1 - s0], [lengths[b]], scale, 0, 0))
    if infinite:  # the last token's own value: the others are computed again
        for b, s0, s1 in kept:
            cache.v[int(cache.page_table[b, (lengths[b] - 1) // 16]), (lengths[b] - 1) % 16] = math.inf
    out, lse = torch.full_like(q, 7.0), torch.full((tokens, group), 7.0, device="cuda")
    mbg.gemv_attn_prompt(cache, q, ints(starts), ints(lengths), out=out, lse=lse, scale=scale)
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    left = torch.ones(tokens, dtype=torch.bool, device="cuda")
    for (b, s0, s1), (ref, tol, rl, lt) in zip(kept, want):
        end = s1 - 1 if infinite else s1
        close(out[s0:end], ref[:end - s0], tol[:end - s0], f"out of {b}")
        close(lse[s0:s1], rl, lt, f"lse of {b}")
        assert (out[end:s1] == math.inf).all()
        left[s0:s1] = False
    assert (out[left] == 7).all() and (lse[left] == 7).all()


@pytest.mark.parametrize("scale", [0.1, 0.0])
@pytest.mark.parametrize("infinite", [False, True])
@pytest.mark.parametrize("starts", [[0, 10, 5, 20], [0, 20, 5, 20], [3, 9, 9, 4, 12, 20], [0, 8, 2 ** 31 - 1, 8, 20], [15, 12, 20],
                                    [0, 6, -3, 6, 20], [-2 ** 31, 5, 4, 20], [0, 0, 20, 19, 20]])
def test_starts_that_fall(starts, infinite, scale):
    check(starts, [40] * (len(starts) - 1), 20, F16, 64, scale, infinite)


@pytest.mark.parametrize("scale", [0.1, 0.0])
@pytest.mark.parametrize("at", [5, 511, 512, 600])
def test_starts_that_fall_among_many_sequences(at, scale):
    """More sequences than a block has threads; the fall lies in the first or the second run of them."""
    starts = list(range(0, 2 * 701, 2))
    starts[at] = starts[at - 1] - 7 if at > 5 else 900
    check(starts, [20] * 700, 1400, BF16, 64, scale, True, group=1)


@pytest.mark.parametrize("scale", [0.1, 0.0])
def test_starts_that_fall_in_long_prompts(scale):
    """Blocks cut between several groups of tiles."""
    check([0, 600, 100, 900, 1000], [2000, 700, 900, 300], 1000, BF16, 128, scale, group=8)


@pytest.mark.parametrize("scale", [0.1, 0.0])
def test_rows_before_the_first_start_are_left_alone(scale):
    cache = make_cache(33, [30, 40], 1, 64, 16, F16)
    q, out = normal(34, (20, 2, 64), F16), torch.full((20, 2, 64), 7.0, dtype=F16, device="cuda")
    mbg.gemv_attn_prompt(cache, q, ints([4, 10, 17]), ints([30, 40]), out=out, scale=scale)
    assert (out[:4] == 7).all() and (out[17:] == 7).all()
    ref, tol, _, _ = prompt_reference(cache, q[4:17], [0, 6, 13], [30, 40], scale, 0, 0)
    close(out[4:17], ref, tol)
