"""The attention's workspace: what calls that misuse it leave, who shares it."""

import pytest

import memory_bound_gemv_gb300 as mbg
from memory_bound_gemv_gb300 import decode

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def make(lengths, heads=1, dim=64, page=16, seed=0, history=False, capacity=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    per = -(-(capacity or max(lengths)) // page)
    k, v = (torch.empty(len(lengths) * per, page, heads, dim, device="cuda").normal_(generator=g).half() for _ in range(2))
    table = torch.randperm(len(lengths) * per, generator=g, device="cuda").to(torch.int32).view(len(lengths), per)
    extra = dict(scores=torch.zeros(len(lengths), heads, per * page, device="cuda")) if history else {}
    return mbg.PagedKV(k, v, table, **extra), torch.tensor(lengths, dtype=torch.int32, device="cuda")


def query(cache, heads, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(cache.batch, heads, cache.head_dim, device="cuda").normal_(generator=g).half()


@pytest.mark.parametrize("lengths", [[70000], [20000] * 7, [3000, 0, 41, 900] * 60])
def test_attn_after_a_call_whose_lengths_changed(lengths):
    """Such a call can leave arrivals uncounted for; the calls after it count their own."""
    cache, n = make(lengths)
    queries = [query(cache, 4, seed) for seed in range(4)]
    good = [mbg.gemv_attn_paged(cache, q, n).clone() for q in queries]
    memory = cache._workspace(4, False, mbg._stream_ptr(None), None)[2]
    counters = memory[:decode._ATTN_COUNTER_BYTES].view(torch.int32)
    for step, q in enumerate(queries):
        counters[2::2] += 60  # more arrivals than are waited for
        out = mbg.gemv_attn_paged(cache, q, n, out=torch.full_like(q, 7.0))
        assert torch.equal(out, good[step]), step
    assert mbg.gemv_get_device_error() == mbg.OK
