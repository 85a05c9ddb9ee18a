"""Eviction plans of rows that fill a cluster's registers, and of rows that do not fit there."""

import numpy as np
import pytest

import memory_bound_gemv_gb300 as mbg

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_decode import F16, evict_reference, make_cache, no_device_error, same_bits  # noqa: E402,F401


@pytest.mark.parametrize("kind", ["normal", "equal", "few values"])
@pytest.mark.parametrize("lengths", [[150001, 140000, 9], [210007, 60, 200001], [65536, 65537, 131072]])
@pytest.mark.parametrize("keep,sinks,recent", [(9000, 4, 512), (59, 0, 100), (139999, 2, 1000)])
def test_evict_plan_and_moves(lengths, keep, sinks, recent, kind):
    cache = make_cache(121, lengths, 2, 8, 64, F16, history=True)
    if kind == "equal":
        cache.scores.fill_(0.25)
    elif kind == "few values":
        cache.scores.copy_(torch.randint(0, 5, cache.scores.shape, device="cuda").float())
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    k, v, sc, st = (t.clone() for t in (cache.k, cache.v, cache.scores, cache.stamps))
    moves, counts = mbg.gemv_kv_evict_plan(cache, lens, keep, sinks=sinks, recent=recent)
    mbg.gemv_kv_evict_apply(cache, moves, counts, lens, keep)
    scn, stn = sc.cpu().numpy(), st.cpu().numpy()
    for b, n in enumerate(lengths):
        for h in range(2):
            want = np.array(evict_reference(scn[b, h], stn[b, h], n, keep, sinks, recent), dtype=np.int32).reshape(-1, 2)
            assert int(counts[b, h]) == len(want)
            got = moves[b, h, :len(want)]
            assert np.array_equal(got.cpu().numpy(), want)
            src, dst = got.long().unbind(-1)
            ps, pd = (cache.page_table[b, x // 64].long() for x in (src, dst))
            for pool in (k, v):
                pool[pd, dst % 64, h] = pool[ps, src % 64, h]
            sc[b, h, dst], st[b, h, dst] = sc[b, h, src], st[b, h, src]
    assert same_bits(cache.k, k) and same_bits(cache.v, v) and same_bits(cache.scores, sc)
    assert torch.equal(cache.stamps, st) and lens.tolist() == [min(n, keep) for n in lengths]
