"""Pages that come back from requests whose lengths or tables are not as they should be.  Whole numbers: equal or wrong."""

import pytest

import memory_bound_gemv_gb300 as mbg
from test_gpu_decode import F16, no_device_error  # noqa: F401
from test_gpu_serve import ints

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def assign(table, lengths, fresh, ring, state, pages, page=4, room=8, shared=None):
    kv = torch.zeros(pages, page, 1, 1, dtype=F16, device="cuda")
    cache = mbg.PagedKV(kv, kv, ints(table))
    pool = mbg.PagePool(ring=ints(ring), state=ints(state))
    n = ints(lengths)
    starts, slots, seq = mbg.gemv_kv_assign(cache, pool, n, ints(fresh), tokens=room, shared=shared)
    assert mbg.gemv_get_device_error() == mbg.ERR_BAD_INDEX
    assert cache.page_table.tolist() == table
    return starts.tolist(), n.tolist(), pool.ring.tolist(), pool.state.tolist()


@pytest.mark.parametrize("room", [8, 30000])  # one block, several
@pytest.mark.parametrize("batch", [3, 1025])
@pytest.mark.parametrize("length", [9, 2 ** 31 - 1, -1])
def test_a_finished_request_of_impossible_length_returns_nothing(length, batch, room):
    """Its row may still name pages that others have by now."""
    table = [[0, 1]] + [[2, 3]] * (batch - 2) + [[4, 5]]
    lengths, fresh = [length] + [8] * (batch - 2) + [7], [-1] + [0] * (batch - 2) + [-1]
    starts, n, ring, state = assign(table, lengths, fresh, [9, -1, -1, -1], [0, 1], 10, room=room)
    assert starts == [0] * (batch + 1) and n == [0] + [8] * (batch - 2) + [0]
    assert ring == [9, 4, 5, -1] and state == [0, 3]
