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


@pytest.mark.parametrize("room", [8, 30000])
@pytest.mark.parametrize("batch", [4, 1030])
def test_pages_that_do_not_exist_do_not_come_back(batch, room):
    """A -1 or a number beyond the pools in the row of a request that is over; shared first pages are not looked at."""
    table = [[0, -1, 2], [3, 4, 10], [-7, 5, 6]] + [[-1, -1, -1]] * (batch - 4) + [[7, 2 ** 31 - 1, 8]]
    lengths, fresh = [12, 9, 10] + [0] * (batch - 4) + [11], [-1, -2, -1] + [0] * (batch - 4) + [-1]
    shared = ints([0, 3, 4] + [0] * (batch - 4) + [0])
    starts, n, ring, state = assign(table, lengths, fresh, [-5] * 12, [10, 1], 10, room=room, shared=shared)
    assert starts == [0] * (batch + 1) and n == [0] * batch
    assert state == [10, 9] and ring[11:] + ring[:7] == [0, 2, 3, 4, 5, 6, 7, 8]  # (the other places hold no free page)


def test_what_exists_comes_back_even_where_more_than_was_lent_is_named():
    """Three pages are lent, four come back, one of which does not exist."""
    _, n, ring, state = assign([[-1, 4], [5, 6]], [8, 8], [-1, -1], [0, 1, 2, 3], [3, 1], 10)
    assert n == [0, 0] and ring == [4, 5, 6, 3] and state == [3, 4]


def test_many_pages_of_a_long_request_come_back():
    """More pages of one request than a block has threads."""
    pages = 2600
    row = [(7 * i) % pages for i in range(2500)]
    row[0], row[1024], row[2499] = -1, pages, -2
    want = [p for i, p in enumerate(row) if i not in (0, 1024, 2499)]
    _, n, ring, state = assign([row], [2500], [-1], [0] * 3000, [2990, 3], pages, page=1)
    assert n == [0] and state == [2990, 3 + len(want)]
    assert (ring[2993:] + ring[:2993])[:len(want)] == want
