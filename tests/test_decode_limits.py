"""Refusals at the limits of the decode-step operators.  No GPU: nothing below is launched."""

import pytest

import memory_bound_gemv_gb300 as mbg

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("shape", [(4, 16, 0, 64), (4, 0, 2, 64), (4, 16, 2, 0)])
def test_caches_without_heads_slots_or_elements_are_refused(shape):
    """A count of 0 heads would divide by zero in the compiled checks, which ends the process."""
    k, table = torch.zeros(shape, dtype=torch.float16), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="pages need slots, heads and elements"):
        mbg.PagedKV(k, k, table)
