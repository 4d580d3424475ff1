"""The description of an 8-bit block cache that a call hands to the library."""
import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu


def test_each_call_has_a_description_of_its_own():
    """A page table put into the cache while another call's arguments are put
    together does not reach that call."""
    ensure_built()
    first, second, third = (torch.zeros((2, 3), dtype=torch.int32, device="cuda") for _ in range(3))
    cache = kvq.Fp8BlockCache(2, 64, 16, 6, 3, page_table=first)
    one = cache.struct()
    cache.page_table = second
    two, other = cache.struct(), cache.struct(third)
    assert [s.page_table for s in (one, two, other)] == [t.data_ptr() for t in (first, second, third)]
    assert all(s.data == cache.pool.data_ptr() and s.format == kvq.FORMAT_FP8_BLOCK for s in (one, two, other))
    cache.page_table = None
    assert cache.struct().page_table is None and two.page_table == second.data_ptr()
