"""The descriptions that the FP4 and FP8 window caches keep between calls: always
the pointers that their tensors have now, whatever became of the tensors before."""
import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq


@pytest.mark.parametrize("nvfp4", [False, True])
def test_fp4_handle_follows_its_tensors(nvfp4):
    cache = kvq.Fp4Cache(2, 64, 16, 4, 2, device="cpu", nvfp4=nvfp4)
    cache.page_table = torch.zeros((2, 2), dtype=torch.int32)
    assert cache.struct() is cache.struct()
    s = cache.struct()
    assert (s.page_table, s.data) == (cache.page_table.data_ptr(), cache.pool.data_ptr())
    # the same tensor object over other memory
    old = cache.page_table.data_ptr()
    cache.page_table.set_(torch.ones((2, 2), dtype=torch.int32))
    assert cache.page_table.data_ptr() != old
    assert cache.struct().page_table == cache.page_table.data_ptr()
    pool = torch.zeros_like(cache.pool)
    cache.pool.set_(pool)
    assert cache.struct().data == pool.data_ptr()
    # another object at the id of one that is gone
    for _ in range(20):
        cache.page_table = None
        cache.page_table = torch.zeros((2, 2), dtype=torch.int32)
        assert cache.struct().page_table == cache.page_table.data_ptr()
    cache.page_table = None
    assert cache.struct().page_table is None
    if nvfp4:
        cache.k_gscale.set_(torch.ones(2))
        assert cache.struct().k_scale == cache.k_gscale.data_ptr()


def test_window_handle_follows_its_tensors():
    ring = kvq.Fp8WindowCache(1, 2, 64, 16, device="cpu")
    assert ring.struct() is ring.struct()
    for name, field in (("k_codes", "data"), ("v_codes", "v_data"), ("k_scales", "k_scale"), ("v_scales", "v_scale")):
        getattr(ring, name).set_(torch.zeros_like(getattr(ring, name)))
        assert getattr(ring.struct(), field) == getattr(ring, name).data_ptr()
