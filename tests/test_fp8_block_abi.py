"""The second part of the C ABI (include/kvq_fp8_block.h) without a GPU: every
declared function is exported and bound, and bad arguments are refused on the
host before anything is enqueued (the pointers here are fake)."""
import ctypes
import os
import re

import pytest

from fp4_kv_cache_kvq_gb300 import build, kvq

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kvq_fp8_block.h")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kvq.load()


def test_every_declared_function_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(kvq_[a-z0-9_]+)\s*\(", text)))
    assert names == ["kvq_fp8_block_append", "kvq_fp8_block_decode_attn", "kvq_fp8_block_dequant",
                     "kvq_fp8_block_pool_bytes", "kvq_fp8_block_prefill_attn",
                     "kvq_fp8_block_prefill_workspace_bytes", "kvq_rope_append", "kvq_rope_table"]
    for name in names:
        assert getattr(lib, name).argtypes is not None, name


def test_pool_bytes(lib):
    assert lib.kvq_fp8_block_pool_bytes(10, 8, 64, 128) == 10 * 8 * (2 * 64 * 128 + 32)
    assert lib.kvq_fp8_block_pool_bytes(3, 2, 256, 64) == 3 * 2 * 4 * (2 * 64 * 64 + 32)
    assert lib.kvq_fp8_block_pool_bytes(3, 2, 16, 64) == 3 * 2 * (2 * 16 * 64 + 16)
    assert lib.kvq_fp8_block_pool_bytes(3, 2, 32, 128) == 3 * 2 * (2 * 32 * 128 + 16)
    for bad in ((-1, 2, 64, 128), (3, 0, 64, 128), (3, 2, 48, 128), (3, 2, 64, 256), (3, 2, 64, 80)):
        assert lib.kvq_fp8_block_pool_bytes(*bad) == 0


def _cache(**kw):
    f = dict(format=kvq.FORMAT_FP8_BLOCK, num_kv_heads=2, head_dim=128, page_size=64, num_pages=4,
             max_pages_per_seq=2, reserved=0, page_table=None, data=4096, v_data=None, k_scale=None, v_scale=None)
    f.update(kw)
    return ctypes.byref(kvq.KvqCacheStruct(**f))


def _rope(lib, c, batch=2, n=1, start=16, lens=None, hq=4, q=32, qs=512, k=64, ks=256, v=128, vs=256, table=256,
          rows=10, rd=128, inter=0, q_out=512, k_out=None):
    return lib.kvq_rope_append(c, batch, n, start, lens, hq, q, qs, k, ks, v, vs, table, rows, rd, inter, q_out,
                               k_out, None, None)


BAD_CACHES = [dict(head_dim=256), dict(head_dim=96), dict(page_size=48), dict(num_kv_heads=0), dict(reserved=1),
              dict(data=None), dict(data=4097), dict(v_data=8192), dict(k_scale=64), dict(v_scale=64), dict(format=7),
              dict(num_pages=3), dict(max_pages_per_seq=0), dict(page_table=6)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_invalid_caches_are_refused(lib, bad):
    c = _cache(**bad)
    assert _rope(lib, c) == 1
    assert lib.kvq_fp8_block_append(c, 2, 1, 16, None, 32, 64, None, None) == 1
    assert lib.kvq_fp8_block_dequant(c, 2, 16, 8, 0, 32, 64, None, None) == 1
    assert lib.kvq_fp8_block_decode_attn(c, 2, 4, 16, 32, 0.1, 64, 0, 128, 1 << 30, None, None) == 1
    assert lib.kvq_fp8_block_prefill_attn(c, 2, 4, 4, 16, None, 32, 0.1, 64, 0, 128, 1 << 30, None, None) == 1


def test_other_entry_points_refuse_the_block_format(lib):
    c = _cache()
    assert lib.kvq_append(c, 2, 1, 16, 32, 64, None, None) == 1
    assert lib.kvq_decode_attn(c, None, 2, 4, 16, 32, 0.1, 64, 128, 1 << 20, None, None) == 1
    assert lib.kvq_prefill_attn(c, 2, 4, 4, 16, 32, 0.1, 64, None, None) == 1
    assert lib.kvq_dequant(c, 2, 16, 8, 0, 32, 64, None, None) == 1
    fp4 = _cache(format=kvq.FORMAT_FP4)
    assert lib.kvq_fp8_block_append(fp4, 2, 1, 16, None, 32, 64, None, None) == 1
    assert lib.kvq_fp8_block_decode_attn(fp4, 2, 4, 16, 32, 0.1, 64, 0, 128, 1 << 30, None, None) == 1


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(n=-1), dict(hq=-1), dict(start=None), dict(k=None), dict(v=None), dict(q=None),
    dict(q_out=None), dict(hq=0), dict(q=40), dict(k=72), dict(v=136), dict(q_out=520), dict(k_out=8),
    dict(qs=516), dict(qs=504), dict(ks=248), dict(vs=260), dict(table=None), dict(table=264), dict(rows=-1),
    dict(rd=24), dict(rd=144), dict(rd=-16), dict(inter=2), dict(q_out=32, qs=520), dict(k_out=64, ks=264)])
def test_rope_append_refusals(lib, bad):
    assert _rope(lib, _cache(), **bad) == 1


def test_rope_append_limits_and_empty_calls(lib):
    ring = _cache(format=kvq.FORMAT_FP8, page_size=128, max_pages_per_seq=0, v_data=8192, k_scale=64, v_scale=64)
    assert _rope(lib, ring) == 2                                    # a window ring
    assert _rope(lib, _cache(num_pages=1 << 29, num_kv_heads=8)) == 2  # page and head indices past 2^31
    assert _rope(lib, _cache(num_pages=1 << 20), batch=1 << 15, n=1 << 20) == 2
    assert _rope(lib, _cache(), batch=0, start=None, k=None, v=None, q=None) == 0
    assert _rope(lib, _cache(), n=0, start=None, k=None, v=None, q=None) == 0
    assert lib.kvq_fp8_block_append(_cache(), 0, 5, None, None, None, None, None, None) == 0
    assert lib.kvq_rope_table(0, 64, 10000.0, None, None) == 0
    for bad in ((-1, 64, 1e4, 64), (4, 63, 1e4, 64), (4, 0, 1e4, 64), (4, 64, 0.0, 64), (4, 64, 1e4, None),
                (4, 64, float("nan"), 64), (4, 64, 1e4, 66)):
        assert lib.kvq_rope_table(*bad, None) == 1, bad


def test_attention_refusals(lib):
    dec = lambda c=None, b=2, hq=4, lens=16, q=32, sc=0.1, out=64, dt=0, ws=128: lib.kvq_fp8_block_decode_attn(  # noqa: E731
        c or _cache(), b, hq, lens, q, sc, out, dt, ws, 1 << 30, None, None)
    pre = lambda c=None, b=2, hq=4, n=4, lens=16, q=32, sc=0.1, out=64, dt=0, ws=128: lib.kvq_fp8_block_prefill_attn(  # noqa: E731
        c or _cache(), b, hq, n, lens, None, q, sc, out, dt, ws, 1 << 30, None, None)
    for f in (dec, pre):
        for bad in (dict(b=0), dict(hq=3), dict(hq=1), dict(lens=None), dict(q=None), dict(out=None), dict(ws=None),
                    dict(q=40), dict(out=68), dict(ws=132), dict(sc=0.0), dict(sc=-1.0), dict(sc=float("inf")),
                    dict(sc=float("nan")), dict(dt=2)):
            assert f(**bad) == 1, bad
        assert f(hq=18) == 2  # nine query heads per kv head
    assert pre(n=0) == 1
    assert lib.kvq_fp8_block_dequant(_cache(), 2, 16, 8, 2, 32, 64, None, None) == 1
    assert lib.kvq_fp8_block_dequant(_cache(), 2, None, 8, 0, 32, 64, None, None) == 1
    assert lib.kvq_fp8_block_dequant(_cache(), 2, 16, 8, 0, 36, 64, None, None) == 1
    for bad in ((0, 4, 2, 128, 4), (2, 3, 2, 128, 4), (2, 4, 2, 128, 0), (2, 4, 0, 128, 4)):
        assert lib.kvq_fp8_block_prefill_workspace_bytes(*bad) == 0
