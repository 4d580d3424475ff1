"""The third part of the C ABI (include/kvq_latent.h) without a GPU: every
declared function is exported and bound, and bad arguments are refused on the
host before anything is enqueued (the pointers here are fake)."""
import ctypes
import os
import re

import pytest
import torch

from fp4_kv_cache_kvq_gb300 import build, kvq

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kvq_latent.h")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kvq.load()


def test_every_declared_function_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(kvq_[a-z0-9_]+)\s*\(", text)))
    assert names == ["kvq_expanded_attn", "kvq_latent_append", "kvq_latent_attn", "kvq_latent_attn_workspace_bytes",
                     "kvq_latent_dequant", "kvq_latent_pool_bytes"]
    for name in names:
        assert getattr(lib, name).argtypes is not None, name


def test_struct_layout():
    assert ctypes.sizeof(kvq.KvqLatentStruct) == 40
    assert kvq.KvqLatentStruct.num_pages.offset == 16 and kvq.KvqLatentStruct.data.offset == 32


def test_pool_bytes(lib):
    assert lib.kvq_latent_pool_bytes(10, 64, 512, 64) == 10 * 64 * 641
    assert lib.kvq_latent_pool_bytes(3, 256, 128, 32) == 3 * 256 * 193
    assert lib.kvq_latent_pool_bytes(1 << 20, 256, 512, 64) == (1 << 28) * 641
    for bad in ((-1, 64, 512, 64), (3, 48, 512, 64), (3, 64, 384, 64), (3, 64, 512, 16), (3, 64, 512, 128),
                (1 << 31, 64, 512, 64)):
        assert lib.kvq_latent_pool_bytes(*bad) == 0


def _cache(**kw):
    f = dict(latent_dim=512, rope_dim=64, page_size=64, max_pages_per_seq=2, num_pages=4, page_table=None, data=4096)
    f.update(kw)
    return ctypes.byref(kvq.KvqLatentStruct(**f))


def _append(lib, c=None, batch=2, n=1, start=16, lens=None, hq=4, q=32, qt=768, qh=192, lat=64, ct=576, k=128, kt=576,
            table=256, rows=10, inter=0, q_out=512, ot=2304, oh=576, k_out=None):
    return lib.kvq_latent_append(c if c is not None else _cache(), batch, n, start, lens, hq, q, qt, qh, lat, ct, k, kt,
                                 table, rows, inter, q_out, ot, oh, k_out, None, None)


def _attn(lib, c=None, batch=2, hq=16, chunk=1, lens=16, clens=None, q=32, scale=0.1, out=64, dtype=1, ws=128,
          nbytes=1 << 40):
    return lib.kvq_latent_attn(c if c is not None else _cache(), batch, hq, chunk, lens, clens, q, scale, out, dtype, ws,
                               nbytes, None, None)


def _dequant(lib, c=None, batch=2, lens=16, max_len=8, dtype=0, c_out=64, k_out=128):
    return lib.kvq_latent_dequant(c if c is not None else _cache(), batch, lens, max_len, dtype, c_out, k_out, None, None)


def _expanded(lib, batch=2, heads=4, d=128, rope=64, chunk=3, max_len=9, lens=16, clens=None, q=32, k=64, kt=1024,
              kh=256, kr=128, rt=576, v=320, vt=1024, vh=256, scale=0.1, out=256, dtype=1):
    return lib.kvq_expanded_attn(batch, heads, d, rope, chunk, max_len, lens, clens, q, k, kt, kh, kr, rt, v, vt, vh,
                                 scale, out, dtype, None, None)


BAD_CACHES = [dict(latent_dim=384), dict(rope_dim=16), dict(page_size=48), dict(max_pages_per_seq=0), dict(num_pages=0),
              dict(num_pages=3), dict(data=None), dict(data=4104), dict(page_table=6)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_invalid_caches_are_refused(lib, bad):
    c = _cache(**bad)
    assert _append(lib, c) == _attn(lib, c) == _dequant(lib, c) == 1


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(n=-1), dict(hq=-1), dict(start=None), dict(lat=None), dict(k=None), dict(q=None),
    dict(q_out=None), dict(hq=0), dict(q=36), dict(lat=72), dict(k=136), dict(q_out=520), dict(k_out=24),
    dict(qt=764), dict(qh=56), dict(qt=576), dict(ct=504), dict(ct=508), dict(kt=60), dict(ot=760), dict(oh=60),
    dict(inter=2), dict(table=264), dict(table=None), dict(rows=-1), dict(q_out=32), dict(k_out=128), dict(k_out=64)])
def test_invalid_appends_are_refused(lib, bad):
    assert _append(lib, **bad) == 1


def test_appends_too_large_for_one_call(lib):
    big = dict(c=_cache(num_pages=1 << 30, max_pages_per_seq=1 << 22))
    assert _append(lib, n=1 << 26, qt=64 * 192, ot=64 * 576, **big) == 2
    assert _append(lib, n=1 << 23, hq=128, qt=128 * 192, ot=128 * 576, **big) == 2


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(hq=0), dict(chunk=-1), dict(lens=None), dict(q=None), dict(out=None), dict(ws=None),
    dict(q=40), dict(out=72), dict(ws=136), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(dtype=2)])
def test_invalid_attention_is_refused(lib, bad):
    assert _attn(lib, **bad) == 1


def test_attention_sizes(lib):
    assert _attn(lib, nbytes=0) == 3
    need = lib.kvq_latent_attn_workspace_bytes
    assert need(2, 16, 512, 1) > 0
    for bad in ((0, 16, 512, 1), (2, 0, 512, 1), (2, 16, 384, 1), (2, 16, 512, 0)):
        assert need(*bad) == 0
    assert _attn(lib, batch=1, hq=128, chunk=1 << 24, c=_cache(num_pages=1 << 20, max_pages_per_seq=1 << 20)) == 2


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(max_len=-1), dict(lens=None), dict(c_out=None), dict(k_out=None),
                                 dict(c_out=72), dict(k_out=136), dict(dtype=2)])
def test_invalid_read_backs_are_refused(lib, bad):
    assert _dequant(lib, **bad) == 1


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(heads=0), dict(d=96), dict(rope=32), dict(chunk=-1), dict(max_len=-1), dict(lens=None),
    dict(q=None), dict(k=None), dict(kr=None), dict(v=None), dict(out=None), dict(q=40), dict(k=72), dict(kr=136),
    dict(v=328), dict(out=264), dict(kt=1020), dict(kh=252), dict(kh=120), dict(kt=512), dict(rt=56), dict(rt=60),
    dict(vt=512), dict(vh=120), dict(scale=0.0), dict(scale=float("inf")), dict(dtype=2)])
def test_invalid_expanded_attention_is_refused(lib, bad):
    assert _expanded(lib, **bad) == 1


def test_empty_calls_enqueue_nothing(lib):
    assert _append(lib, batch=0) == _append(lib, n=0) == 0
    assert _attn(lib, batch=0) == _attn(lib, chunk=0) == 0
    assert _dequant(lib, batch=0) == _dequant(lib, max_len=0) == 0
    assert _expanded(lib, batch=0) == _expanded(lib, chunk=0) == 0


def test_row_strides():
    """What the binding takes as evenly spaced tokens and heads (CPU tensors stand in: device -1)."""
    bf = dict(dtype=torch.bfloat16)
    x = torch.zeros((3, 5, 4, 192), **bf)
    assert kvq._row_strides(-1, x[..., 128:], "q", True)[:2] == (768, 192)
    assert kvq._row_strides(-1, x, "q", True)[:2] == (768, 192)
    assert kvq._row_strides(-1, x[:, :, 1:2, 128:], "q", True)[:2] == (768, 64)
    assert kvq._row_strides(-1, x[:, :1, :, 128:], "q", True)[0] == 5 * 768
    assert kvq._row_strides(-1, x[:1, :1, :, 128:], "q", True)[:2] == (768, 192)
    assert kvq._row_strides(-1, x[:, :, 0, :64], "c", False)[0] == 768
    for bad in (x.transpose(1, 2), x.transpose(2, 3), x[:, :3], x[..., ::2], x.float()):
        with pytest.raises(ValueError):
            kvq._row_strides(-1, bad, "q", True)
    with pytest.raises(ValueError):
        kvq._row_strides(-1, x[:1, :1, :1].expand(3, 5, 4, 192), "q", True)


def test_geometry_is_checked(lib):
    with pytest.raises(ValueError):
        kvq.LatentCache(384, 64, 64, 4, 2, device="cpu")
    with pytest.raises(ValueError):
        kvq.LatentCache(512, 16, 64, 4, 2, device="cpu")
