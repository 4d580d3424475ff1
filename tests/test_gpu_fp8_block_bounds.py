"""The bounds-checked build of the library on the rotary append and the 8-bit
block cache: on every case no checked index leaves its buffer (the flag stays
clear) and the results equal the normal build's."""
import math

import pytest
import torch

from fp4_kv_cache_kvq_gb300 import build, kvq
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def libs():
    normal = ensure_built()
    path = build.build(bounds=True)
    saved, old = kvq._lib, kvq.LIB_PATH
    kvq._lib, kvq.LIB_PATH = None, path
    try:
        checked = kvq.load()
    finally:
        kvq._lib, kvq.LIB_PATH = saved, old
    return normal, checked


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _run(lib, d, G, page, H, lens, n, seed):
    saved = kvq._lib
    kvq._lib = lib
    try:
        g = torch.Generator().manual_seed(seed)
        B, T = len(lens), max(lens)
        mp = -(-(T + n) // page)
        table = torch.randperm(B * mp, generator=g).to(torch.int32).view(B, mp).cuda()
        cache = kvq.Fp8BlockCache(H, d, page, B * mp, mp, page_table=table)
        err = _ints([0])
        rope = kvq.rope_table(T + n, d)
        x = torch.randn((B, T, (G + 2) * H, d), generator=g).to(BF).cuda()
        kvq.rope_append(cache, _ints([0] * B), x[:, :, :G * H], x[:, :, G * H:(G + 1) * H], x[:, :, (G + 1) * H:], rope,
                        new_lens=_ints(lens), err=err)
        y = torch.randn((B, n, (G + 2) * H, d), generator=g).to(BF).cuda()
        q = kvq.rope_append(cache, _ints(lens), y[:, :, :G * H], y[:, :, G * H:(G + 1) * H], y[:, :, (G + 1) * H:], rope,
                            interleaved=True, err=err)
        now = _ints([m + n for m in lens])
        outs = [q, kvq.prefill_attn(cache, now, q, err=err), kvq.decode_attn(cache, now, q[:, -1].contiguous(), err=err),
                *kvq.dequant(cache, now, T + n, err=err)]
        fp4 = kvq.Fp4Cache(H, d, page, B * mp, mp, page_table=table)
        kvq.rope_append(fp4, _ints(lens), y[:, :, :G * H], y[:, :, G * H:(G + 1) * H], y[:, :, (G + 1) * H:], rope, err=err)
        torch.cuda.synchronize()
        return outs + [cache.pool, fp4.pool], err.item()
    finally:
        kvq._lib = saved


@pytest.mark.parametrize("d,G,page,H,lens,n", [
    (64, 1, 16, 3, [0, 1, 17, 300], 3), (64, 8, 256, 1, [700, 33], 40), (128, 4, 64, 2, [128, 5, 63], 1),
    (128, 7, 32, 2, [90, 400], 150), (128, 8, 128, 5, [129], 17)])
def test_no_index_leaves_its_buffer(libs, d, G, page, H, lens, n):
    (a, fa), (b, fb) = (_run(lib, d, G, page, H, lens, n, d + n) for lib in libs)
    assert fa == fb == 0
    for x, y in zip(a, b):
        assert torch.equal(x, y) and torch.isfinite(x.float()).all()
    assert not math.isnan(a[1].abs().max().item())
