"""The latent operators in the bounds-checked build (-DKVQ_DEBUG_BOUNDS): no index leaves its
buffer, and the results are those of the ordinary build."""
import pytest
import torch

from fp4_kv_cache_kvq_gb300 import build, kvq
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _run():
    g = torch.Generator(device="cuda").manual_seed(1)
    out, err = [], _ints([0])
    for L, R, page, lens in ((512, 64, 16, [1, 333, 64, 0]), (256, 32, 128, [700, 5]), (128, 64, 64, [129] * 9)):
        B, n = len(lens), max(lens)
        mp = -(-n // page)
        table = torch.randperm(B * mp, generator=torch.Generator().manual_seed(2)).to(torch.int32).view(B, mp).cuda()
        cache = kvq.LatentCache(L, R, page, B * mp, mp, page_table=table)
        down, qp = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((B, n, L + R), (B, n, 6, 96 + R)))
        qr = kvq.latent_append(cache, _ints([0] * B), qp[..., 96:], down[..., :L], down[..., L:], kvq.rope_table(n, R),
                               new_lens=_ints(lens), err=err)
        q = torch.randn((B, 3, 6, L + R), generator=g, device="cuda").to(BF)
        seq = _ints(lens)
        out += [cache.pool.clone(), kvq.decode_attn(cache, seq, q[:, 0].contiguous(), 0.1, err=err),
                kvq.prefill_attn(cache, seq, q, 0.1, chunk_lens=_ints([min(3, x) for x in lens]), err=err),
                *kvq.dequant(cache, seq, n, err=err)]
        out += [qr[b, :m] for b, m in enumerate(lens)]
    return out, err.item()


def test_the_checked_build_raises_no_flag_and_gives_the_same():
    ensure_built()
    want, flag = _run()
    assert flag == 0
    path = build.build(bounds=True)
    old = kvq.LIB_PATH, kvq._lib
    try:
        kvq.LIB_PATH, kvq._lib = path, None
        got, flag = _run()
        torch.cuda.synchronize()
    finally:
        kvq.LIB_PATH, kvq._lib = old
    assert flag == 0
    for a, b in zip(want, got):
        assert torch.equal(a, b)
