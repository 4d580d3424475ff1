"""Attention over the 8-bit block cache with weight on chosen positions: the first and
last, both sides of block, page, tile and range borders.  Each case shows by itself
that a zero result, a result without one of those tokens and a result with the token
behind the mask would lie outside the row's bound (tests/attn_bounds.py)."""
import math

import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests import attn_bounds
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def positions(T, page, g, count=14):
    """Up to `count` positions of 0 .. T - 1: ends, both sides of borders, random ones."""
    pick = {0, T - 1, T // 2}
    for step in (16, page, 64, 128, 1024):
        for at in (step, (T // step) * step, (T // step // 2) * step):
            pick |= {at - 1, at}
    pick = sorted(p for p in pick if 0 <= p < T)
    keep = [0, T - 1]
    order = torch.randperm(len(pick), generator=g).tolist()
    for i in order:
        if len(set(keep)) < count:
            keep.append(pick[i])
    return sorted(set(keep))


def planted(T, H, d, page, plants_of, seed):
    """A paged cache of one sequence, filled in chunks: small random keys, and for query
    head g of kv head h a large element of channel 2g at plants_of[g]."""
    g = _gen(seed)
    mp = -(-T // page)
    table = torch.randperm(mp + 3, generator=torch.Generator().manual_seed(seed))[:mp].to(torch.int32).view(1, mp).cuda()
    cache = kvq.Fp8BlockCache(H, d, page, mp + 3, mp, page_table=table)
    cache.pool.random_(0, 256, generator=g)
    for t0 in range(0, T, 16384):
        n = min(16384, T - t0)
        k = torch.randn((1, n, H, d), generator=g, device="cuda") * 0.5
        v = torch.randn((1, n, H, d), generator=g, device="cuda")
        k[..., :16:2] = 0.0
        for c, plants in enumerate(plants_of):
            at = torch.tensor([p - t0 for p in plants if t0 <= p < t0 + n], dtype=torch.long, device="cuda")
            k[:, at, :, 2 * c] = 16.0
        kvq.append(cache, _ints([t0]), k.to(BF), v.to(BF))
    return cache


def queries(rows, H, G, d, T, seed):
    """bf16 [rows][H G][d]: small random elements, and in head g's channel 2g what lifts a
    plant's weight to about 2^5 T of a random token's."""
    q = torch.randn((rows, H, G, d), generator=_gen(seed), device="cuda") * 0.3
    q[..., :16:2] = 0.0
    for g in range(G):
        q[:, :, g, 2 * g] = math.log(32.0 * T) * math.sqrt(d) / 16.0
    return q.reshape(rows, H * G, d).to(BF)


def check(cache, T, q, out, last, plants_of, prefill, dtype):
    rows, hq, d = q.shape
    H = cache.num_kv_heads
    g, scale = hq // H, 1.0 / math.sqrt(d)
    K, V = kvq.dequant(cache, _ints([T]), T)
    blocks = (T + 15) // 16
    pt, G, P = cache.page_table[0].long(), cache.group, cache.page_size
    b = torch.arange(blocks, device="cuda") * 16
    raw = cache.pool[pt[b // P], :, (b % P) // G]                       # [blocks][H][bytes]
    sc = raw[..., 2 * G * d:2 * G * d + G // 2].contiguous().view(torch.float32).view(blocks, H, G // 16, 2)
    vs = sc[torch.arange(blocks, device="cuda"), :, (b % G) // 16, 1].repeat_interleave(16, 0)[:T]
    for h in range(H):
        for i in range(g):
            x = q[:, h * g + i:h * g + i + 1]
            k, v = K[0, :, h].double(), V[0, :, h].double()
            want, p = attn_bounds.attend(x, k, v, scale, last)
            tol = attn_bounds.bound(x, k, v, p, scale, vs[:, h] if prefill else None, dtype, want)
            off = (out[:, h * g + i:h * g + i + 1].double() - want).abs()
            assert (off <= tol).all(), (h, i, (off / tol).max().item())
            # what the bound tells apart, row by row: some channel has to leave it
            assert ((want.abs() > tol).any(-1)).all()
            s = (x[:, 0].double() @ k.T) * scale
            for at in plants_of[i]:
                w = p[:, 0, at]
                seen = w > 0
                without = (want[:, 0] - w[:, None] * v[at]) / (1 - w[:, None]).clamp(min=1e-300)
                gone = ((without - want[:, 0]).abs() > tol[:, 0]).any(-1) | (w > 0.999999)
                assert (gone | ~seen).all(), (h, i, at)
            for r in range(rows):                                       # one token past the mask
                at = int(last[r]) + 1
                if at < T and at in plants_of[i]:
                    e = torch.exp(s[r, at] - torch.logsumexp(s[r, :at], 0))
                    more = (want[r, 0] + e * v[at]) / (1 + e)
                    assert ((more - want[r, 0]).abs() > tol[r, 0]).any(), (h, i, r)


@pytest.mark.parametrize("T,H,G,d,page,dtype", [
    (1, 2, 4, 128, 64, torch.float32), (17, 2, 8, 64, 16, BF), (130, 3, 5, 128, 32, torch.float32),
    (1000, 2, 8, 128, 64, torch.float32), (1000, 2, 3, 64, 256, BF), (5000, 1, 8, 64, 128, torch.float32),
    (20001, 2, 4, 128, 16, BF), (70001, 1, 2, 128, 256, torch.float32), (70001, 1, 3, 64, 64, torch.float32)])
def test_decode(T, H, G, d, page, dtype):
    g = torch.Generator().manual_seed(T)
    plants_of = [positions(T, page, g) for _ in range(G)]
    cache = planted(T, H, d, page, plants_of, seed=T + d)
    q = queries(1, H, G, d, T, seed=3)
    out = torch.empty((1, H * G, d), dtype=dtype, device="cuda")
    err = _ints([0])
    kvq.decode_attn(cache, _ints([T]), q, out=out, err=err)
    assert err.item() == 0
    check(cache, T, q, out, torch.tensor([T - 1]), plants_of, False, dtype)


@pytest.mark.parametrize("T,n,H,G,d,page,dtype", [
    (5, 5, 2, 4, 128, 64, torch.float32), (130, 33, 2, 8, 64, 16, BF), (300, 300, 1, 4, 128, 32, torch.float32),
    (1000, 1, 2, 8, 128, 64, torch.float32), (2600, 70, 1, 3, 64, 256, torch.float32), (2600, 200, 1, 8, 128, 64, BF),
    (9001, 5, 2, 8, 128, 16, torch.float32), (40001, 20, 1, 2, 128, 128, torch.float32), (40001, 9, 1, 8, 64, 64, BF)])
def test_prefill(T, n, H, G, d, page, dtype):
    """Plants at the mask's edge of some rows too: a row's last position, the one behind it."""
    g = torch.Generator().manual_seed(T + n)
    plants_of = [sorted(set(positions(T, page, g, 10)) | {T - n, T - 1 - n // 2, min(T - 1, T - n // 2)}) for _ in range(G)]
    cache = planted(T, H, d, page, plants_of, seed=T + d)
    q = queries(n, H, G, d, T, seed=4)
    out = torch.empty((1, n, H * G, d), dtype=dtype, device="cuda")
    err = _ints([0])
    kvq.prefill_attn(cache, _ints([T]), q[None].contiguous(), out=out, err=err)
    assert err.item() == 0
    check(cache, T, q, out[0], torch.arange(T - n, T), plants_of, True, dtype)


def test_decode_and_prefill_agree_within_their_bounds():
    T, H, G, d = 1000, 2, 4, 128
    g = torch.Generator().manual_seed(1)
    plants_of = [positions(T, 64, g) for _ in range(G)]
    cache = planted(T, H, d, 64, plants_of, seed=2)
    q = queries(1, H, G, d, T, seed=5)
    a = kvq.decode_attn(cache, _ints([T]), q)
    b = kvq.prefill_attn(cache, _ints([T]), q[None].contiguous())[0]
    K, V = kvq.dequant(cache, _ints([T]), T)
    vmax = V[0].abs().amax(-1).double()  # a block's scale is over 1 and under 2 448ths of its largest value
    for h in range(H):
        rows = slice(h * G, (h + 1) * G)
        want, p = attn_bounds.attend(q[:, rows], K[0, :, h], V[0, :, h], 1 / math.sqrt(d), torch.tensor([T - 1]))
        scale = torch.stack([vmax[i // 16 * 16:i // 16 * 16 + 16, h].amax() for i in range(T)]) * 2 / 448
        tol = sum(attn_bounds.bound(q[:, rows], K[0, :, h], V[0, :, h], p, 1 / math.sqrt(d), s, v_least=l)
                  for s, l in ((None, None), (scale, scale / 2)))
        assert ((a[:, rows].double() - b[:, rows].double()).abs() <= tol).all()
        assert (tol < 0.05 * want.abs().amax()).all()
