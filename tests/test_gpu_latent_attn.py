"""Attention over the latent cache (kvq_latent_attn: one token per sequence and
chunks) against float64 attention over the values that the cache holds
(tests/latent_reference.py reads the pool's bytes), row by row against
latent_reference.attn_bound."""
import math

import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests import latent_reference as ref
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


def build(lens, L, R, page, paged=True, seed=0, k_scale=1.0, c_scale=1.0, spread=0.4, spare=0):
    """A cache filled through kvq.latent_append over a pool of random bytes."""
    B, g = len(lens), _gen(seed)
    mp = max(1, -(-(max(lens) + spare) // page))
    table = torch.randperm(B * mp, generator=torch.Generator().manual_seed(seed)).to(torch.int32).view(B, mp).cuda() if paged else None
    cache = kvq.LatentCache(L, R, page, B * mp, mp, page_table=table)
    cache.pool.random_(0, 256, generator=g)
    n = max(max(lens), 1)
    for b in range(B):  # a sequence at a time: long ones do not make the batch's inputs large
        m = lens[b]
        if m == 0:
            continue
        c = torch.randn((1, m, L), generator=g, device="cuda") * c_scale
        c[..., [1, L // 2]] *= 4.0
        c *= torch.exp(spread * torch.randn((1, m, 1), generator=g, device="cuda"))
        k = torch.randn((1, m, R), generator=g, device="cuda") * k_scale
        row = None if table is None else table[b:b + 1].contiguous()
        if row is None:
            row = torch.arange(b * mp, (b + 1) * mp, dtype=torch.int32, device="cuda")[None]
        kvq.latent_append(cache, _ints([0]), None, c.to(BF), k.to(BF), None, page_table=row)
    return cache


def queries(B, n, H, L, R, seed, q_scale=1.0):
    return (torch.randn((B, n, H, L + R), generator=_gen(seed), device="cuda") * q_scale).to(BF)


def check(out, q, cache, lens, n_of, scale):
    """out [B][n][H][L] against the definition; n_of[b] valid rows of sequence b."""
    L, R, worst = cache.latent_dim, cache.rope_dim, 0.0
    for b, T in enumerate(lens):
        n = n_of[b]
        if n == 0:
            continue
        got = out[b, :n].double()
        if T == 0:
            assert not got.any()
            continue
        codes, e = ref.read_pool(cache.pool, cache.page_table, cache.max_pages_per_seq, b, T, cache.page_size, L, R)
        c, k = ref.decode(codes, e, L)
        s = ref.power(e - 127)
        H = q.shape[2]
        step = max(1, (1 << 24) // (H * T))
        for i in range(0, n, step):
            x = q[b, i:min(n, i + step)]
            last = torch.arange(T - n + i, T - n + i + x.shape[0]).repeat_interleave(H)
            x = x.reshape(-1, L + R)
            p = ref.weights(x, torch.cat([c, k], -1), scale, last)
            want = p @ c
            tol = ref.attn_bound(x, c, k, s, p, scale, out.dtype, want)
            off = (got[i:i + step].reshape(-1, L) - want).abs()
            assert (off <= tol).all(), (b, i, (off / tol).nan_to_num(9e9).max().item())
            worst = max(worst, (off / tol).nan_to_num(0.0).max().item())
    return worst


def decode(lens, H, L, R, page, seed=0, dtype=torch.float32, scale=None, q_scale=0.5, **kw):
    cache = build(lens, L, R, page, seed=seed, **kw)
    q = queries(len(lens), 1, H, L, R, seed + 1, q_scale)
    scale = 1.0 / math.sqrt(128 + R) if scale is None else scale
    err = _ints([0])
    out = torch.full((len(lens), H, L), float("nan"), dtype=dtype, device="cuda")
    assert kvq.decode_attn(cache, _ints(lens), q[:, 0], scale, out=out, err=err) is out
    assert err.item() == 0
    return check(out[:, None], q, cache, lens, [1] * len(lens), scale)


def chunk(lens, n_of, n, H, L, R, page, seed=0, dtype=BF, scale=None, q_scale=0.5, **kw):
    cache = build(lens, L, R, page, seed=seed, **kw)
    B = len(lens)
    q = queries(B, n, H, L, R, seed + 1, q_scale)
    scale = 1.0 / math.sqrt(128 + R) if scale is None else scale
    err = _ints([0])
    out = torch.full((B, n, H, L), 3.0, dtype=dtype, device="cuda")
    pad = None if n_of is None else _ints(n_of)
    n_of = [n] * B if n_of is None else n_of
    kvq.prefill_attn(cache, _ints(lens), q, scale, out=out, chunk_lens=pad, err=err)
    assert err.item() == 0
    for b in range(B):
        assert (out[b, n_of[b]:] == 3.0).all()
    return check(out, q, cache, lens, n_of, scale)


@pytest.mark.parametrize("L,R", [(128, 32), (128, 64), (256, 32), (256, 64), (512, 32), (512, 64)])
@pytest.mark.parametrize("H", [1, 16, 40, 128])
def test_decode_sizes(L, R, H):
    decode([1, 300, 17, 64], H, L, R, 64, seed=H, dtype=BF if H % 16 else torch.float32)


@pytest.mark.parametrize("H", [2, 3, 7, 15, 17, 31, 33, 63, 64, 65, 96, 127, 130, 200])
def test_decode_heads(H):
    decode([70, 0, 129], H, 256, 64, 32, seed=H)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("paged", [False, True])
def test_decode_pages_and_odd_lengths(page, paged):
    decode([1, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 0, 1000, 255], 16, 512, 64, page, seed=page, paged=paged)


def test_decode_many_short_sequences():
    g = torch.Generator().manual_seed(5)
    decode(torch.randint(0, 90, (400,), generator=g).tolist(), 8, 128, 64, 16, seed=6)


def test_decode_long_and_short():
    decode([70001, 3, 0, 9000], 20, 512, 64, 256, seed=7)
    decode([30011], 128, 512, 64, 64, seed=8, dtype=BF)


@pytest.mark.parametrize("scale,q_scale,k_scale,c_scale", [
    (0.003, 1.0, 1.0, 1.0), (1.0, 1.0, 1.0, 1.0), (0.1, 1e-20, 1e18, 1e18), (0.1, 1e15, 1e-15, 1e-15),
    (0.1, 0.5, 30.0, 1.0), (0.1, 0.5, 0.01, 1.0)])
def test_decode_ranges(scale, q_scale, k_scale, c_scale):
    """Flat and peaked weights; extreme magnitudes; key parts far above and below the latent."""
    decode([500, 33], 20, 256, 64, 64, seed=9, scale=scale, q_scale=q_scale, k_scale=k_scale, c_scale=c_scale)


def test_decode_values_of_very_different_tokens():
    """Scales over many binades: a row's precision goes by what it attends."""
    decode([700, 129], 24, 512, 64, 64, seed=10, spread=6.0, q_scale=1e-3)
    decode([700, 129], 24, 128, 32, 64, seed=11, spread=20.0, q_scale=1e-9)


@pytest.mark.parametrize("L,R,H", [(512, 64, 16), (512, 32, 128), (256, 64, 20), (128, 32, 5)])
@pytest.mark.parametrize("n", [1, 2, 5, 33, 130])
def test_chunks(L, R, H, n):
    chunk([n, n + 1, n + 63, 900], None, n, H, L, R, 64, seed=n + H)


def test_chunks_of_a_padded_batch():
    chunk([300, 64, 17, 500, 5], [40, 64, 0, 1, 5], 64, 12, 256, 64, 16, seed=3)
    chunk([1000, 7], [200, 3], 200, 64, 512, 64, 128, seed=4, dtype=torch.float32)


def test_a_prompt_of_its_own():
    chunk([777], None, 777, 16, 512, 64, 64, seed=5)


def test_padded_chunk_of_one():
    chunk([300, 64, 9], [1, 0, 1], 1, 16, 512, 64, 64, seed=6)


def planted(T, seed, L=256, R=64):
    """A cache whose latents are position marks: token t has 1 at channel t % L, and keys that single queries pick."""
    cache = build([T], L, R, 64, seed=seed, c_scale=1.0, spread=0.0)
    return cache


def test_each_position_counts():
    """A query with nearly all its weight on one chosen position returns that token: first
    and last positions, tile and page borders.  A lost or shifted token leaves the bound."""
    T, L, R = 4100, 256, 64
    cache = planted(T, 12)
    codes, e = ref.read_pool(cache.pool, cache.page_table, cache.max_pages_per_seq, 0, T, 64, L, R)
    c, k = ref.decode(codes, e, L)
    at = [0, 1, 7, 8, 31, 32, 63, 64, 127, 128, 2047, 2048, 2049, 4031, 4032, 4095, 4096, 4098, 4099]
    q = (torch.cat([c, k], -1)[at] * 0.5).to(BF)[None]                      # [1][heads][L + R]
    out = kvq.decode_attn(cache, _ints([T]), q, 1.0)
    p = ref.weights(q[0], torch.cat([c, k], -1), 1.0, torch.full((len(at),), T - 1))
    assert (p.amax(-1) > 0.99).all() and p.argmax(-1).tolist() == at
    check(out[:, None], q[:, None], cache, [T], [1], 1.0)


def test_a_sink_leaves_the_rest_its_precision():
    """One token with nearly all the weight and a tiny value beside thousands of equal ones at
    2^-17 of it: their sum survives."""
    T, L, R = 5000, 512, 64
    g = _gen(13)
    c = torch.randn((1, T, L), generator=g, device="cuda")
    k = torch.zeros((1, T, R), device="cuda")
    c[0, 0] *= 1e-4
    k[0, 0, 0] = 11.8 * 2
    cache = kvq.LatentCache(L, R, 64, 80, 80)
    kvq.latent_append(cache, _ints([0]), None, c.to(BF), k.to(BF), None)
    q = torch.zeros((1, 16, L + R), dtype=BF, device="cuda")
    q[..., L] = 0.5
    out = kvq.decode_attn(cache, _ints([T]), q, 1.0)
    check(out[:, None], q[:, None], cache, [T], [1], 1.0)
    codes, e = ref.read_pool(cache.pool, None, 80, 0, T, 64, L, R)
    lat, key = ref.decode(codes, e, L)
    p = ref.weights(q[0], torch.cat([lat, key], -1), 1.0, torch.full((16,), T - 1))
    want = p @ lat
    assert ((out[0].double() - want).norm() / want.norm()).item() < 0.05


def test_causal_rows_do_not_see_later_tokens():
    """Tokens behind a row change nothing in it, whatever they hold."""
    T, n, H, L, R = 200, 70, 20, 256, 64
    a, b = build([T], L, R, 64, seed=14), build([T], L, R, 64, seed=14)
    c = torch.randn((1, 1, L), generator=_gen(1), device="cuda").to(BF) * 1000
    k = torch.randn((1, 1, R), generator=_gen(2), device="cuda").to(BF) * 1000
    nan = torch.full((1, 1, L), float("nan"), dtype=BF, device="cuda")
    kvq.latent_append(b, _ints([150]), None, c, k, None)
    kvq.latent_append(b, _ints([180]), None, nan, k, None)
    q = queries(1, n, H, L, R, 15)
    x, y = (kvq.prefill_attn(m, _ints([T]), q, 0.1) for m in (a, b))
    assert torch.equal(x[:, :20], y[:, :20])                    # rows at positions 130 .. 149
    assert torch.isfinite(y[:, :50]).all() and torch.isnan(y[:, 50:]).all()


def test_nan_queries_stay_in_their_rows():
    cache = build([300, 40], 512, 64, 64, seed=16)
    q = queries(2, 1, 20, 512, 64, 17)[:, 0]
    want = kvq.decode_attn(cache, _ints([300, 40]), q, 0.1)
    bad = q.clone()
    bad[0, 3, 5], bad[1, 19, 570] = float("nan"), float("inf")
    got = kvq.decode_attn(cache, _ints([300, 40]), bad, 0.1)
    assert torch.isnan(got[0, 3]).all() and torch.isnan(got[1, 19]).all()
    keep = torch.ones((2, 20), dtype=torch.bool)
    keep[0, 3] = keep[1, 19] = False
    assert torch.equal(got[keep.cuda()], want[keep.cuda()])


def test_flags_and_missing_pages():
    L, R, H = 256, 64, 16
    cache = build([100, 100, 100], L, R, 16, seed=18)
    q = queries(3, 1, H, L, R, 19)
    err = _ints([0])
    out = torch.full((3, H, L), 3.0, device="cuda")
    kvq.decode_attn(cache, _ints([100, -1, 0]), q[:, 0], 0.1, out=out, err=err)
    assert err.item() == kvq.FLAG_BAD_LENGTH and not out[1:].any()
    check(out[:1, None], q[:1], cache, [100], [1], 0.1)
    # a chunk longer than its sequence; a chunk length out of range
    err.zero_()
    qc = queries(3, 7, H, L, R, 20)
    out = torch.full((3, 7, H, L), 3.0, device="cuda")
    kvq.prefill_attn(cache, _ints([3, 50, 100]), qc, 0.1, out=out, chunk_lens=_ints([5, 8, 7]), err=err)
    assert err.item() == kvq.FLAG_BAD_LENGTH
    assert not out[0, :5].any() and (out[0, 5:] == 3.0).all() and (out[1] == 3.0).all()
    check(out[2:], qc[2:], _view(cache, 2), [100], [7], 0.1)
    # a page that is not there: its tokens are left out
    err.zero_()
    table = cache.page_table.clone()
    cache.page_table = table
    good = cache.page_table[0, 2].item()
    table[0, 2] = cache.num_pages
    got = kvq.decode_attn(cache, _ints([100, 100, 100]), q[:, 0], 0.1, err=err)
    assert err.item() == kvq.FLAG_PAGE_OOB
    table[0, 2] = good
    codes, e = ref.read_pool(cache.pool, table, cache.max_pages_per_seq, 0, 100, 16, L, R)
    c, k = ref.decode(codes, e, L)
    keep = torch.ones(100, dtype=torch.bool)
    keep[32:48] = False
    c, k, s = c[keep], k[keep], ref.power(e[keep] - 127)
    p = ref.weights(q[0, 0], torch.cat([c, k], -1), 0.1, torch.full((H,), 83))
    assert ((got[0].double() - p @ c).abs() <= ref.attn_bound(q[0, 0], c, k, s, p, 0.1)).all()
    # lengths past what the page table holds
    err.zero_()
    got = kvq.decode_attn(cache, _ints([10 ** 9, 100, 100]), q[:, 0], 0.1, err=err)
    assert err.item() == kvq.FLAG_PAGE_OOB and torch.isfinite(got[1:]).all()


def _view(cache, b):
    """The cache of sequence b alone."""
    return kvq.LatentCache(cache.latent_dim, cache.rope_dim, cache.page_size, cache.num_pages, cache.max_pages_per_seq,
                           page_table=cache.page_table[b:b + 1].contiguous(), pool=cache.pool)


def test_all_pages_missing_gives_zero_rows():
    cache = build([100], 128, 64, 16, seed=21)
    cache.page_table = torch.full_like(cache.page_table, -1)
    err = _ints([0])
    out = torch.full((1, 9, 128), 3.0, device="cuda")
    kvq.decode_attn(cache, _ints([100]), queries(1, 1, 9, 128, 64, 22)[:, 0], 0.1, out=out, err=err)
    assert err.item() == kvq.FLAG_PAGE_OOB and not out.any()


def test_repeated_calls_give_the_same_bytes():
    cache = build([5000, 333, 64], 512, 64, 64, seed=23)
    q = queries(3, 3, 40, 512, 64, 24)
    ws = torch.empty(kvq.latent_workspace_bytes(3, 40, 512, 3), dtype=torch.uint8, device="cuda")
    want = kvq.prefill_attn(cache, _ints([5000, 333, 64]), q, 0.1)
    for _ in range(20):
        ws.random_(0, 256)
        assert torch.equal(want, kvq.prefill_attn(cache, _ints([5000, 333, 64]), q, 0.1, workspace=ws))


def test_refusals():
    cache = build([20], 128, 32, 16, seed=25)
    q, lens = queries(1, 1, 4, 128, 32, 26)[:, 0], _ints([20])
    for bad in (dict(q=q[..., :128]), dict(q=q.float()), dict(q=q[:, None]), dict(lens=lens.long()), dict(scale=None),
                dict(out=torch.empty((1, 4, 160), device="cuda")), dict(out=torch.empty((1, 4, 128), device="cuda", dtype=torch.float16)),
                dict(lens=_ints([20, 20])), dict(swa=object()), dict(kernel="tcgen05")):
        args = dict(lens=lens, q=q, scale=0.1) | bad
        with pytest.raises(ValueError):
            kvq.decode_attn(cache, args.pop("lens"), args.pop("q"), args.pop("scale"), **args)
    with pytest.raises(ValueError):
        kvq.prefill_attn(cache, lens, q, 0.1)
    with pytest.raises(kvq.KvqError):
        kvq.decode_attn(cache, lens, q, 0.1, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
