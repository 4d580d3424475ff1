"""kvq_latent_append and kvq_latent_dequant, bit for bit against the definitions
in float64 (tests/latent_reference.py): codes, exponents, rotated parts, the
bytes that a call leaves alone, flags."""
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


def make_cache(B, L, R, page, positions, paged=True, seed=0):
    """A cache over a pool of random bytes (NaN codes among them, as a recycled pool holds)."""
    mp = max(1, -(-positions // page))
    table = torch.randperm(B * mp, generator=torch.Generator().manual_seed(seed)).to(torch.int32).view(B, mp).cuda() if paged else None
    cache = kvq.LatentCache(L, R, page, B * mp, mp, page_table=table)
    cache.pool.random_(0, 256, generator=_gen(seed))
    return cache


def values(shape, seed, spread=0.0):
    x = torch.randn(shape, generator=_gen(seed), device="cuda")
    return (x * torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=_gen(seed + 999), device="cuda"))).to(BF)


def stored(cache, b, n):
    return ref.read_pool(cache.pool, cache.page_table, cache.max_pages_per_seq, b, n, cache.page_size, cache.latent_dim,
                         cache.rope_dim)


def run(L, R, page, start, n, lens=None, H=3, inter=False, paged=True, seed=0, packed=False, table=True, spread=1.0):
    B = len(start)
    cache = make_cache(B, L, R, page, max(start) + n + 9, paged, seed)
    before = cache.pool.clone()
    if packed:
        down = values((B, n, L + R + 8), seed + 1, spread)
        c, k = down[..., :L], down[..., L:L + R]
        q = values((B, n, H, 40 + R), seed + 2)[..., 40:]
        whole = torch.full((B, n, H, L + R), 7.0, dtype=BF, device="cuda")
        q_out = whole[..., L:]
    else:
        c, k, q = values((B, n, L), seed + 1, spread), values((B, n, R), seed + 3, spread), values((B, n, H, R), seed + 2)
        whole = q_out = torch.full((B, n, H, R), 7.0, dtype=BF, device="cuda")
    k_out = torch.full((B, n, R), 5.0, dtype=BF, device="cuda")
    tab = kvq.rope_table(max(start) + n, R) if table else None
    err = _ints([0])
    got = kvq.latent_append(cache, _ints(start), q, c, k, tab, interleaved=inter,
                            new_lens=None if lens is None else _ints(lens), q_out=q_out, k_out=k_out, err=err)
    assert got is q_out and err.item() == 0
    kr = ref.rotate32(k, start, tab, inter) if table else k
    qr = ref.rotate32(q, start, tab, inter) if table else q
    if packed:
        assert (whole[..., :L] == 7.0).all()
    want = before.clone()
    for b in range(B):
        m = n if lens is None else lens[b]
        assert torch.equal(q_out[b, :m], qr[b, :m]) and (q_out[b, m:] == 7.0).all()
        assert torch.equal(k_out[b, :m], kr[b, :m]) and (k_out[b, m:] == 5.0).all()
        codes, e = ref.encode(c[b, :m], kr[b, :m])
        have, have_e = stored(cache, b, start[b] + m)
        assert torch.equal(have[start[b]:], codes) and torch.equal(have_e[start[b]:], e.long())
        # write the expected bytes over the old pool: everything else stays
        G, row = cache.group, L + 2 * R
        t = torch.arange(start[b], start[b] + m, device="cuda")
        phys = (b * cache.max_pages_per_seq + t // page) if cache.page_table is None else cache.page_table[b].long()[t // page]
        lt, ch = (t % G)[:, None], torch.arange(row, device="cuda")[None]
        off = (lt // 8) * (8 * row) + (ch // 16) * 128 + (lt % 8) * 16 + ch % 16
        grp = (t % page) // G
        want[phys[:, None], grp[:, None], off] = cache.pool[phys[:, None], grp[:, None], off]
        want[phys, grp, G * row + t % G] = cache.pool[phys, grp, G * row + t % G]
    assert torch.equal(want, cache.pool)
    return cache


@pytest.mark.parametrize("L", [128, 256, 512])
@pytest.mark.parametrize("R", [32, 64])
@pytest.mark.parametrize("inter", [False, True])
def test_sizes(L, R, inter):
    run(L, R, 64, [0, 5, 70], 37, lens=[37, 0, 20], inter=inter, seed=L + R)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("paged", [False, True])
def test_pages_and_odd_starts(page, paged):
    run(512, 64, page, [0, 1, 7, 8, 15, 63, 255], 19, paged=paged, seed=page)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 300])
def test_packed_projections(n):
    run(256, 64, 32, [3, 0, 40, 9], n, packed=True, seed=n, H=5, inter=n % 2 == 1)


def test_without_rotation_and_without_queries():
    run(512, 32, 64, [0, 11], 21, table=False)
    cache = make_cache(2, 128, 64, 16, 40)
    c, k = values((2, 9, 128), 1), values((2, 9, 64), 2)
    assert kvq.latent_append(cache, _ints([4, 0]), None, c, k, None) is None
    for b, sp in enumerate((4, 0)):
        codes, e = ref.encode(c[b], k[b])
        have, have_e = stored(cache, b, sp + 9)
        assert torch.equal(have[sp:], codes) and torch.equal(have_e[sp:], e.long())


def test_rotation_in_place():
    cache, tab = make_cache(2, 128, 64, 64, 30), kvq.rope_table(40, 64)
    q = values((2, 6, 4, 96), 3)[..., 32:]
    want = ref.rotate32(q, [2, 9], tab, False)
    kvq.latent_append(cache, _ints([2, 9]), q, values((2, 6, 128), 1), values((2, 6, 64), 2), tab, q_out=q)
    assert torch.equal(q, want)


def test_extreme_magnitudes():
    """Every exponent of bf16, amax next to 448 s on both sides, zero and subnormal tokens,
    key parts far above and far below the latent."""
    L, R = 128, 32
    rows = []
    for e in range(-133, 128, 3):
        for f in (1.0, 1.7421875, 1.75, 1.7578125, 1.9921875):
            rows.append(f * 2.0 ** e)
    amax = torch.tensor(rows + [0.0, 2.0 ** -133], dtype=torch.float64, device="cuda").to(BF).double()
    n = amax.numel()
    c = (amax[:, None] * (2 * torch.rand((n, L), generator=_gen(1), device="cuda", dtype=torch.float64) - 1)).to(BF)
    c[:, 3] = amax.to(BF)
    k = (torch.randn((n, R), generator=_gen(2), device="cuda").double() * amax[:, None] *
         torch.exp2(torch.randint(-20, 1, (n, 1), generator=_gen(3), device="cuda").double()) * 0.2).to(BF)
    k[::5] *= 16.0
    k = torch.where(torch.isfinite(k), k, torch.zeros_like(k))
    cache = make_cache(1, L, R, 64, n)
    err = _ints([0])
    kvq.latent_append(cache, _ints([0]), None, c[None].contiguous(), k[None].contiguous(), None, err=err)
    assert err.item() == 0
    codes, e = ref.encode(c, k)
    have, have_e = stored(cache, 0, n)
    assert torch.equal(have_e, e.long()) and torch.equal(have, codes)


def test_a_key_part_is_held_with_all_its_bits():
    """Down to 2^-9 of the token's largest magnitude the key part reads back as it was: the
    largest is over 224 s, E4M3's smallest step is 2^-9 s, and a bf16 value of 2^-2 s and more
    (224 s * 2^-9.8) is a multiple of it.  Below, half a step is 2^-10 s, under 2^-17 of the largest."""
    c = values((1, 500, 512), 5)
    k = values((1, 500, 64), 6)
    cache = make_cache(1, 512, 64, 64, 500)
    kvq.latent_append(cache, _ints([0]), None, c, k, None)
    _, back = kvq.dequant(cache, _ints([500]), 500)
    top = torch.maximum(c.abs().amax(-1), k.abs().amax(-1)).double()[..., None]
    off = (back.double() - k.double()).abs()
    assert (off[k.double().abs() >= 2.0 ** -9 * top.expand_as(off)] == 0).all()
    assert (off <= 2.0 ** -17 * top).all()


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("L,R,page", [(512, 64, 64), (128, 32, 16), (256, 64, 128)])
def test_read_back(dtype, L, R, page):
    lens, most = [0, 1, 100, 77], 100
    cache = make_cache(4, L, R, page, most)
    c, k = values((4, most, L), 1, 1.0), values((4, most, R), 2, 1.0)
    kvq.latent_append(cache, _ints([0] * 4), None, c, k, None, new_lens=_ints(lens))
    err = _ints([0])
    got = kvq.dequant(cache, _ints(lens), most, dtype=dtype, err=err)
    assert err.item() == 0
    for b, n in enumerate(lens):
        codes, e = stored(cache, b, max(n, 1))
        for x, w in zip(got, ref.decode(codes, e, L)):
            assert torch.equal(x[b, :n], w[:n].to(dtype)) and not x[b, n:].any()


def test_a_token_with_inf_or_nan_is_marked():
    cache = make_cache(1, 128, 32, 16, 40)
    c, k = values((1, 40, 128), 1), values((1, 40, 32), 2)
    c[0, 3, 100], c[0, 20, 0], k[0, 33, 31] = float("inf"), float("nan"), float("-inf")
    err = _ints([0])
    kvq.latent_append(cache, _ints([0]), None, c, k, None, err=err)
    assert err.item() == kvq.FLAG_NONFINITE
    codes, e = ref.encode(c[0], k[0])
    have, have_e = stored(cache, 0, 40)
    assert (e[[3, 20, 33]] == 255).all() and torch.equal(have, codes) and torch.equal(have_e, e.long())
    lat, key = kvq.dequant(cache, _ints([40]), 40)
    bad = torch.isnan(lat[0]).all(-1)
    assert bad.nonzero()[:, 0].tolist() == [3, 20, 33] == torch.isnan(key[0]).all(-1).nonzero()[:, 0].tolist()
    assert torch.isfinite(lat[0][~bad]).all()


def test_flags():
    L, R, page = 128, 32, 16
    tab = kvq.rope_table(20, R)
    c, k, q = values((3, 8, L), 1), values((3, 8, R), 2), values((3, 8, 2, R), 3)

    def go(start, lens=None, table=tab, page_table=None):
        cache = make_cache(3, L, R, page, 64, seed=4)
        before = cache.pool.clone()
        out = torch.full_like(q, 9.0)
        err = _ints([0])
        kvq.latent_append(cache, _ints(start), q, c, k, table, new_lens=None if lens is None else _ints(lens), q_out=out,
                          err=err, page_table=page_table)
        return err.item(), cache, before, out

    flag, cache, before, out = go([0, -1, 5], [8, 8, 9])
    assert flag == kvq.FLAG_BAD_LENGTH and (out[1:] == 9.0).all() and not (out[0] == 9.0).any()
    assert (cache.pool != before).any(-1).nonzero()[:, 0].unique().tolist() == [int(cache.page_table[0, 0])]
    flag, cache, before, out = go([0, 14, 30])
    assert flag == kvq.FLAG_POSITION
    assert not (out[1, :6] == 9.0).any() and (out[1, 6:] == 9.0).all() and (out[2] == 9.0).all()
    table = torch.tensor([[0, 1, 2, 3], [4, -1, 6, 7], [8, 12, 10, 11]], dtype=torch.int32, device="cuda")
    flag, cache, before, out = go([0, 12, 12], page_table=table)
    assert flag == kvq.FLAG_PAGE_OOB and torch.equal(out, ref.rotate32(q, [0, 12, 12], tab, False))
    flag, cache, before, out = go([60, 0, 0], table=None)   # past the page table's row
    assert flag == kvq.FLAG_PAGE_OOB


def test_a_pool_past_32_bit_offsets():
    """Pages whose byte offsets pass 2^32."""
    L, R, page, pages = 512, 64, 256, 30000
    assert pages * page * 641 > 2 ** 32
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    cache = kvq.LatentCache(L, R, page, pages, 3, page_table=table)
    c, k = values((1, 600, L), 1), values((1, 600, R), 2)
    kvq.latent_append(cache, _ints([0]), None, c, k, None)
    codes, e = ref.encode(c[0], k[0])
    have, have_e = stored(cache, 0, 600)
    assert torch.equal(have, codes) and torch.equal(have_e, e.long())
    lat, _ = kvq.dequant(cache, _ints([600]), 600)
    assert torch.equal(lat[0].double(), ref.decode(codes, e, L)[0])


def test_refusals():
    cache = make_cache(2, 128, 32, 16, 32)
    c, k, q, tab = values((2, 3, 128), 1), values((2, 3, 32), 2), values((2, 3, 2, 32), 3), kvq.rope_table(40, 32)
    start = _ints([0, 0])
    with pytest.raises(ValueError):
        kvq.latent_append(kvq.Fp8BlockCache(1, 128, 16, 2, 1), start, q, c, k, tab)
    for bad in (dict(c=c[..., :64]), dict(k=k[:, :2]), dict(q=q[..., :16]), dict(c=c.float()), dict(k=k.cpu()),
                dict(start=_ints([0])), dict(start=start.long()), dict(table=kvq.rope_table(40, 64)),
                dict(q_out=torch.empty_like(q)[:, :2]), dict(q=None, q_out=q), dict(k_out=k[..., :16]),
                dict(new_lens=_ints([1])), dict(page_table=_ints([[0, 1]]))):
        args = dict(start=start, q=q, c=c, k=k, table=tab) | bad
        with pytest.raises(ValueError):
            kvq.latent_append(cache, args.pop("start"), args.pop("q"), args.pop("c"), args.pop("k"), args.pop("table"), **args)
    with pytest.raises(ValueError):
        kvq.dequant(cache, start, 4, dtype=torch.float16)
