"""Attention over the 8-bit block cache (kvq_fp8_block_decode_attn and
kvq_fp8_block_prefill_attn) against float64 attention over the cache's
dequantised values (kvq_fp8_block_dequant, itself checked bit for bit), with
the tolerance of block8_reference.tolerance, counted from the roundings."""
import math

import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests import block8_reference as ref
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


def build(lens, H, d, page, paged=True, seed=0, k_scale=1.0, v_spread=0.5, spare=0):
    """A cache filled through kvq.append from a pool of random bytes (NaN codes
    and scales among them, as a recycled pool holds)."""
    B, g = len(lens), _gen(seed)
    mp = max(1, -(-(max(lens) + spare) // page))
    table = torch.randperm(B * mp, generator=torch.Generator().manual_seed(seed)).to(torch.int32).view(B, mp).cuda() if paged else None
    cache = kvq.Fp8BlockCache(H, d, page, B * mp, mp, page_table=table)
    cache.pool.random_(0, 256, generator=g)
    n = max(max(lens), 1)
    k = torch.randn((B, n, H, d), generator=g, device="cuda") * k_scale
    k[..., [1, d // 2]] *= 4.0
    v = torch.randn((B, n, H, d), generator=g, device="cuda")
    v *= torch.exp(v_spread * torch.randn((B, n, H, 1), generator=g, device="cuda"))
    kvq.append(cache, _ints([0] * B), k.to(BF), v.to(BF), new_lens=_ints(lens))
    return cache


def check(out, q, cache, lens, n_of, scale, prefill):
    """out, q [B][c][Hq][d]; n_of[b] valid rows of sequence b."""
    B, c, hq, d = q.shape
    g = hq // cache.num_kv_heads
    worst = 0.0
    K, V = kvq.dequant(cache, _ints(lens), max(max(lens), 1))
    for b in range(B):
        n, T = n_of[b], lens[b]
        if n == 0:
            continue
        last = torch.arange(T - n, T)
        for h in range(cache.num_kv_heads):
            rows = q[b, :n, h * g:(h + 1) * g]
            v = V[b, :T, h]
            want, A, bq = ref.attend(rows, K[b, :T, h], v, scale, last)
            got = out[b, :n, h * g:(h + 1) * g].double()
            if T == 0:
                assert not got.any()
                continue
            tol = ref.tolerance(d, T, float(v.abs().max()), A, bq if prefill else None, out.dtype, want.abs())
            off = (got - want).abs()
            assert (off <= tol).all(), (b, h, (off / tol).max().item())
            worst = max(worst, (off / tol).nan_to_num(0.0).max().item())
    return worst


def decode(lens, H, G, d, page, seed=0, dtype=torch.float32, scale=None, q_scale=1.0, **kw):
    cache = build(lens, H, d, page, seed=seed, **kw)
    q = (torch.randn((len(lens), H * G, d), generator=_gen(seed + 1), device="cuda") * q_scale).to(BF)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    err = _ints([0])
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    kvq.decode_attn(cache, _ints(lens), q, scale, out=out, err=err)
    assert err.item() == 0
    return check(out[:, None], q[:, None], cache, lens, [1] * len(lens), scale, False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_decode_heads(d, G):
    decode([1, 300, 17, 64], 2, G, d, 64, seed=G, dtype=BF if G % 2 else torch.float32)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("paged", [False, True])
def test_decode_pages_and_odd_lengths(page, paged):
    decode([1, 15, 16, 17, 63, 64, 65, 127, 129, 0, 1000, 255], 3, 4, 128, page, seed=page, paged=paged)


def test_decode_many_short_and_one_long():
    g = torch.Generator().manual_seed(5)
    decode(torch.randint(0, 90, (300,), generator=g).tolist(), 2, 8, 64, 16, seed=6)
    decode([70001, 3], 1, 2, 128, 256, seed=7)


@pytest.mark.parametrize("scale,q_scale,k_scale", [(0.01, 1.0, 1.0), (1.0, 1.0, 1.0), (0.1, 1e-20, 1e20), (0.1, 1e15, 1e-15)])
def test_decode_ranges(scale, q_scale, k_scale):
    """Flat and peaked weights; queries and keys of extreme magnitudes."""
    decode([500, 33], 2, 4, 128, 64, seed=8, scale=scale, q_scale=q_scale, k_scale=k_scale)


def test_decode_values_of_very_different_blocks():
    """V blocks over many binades, some all zero (scale 2^-126), beside an
    attention sink."""
    cache = build([400], 2, 128, 64, seed=9, v_spread=6.0)
    g = _gen(10)
    z = torch.zeros((1, 32, 2, 128), dtype=BF, device="cuda")
    k = torch.randn((1, 32, 2, 128), generator=g, device="cuda").to(BF)
    kvq.append(cache, _ints([0]), k, z)
    q = torch.randn((1, 1, 16, 128), generator=g, device="cuda").to(BF)
    for lens in ([400], [32], [20]):
        out = kvq.decode_attn(cache, _ints(lens), q[:, 0].contiguous())
        check(out[:, None], q, cache, lens, [1], 1 / math.sqrt(128), False)
        pre = kvq.prefill_attn(cache, _ints(lens), q)
        check(pre, q, cache, lens, [1], 1 / math.sqrt(128), True)
    assert not kvq.decode_attn(cache, _ints([20]), q[:, 0].contiguous()).any()


def prefill(lens, n, H, G, d, page, seed=0, dtype=torch.float32, ragged=None, scale=None, q_scale=1.0, **kw):
    cache = build(lens, H, d, page, seed=seed, **kw)
    B = len(lens)
    q = (torch.randn((B, n, H * G, d), generator=_gen(seed + 1), device="cuda") * q_scale).to(BF)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    err = _ints([0])
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    kvq.prefill_attn(cache, _ints(lens), q, scale, out=out, err=err, chunk_lens=None if ragged is None else _ints(ragged))
    assert err.item() == 0
    n_of = [n] * B if ragged is None else ragged
    for b in range(B):
        assert (out[b, n_of[b]:] == 7.0).all()  # padding rows stay as they were
    return check(out, q, cache, lens, n_of, scale, True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_prefill_heads(d, G):
    prefill([300, 181], 70, 2, G, d, 64, seed=G, dtype=BF if G % 2 else torch.float32)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("paged", [False, True])
def test_prefill_pages(page, paged):
    prefill([520, 129, 40], 40, 2, 8, 128, page, seed=page, paged=paged)


@pytest.mark.parametrize("n,lens", [(1, [1, 128, 129, 1000]), (2, [2, 17]), (128, [128, 255]), (129, [129, 300]),
                                    (300, [300, 700]), (33, [5000])])
def test_prefill_chunk_lengths(n, lens):
    """One token, chunks that are the whole cache, chunks around a tile; few
    rows (the positions split over CTAs) and many."""
    prefill(lens, n, 2, 8, 128, 64, seed=n)
    prefill(lens, n, 1, 1, 64, 16, seed=n + 1, dtype=BF)


@pytest.mark.parametrize("d,G,page,n", [(128, 8, 64, 5), (64, 3, 16, 40), (128, 1, 32, 128), (64, 8, 256, 1)])
def test_prefill_few_rows_over_many_tiles(d, G, page, n):
    """More (sequence, head) units than SMs: one CTA walks all of a unit's tiles, from
    one to 21, with its two halves at every second one."""
    lens = [max(n, x) for x in (1, 127, 128, 129, 256, 257, 385, 512, 640, 641, 900, 1024, 1300, 2001, 2600)] * 3
    prefill(lens, n, 4, G, d, page, seed=n, ragged=[n - i % min(n, 3) for i in range(len(lens))])

def test_prefill_without_a_split():
    """A grid larger than the GPU: one CTA walks all positions of its rows."""
    prefill([900, 650], 640, 8, 8, 128, 64, seed=21)
    prefill([900, 650, 700], 640, 8, 8, 64, 32, seed=22, ragged=[640, 3, 511])


def test_prefill_padded_batches():
    prefill([300, 64, 700, 5], 50, 2, 4, 128, 32, seed=3, ragged=[50, 0, 1, 5])
    prefill([90, 0, 33], 33, 1, 7, 64, 64, seed=4, ragged=[20, 0, 33], dtype=BF)


@pytest.mark.parametrize("scale,q_scale,k_scale", [(0.01, 1.0, 1.0), (1.0, 1.0, 1.0), (0.1, 1e-20, 1e20), (0.1, 1e15, 1e-15)])
def test_prefill_ranges(scale, q_scale, k_scale):
    prefill([500, 133], 30, 2, 4, 128, 64, seed=8, scale=scale, q_scale=q_scale, k_scale=k_scale)


def test_prefill_values_over_many_binades():
    prefill([1000], 200, 2, 8, 128, 64, seed=9, v_spread=5.0)


def test_rising_scores():
    """Scores that rise along the positions raise the running maximum in every
    tile and block (and in the second half of a tile)."""
    for d in (64, 128):
        T, H, G = 700, 1, 8
        k = torch.zeros((1, T, H, d), device="cuda")
        k[..., 0] = torch.arange(T, device="cuda")[None, :, None] * 0.5
        v = torch.randn((1, T, H, d), generator=_gen(3), device="cuda")
        cache = kvq.Fp8BlockCache(H, d, 64, 11, 11)
        kvq.append(cache, _ints([0]), k.to(BF), v.to(BF))
        q = torch.zeros((1, 90, H * G, d), dtype=BF, device="cuda")
        q[..., 0] = torch.linspace(0.1, 4.0, 90 * G, device="cuda").view(1, 90, G).to(BF)
        out = kvq.prefill_attn(cache, _ints([T]), q, 1.0)
        check(out, q, cache, [T], [90], 1.0, True)
        dec = kvq.decode_attn(cache, _ints([T]), q[:, 5].contiguous(), 1.0)
        check(dec[:, None], q[:, 5:6], cache, [T], [1], 1.0, False)


def test_imported_scales():
    """Readers take any finite scale, not only powers of two (and zero)."""
    cache = build([200], 2, 128, 64, seed=12)
    G = cache.group
    sc = cache.pool[..., 2 * G * 128:].view(torch.float32)
    sc.copy_(torch.rand(sc.shape, generator=_gen(13), device="cuda") * 0.01 + 0.001)
    sc[0, 0, 0, :2] = 0.0
    cache.pool[..., :2 * G * 128].copy_((cache.pool[..., :2 * G * 128] & 0x80) | (cache.pool[..., :2 * G * 128] & 0x7F).clamp(max=0x7E))
    q = torch.randn((1, 40, 8, 128), generator=_gen(14), device="cuda").to(BF)
    dec = kvq.decode_attn(cache, _ints([200]), q[:, 0].contiguous())
    check(dec[:, None], q[:, :1], cache, [200], [1], 1 / math.sqrt(128), False)
    # (the prefill rounds sV / sV_ref and its product with a code to f16: 2^-11 each, inside 2 x 2^-11 more)
    out = kvq.prefill_attn(cache, _ints([200]), q)
    K, V = kvq.dequant(cache, _ints([200]), 200)
    for h in range(2):
        want, A, bq = ref.attend(q[0, :, 4 * h:4 * h + 4], K[0, :, h], V[0, :, h], 1 / math.sqrt(128), torch.arange(160, 200))
        vmax = float(V[0, :, h].abs().max())
        tol = ref.tolerance(128, 200, vmax, A, bq) + 2 * 2.0 ** -11 * vmax
        assert (out[0, :, 4 * h:4 * h + 4].double() - want).abs().max().item() <= tol


def test_bad_pages_are_left_out():
    """A page that is not valid loses its tokens and nothing else."""
    H, G, d = 2, 4, 128
    for page, bad in ((16, 3), (32, 1), (64, 2), (128, 1)):
        T = 300
        cache = build([T, T], H, d, page, seed=page)
        q = torch.randn((2, 20, H * G, d), generator=_gen(1), device="cuda").to(BF)
        K, V = kvq.dequant(cache, _ints([T, T]), T)
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[bad * page:(bad + 1) * page] = False
        for value in (-1, cache.num_pages, 1 << 30):
            saved = cache.page_table.clone()
            cache.page_table[0, bad] = value
            e1, e2, e3 = _ints([0]), _ints([0]), _ints([0])
            dec = kvq.decode_attn(cache, _ints([T, T]), q[:, -1].contiguous(), err=e1)
            pre = kvq.prefill_attn(cache, _ints([T, T]), q, err=e2)
            kd, _ = kvq.dequant(cache, _ints([T, T]), T, err=e3)
            assert e1.item() == e2.item() == e3.item() == kvq.FLAG_PAGE_OOB
            assert not kd[0, ~keep].any() and torch.equal(kd[0, keep], K[0, keep]) and torch.equal(kd[1], K[1])
            cache.page_table.copy_(saved)
            for b in range(2):
                ok = keep if b == 0 else torch.ones_like(keep)
                at = torch.nonzero(ok)[:, 0]
                for h in range(H):
                    last = (at[None] <= torch.arange(T - 20, T, device="cuda")[:, None]).sum(1) - 1
                    want, A, bq = ref.attend(q[b, :, h * G:(h + 1) * G], K[b, at, h], V[b, at, h], 1 / math.sqrt(d), last)
                    tol = ref.tolerance(d, T, float(V[b, :, h].abs().max()), A, bq)
                    assert (pre[b, :, h * G:(h + 1) * G].double() - want).abs().max() <= tol
                    assert (dec[b, h * G:(h + 1) * G].double() - want[-1]).abs().max() <= tol


def test_bad_lengths():
    cache = build([100, 100], 2, 64, 32, seed=2)
    q = torch.randn((2, 10, 4, 64), generator=_gen(1), device="cuda").to(BF)
    good = kvq.prefill_attn(cache, _ints([100, 100]), q)
    dgood = kvq.decode_attn(cache, _ints([100, 100]), q[:, 0].contiguous())
    err = _ints([0])
    out = kvq.prefill_attn(cache, _ints([100, 9]), q, err=err)      # shorter than the chunk
    assert err.item() == kvq.FLAG_BAD_LENGTH and not out[1].any() and torch.equal(out[0], good[0])
    for n in (-1, 11):
        err, out = _ints([0]), torch.full(q.shape, 7.0, device="cuda")
        kvq.prefill_attn(cache, _ints([100, 100]), q, out=out, err=err, chunk_lens=_ints([10, n]))
        assert err.item() == kvq.FLAG_BAD_LENGTH and (out[1] == 7.0).all() and torch.equal(out[0], good[0])
    err = _ints([0])
    out = kvq.decode_attn(cache, _ints([100, -5]), q[:, 0].contiguous(), err=err)
    assert err.item() == kvq.FLAG_BAD_LENGTH and not out[1].any() and torch.equal(out[0], dgood[0])
    err = _ints([0])
    out = kvq.decode_attn(cache, _ints([100, 200]), q[:, 0].contiguous(), err=err)  # past the page table
    assert err.item() == kvq.FLAG_PAGE_OOB and torch.equal(out[0], dgood[0])
    err = _ints([0])
    out = kvq.prefill_attn(cache, _ints([100, 5000]), q, err=err)
    assert err.item() == kvq.FLAG_PAGE_OOB and torch.equal(out[0], good[0])
    err = _ints([0])
    kd, _ = kvq.dequant(cache, _ints([100, -1]), 50, err=err)
    assert err.item() == kvq.FLAG_BAD_LENGTH and not kd[1].any()


def test_nonfinite_queries_stay_in_their_rows():
    cache = build([200], 1, 128, 64, seed=4)
    q = torch.randn((1, 4, 4, 128), generator=_gen(2), device="cuda").to(BF)
    good, dgood = kvq.prefill_attn(cache, _ints([200]), q), kvq.decode_attn(cache, _ints([200]), q[:, 3].contiguous())
    for value in (float("nan"), float("inf")):
        x = q.clone()
        x[0, 3, 1, 7] = value
        out, dec = kvq.prefill_attn(cache, _ints([200]), x), kvq.decode_attn(cache, _ints([200]), x[:, 3].contiguous())
        assert out[0, 3, 1].isnan().all() and dec[0, 1].isnan().all()
        keep = [0, 2, 3]
        assert torch.equal(out[0, :3], good[0, :3]) and torch.equal(out[0, 3, keep], good[0, 3, keep])
        assert torch.equal(dec[0, keep], dgood[0, keep])


@pytest.mark.parametrize("lens", [[16, 40], [3, 9000]])
def test_nan_keys_reach_their_rows(lens):
    """A sequence whose keys are all NaN gives NaN, also where a warp or a range has
    seen no other score; the other sequence stays as it is."""
    H, G, d = 2, 4, 128
    cache = build(lens, H, d, 64, seed=21)
    q = torch.randn((2, H * G, d), generator=_gen(22), device="cuda").to(BF)
    want = kvq.decode_attn(cache, _ints(lens), q)
    pre = kvq.prefill_attn(cache, _ints(lens), q[:, None].contiguous())
    err = _ints([0])
    nan = torch.full((2, lens[0], H, d), float("nan"), dtype=BF, device="cuda")
    kvq.append(cache, _ints([0, 0]), nan, torch.ones_like(nan), new_lens=_ints([lens[0], 0]), err=err)
    assert err.item() == kvq.FLAG_NONFINITE
    out = kvq.decode_attn(cache, _ints(lens), q)
    assert out[0].isnan().all() and torch.equal(out[1], want[1])
    out = kvq.prefill_attn(cache, _ints(lens), q[:, None].contiguous())
    assert out[0].isnan().all() and torch.equal(out[1], pre[1])

def test_decode_and_prefill_agree_and_repeat():
    lens = [1000, 77, 129]
    cache = build(lens, 2, 128, 64, seed=5)
    q = torch.randn((3, 8, 128), generator=_gen(6), device="cuda").to(BF)
    a = kvq.decode_attn(cache, _ints(lens), q)
    b = kvq.prefill_attn(cache, _ints(lens), q[:, None].contiguous())[:, 0]
    assert (a - b).abs().max().item() <= 3e-3 * 20
    for _ in range(5):  # no order of atomics or of CTAs shows
        assert torch.equal(kvq.decode_attn(cache, _ints(lens), q), a)
        assert torch.equal(kvq.prefill_attn(cache, _ints(lens), q[:, None].contiguous())[:, 0], b)


def test_python_and_workspace_refusals():
    cache = build([64, 64], 2, 64, 32, seed=2)
    q = torch.zeros((2, 4, 64), dtype=BF, device="cuda")
    lens = _ints([64, 64])
    ring = kvq.Fp8WindowCache(2, 2, 64, 16)
    for kw in (dict(swa=ring), dict(kernel="tcgen05"), dict(out=torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda")),
               dict(out=torch.zeros((1, 4, 64), device="cuda")), dict(err=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            kvq.decode_attn(cache, lens, q, **kw)
    for a in ((lens, q.float()), (lens.long(), q), (_ints([64]), q), (lens, q[..., :32].contiguous()), (lens, q[:, None])):
        with pytest.raises(ValueError):
            kvq.decode_attn(cache, *a)
        with pytest.raises(ValueError):
            kvq.prefill_attn(cache, a[0], a[1] if a[1].dim() == 3 else a[1][:, 0])
    small = torch.zeros(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(kvq.KvqError) as e:
        kvq.decode_attn(cache, lens, q, workspace=small)
    assert e.value.status == 3
    with pytest.raises(kvq.KvqError) as e:
        kvq.prefill_attn(cache, lens, q[:, None].contiguous(), workspace=small)
    assert e.value.status == 3
    fp4 = kvq.Fp4Cache(2, 64, 32, 4, 2)
    with pytest.raises(ValueError):
        kvq.prefill_attn(fp4, lens, q[:, None].contiguous(), chunk_lens=lens)
    with pytest.raises(kvq.KvqError) as e:
        kvq.decode_attn(cache, lens, torch.zeros((2, 18, 64), dtype=BF, device="cuda"))
    assert e.value.status == 2


def test_pool_offsets_past_32_bits_and_far_positions():
    """Pages at the far end of a pool of more than 2^32 bytes, and a sequence of
    131,079 positions."""
    d, H, G, page, mp, pages = 128, 2, 8, 256, 520, 33000  # 33000 x 2 x 4 x 16416 bytes = 4.33 GB
    table = torch.randint(32900, pages, (1, mp), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    cache = kvq.Fp8BlockCache(H, d, page, pages, mp, page_table=table)
    for pg in range(32900, pages):  # each page filled through a table of its own
        k = torch.randn((1, page, H, d), generator=_gen(pg), device="cuda").to(BF)
        one = torch.full((1, mp), pg, dtype=torch.int32, device="cuda")
        kvq.append(cache, _ints([0]), k, (k.float() * 0.5 + 1.0).to(BF), page_table=one)
    T = 131079
    q = torch.randn((1, 3, H * G, d), generator=_gen(5), device="cuda").to(BF)
    err = _ints([0])
    dec = kvq.decode_attn(cache, _ints([T]), q[:, 2].contiguous(), err=err)
    pre = kvq.prefill_attn(cache, _ints([T]), q, err=err)
    assert err.item() == 0
    check(dec[:, None], q[:, 2:], cache, [T], [1], 1 / math.sqrt(d), False)
    check(pre, q, cache, [T], [3], 1 / math.sqrt(d), True)


def test_a_large_batch_of_single_tokens():
    """3000 sequences (24,000 units), lengths 0 to 3."""
    B, H, G, d = 3000, 8, 1, 64
    lens = torch.randint(0, 4, (B,), generator=torch.Generator().manual_seed(2)).tolist()
    cache = build(lens, H, d, 16, seed=3)
    q = torch.randn((B, 1, H * G, d), generator=_gen(4), device="cuda").to(BF)
    dec = kvq.decode_attn(cache, _ints(lens), q[:, 0].contiguous())
    K, V = kvq.dequant(cache, _ints(lens), 4)
    s = torch.einsum("bhd,bthd->bht", q[:, 0].double(), K.double()) / math.sqrt(d)
    s = s.masked_fill(torch.arange(4, device="cuda") >= _ints(lens)[:, None, None], -math.inf)
    want = torch.einsum("bht,bthd->bhd", torch.softmax(s, -1).nan_to_num(0.0), V.double())
    vmax = V.abs().amax((1, 3))[..., None].double()
    a = (q[:, 0].double().abs()[:, None] * K.double().abs()).sum(-1).max().item() / math.sqrt(d) * math.log2(math.e)
    tol = ref.tolerance(d, 4, 1.0, a) * vmax
    assert ((dec.double() - want).abs() <= tol).all()
    n = torch.tensor([min(1, x) for x in lens], dtype=torch.int32, device="cuda")
    pre = kvq.prefill_attn(cache, _ints(lens), q, chunk_lens=n)
    bq = (q[:, 0].double().abs().amax(-1)[:, None] * K.double().abs().sum(-1)).max().item() / math.sqrt(d) * math.log2(math.e)
    assert ((pre[:, 0].double() - want).abs() <= ref.tolerance(d, 4, 1.0, a, bq) * vmax).all()


def test_an_explicit_stream():
    """Work on a stream given to the call, buffers made by it included, while the
    current stream is busy with other memory."""
    lens = [900, 77]
    cache = build(lens, 2, 128, 64, seed=6)
    q = torch.randn((2, 30, 8, 128), generator=_gen(7), device="cuda").to(BF)
    want, dwant = kvq.prefill_attn(cache, _ints(lens), q), kvq.decode_attn(cache, _ints(lens), q[:, 3].contiguous())
    n, q3 = _ints(lens), q[:, 3].contiguous()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        noise = torch.randn((1 << 22,), device="cuda")
        del noise  # its memory is free for the current stream while the kernel that fills it runs
        out = kvq.prefill_attn(cache, n, q, stream=side)
        dec = kvq.decode_attn(cache, n, q3, stream=side)
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(dec, dwant)


def test_lengths_far_past_the_pages_end_soon():
    """A length of 2^31 - 1 reads what the pages hold, flags the rest and returns
    at once, in every form of the kernels."""
    for mp, page, B in ((2, 16, 1), (40, 64, 2), (600, 16, 1), (300, 16, 40)):
        cap = mp * page
        cache = build([cap] * B, 2, 128, page, seed=mp)
        q = torch.randn((B, 8, 128), generator=_gen(3), device="cuda").to(BF)
        want = kvq.decode_attn(cache, _ints([cap] * B), q)
        far, err = _ints([2 ** 31 - 1] * B), _ints([0])
        out = kvq.decode_attn(cache, far, q, err=err)
        assert err.item() == kvq.FLAG_PAGE_OOB and torch.equal(out, want)
        err = _ints([0])
        pre = kvq.prefill_attn(cache, far, q[:, None].contiguous(), err=err)
        assert err.item() == kvq.FLAG_PAGE_OOB
        check(pre, q[:, None], cache, [cap] * B, [1] * B, 1 / math.sqrt(128), True)
