"""kvq_rope_append, kvq_fp8_block_append, kvq_rope_table and
kvq_fp8_block_dequant against the host reference: codes, scales and rotated
values bit for bit (every step of the definition is exact or one rounding, so
the tolerance is 0; against float64 the rotation is held to its roundings)."""
import ctypes

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


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tokens(g, B, n, H, d):
    x = torch.randn((B, n, H, d), generator=g) * torch.exp(torch.randn((B, n, H, 1), generator=g))
    return x.to(BF)


def _make(B, H, d, page, capacity, paged, g):
    mp = -(-capacity // page)
    table = None
    if paged:
        table = torch.randperm(B * mp, generator=g).to(torch.int32).view(B, mp).cuda()
    return kvq.Fp8BlockCache(H, d, page, B * mp, mp, page_table=table), mp


def _same(cache, mp, want, lens):
    for b, n in enumerate(lens):
        if n == 0:
            continue
        codes, scales = ref.read_pool(cache.pool, cache.page_table, mp, b, n, cache.page_size, cache.head_dim)
        assert torch.equal(codes, want.codes[:, b, :n]), b
        assert torch.equal(scales, want.scales[:, b, :-(-n // 16)]), b


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,paged", [(16, True), (32, False), (64, True), (128, True), (256, False)])
def test_block_append_sequence(d, page, paged):
    """Appends of many lengths from odd starts: blocks begun, filled, raised
    (louder tokens later) and cut; a padded batch; then back over old
    positions (a rejected draft) and a sequence begun again on used pages."""
    B, H, cap = 3, 2, 512
    g = _gen(d + page)
    cache, mp = _make(B, H, d, page, cap, paged, g)
    want = ref.BlockCache(B, H, d, cap)
    at = [0, 5, 33]
    first = _tokens(g, B, 40, H, d)
    err = _ints([0])
    for step, n in enumerate([40, 1, 1, 17, 3, 60, 1, 16]):
        lens = None if step in (0, 2) else [n, max(0, n - 1 - step), (n + 1) // 2]
        if step == 0:
            lens, starts = [at[0] + 40, at[1], at[2]], [0, 0, 0]
        else:
            starts = list(at)
        k, v = _tokens(g, B, n, H, d), _tokens(g, B, n, H, d)
        if step == 0:
            k, lens = first, [40, 5, 33]
        k = (k.float() * 2.0 ** (step - 3)).to(BF)
        v = (v.float() * 2.0 ** (3 * (step % 3) - 3)).to(BF)
        kvq.append(cache, _ints(starts), k.cuda(), v.cuda(), err=err, new_lens=None if lens is None else _ints(lens))
        want.append(starts, k, v, lens)
        at = [s + (n if lens is None else lens[i]) for i, s in enumerate(starts)]
        _same(cache, mp, want, at)
    back = [a - 9 for a in at]
    k, v = _tokens(g, B, 4, H, d), _tokens(g, B, 4, H, d)
    kvq.append(cache, _ints(back), k.cuda(), v.cuda(), err=err)
    want.append(back, k, v)
    _same(cache, mp, want, [a + 4 for a in back])
    kvq.append(cache, _ints([0] * B), (k.float() * 1e-3).to(BF).cuda(), v.cuda(), err=err)
    want.append([0] * B, (k.float() * 1e-3).to(BF), v)
    _same(cache, mp, want, [4] * B)
    assert err.item() == 0


def test_block_append_extreme_values():
    """Zeros, the smallest and largest bf16 values, the borders of a scale
    (448, 449 and 450 times a power of two), ties of the E4M3 rounding."""
    d, H = 64, 1
    g = _gen(3)
    rows = torch.randn((1, 16 * 10, H, d), generator=g)
    rows[:, :16] = 0.0
    rows[:, 16:32] = 2.0 ** -133
    rows[:, 32:48] *= 3e38 / 6
    rows[:, 48, :, 0], rows[:, 48:64, :, 1:] = 448.0, 1.0
    rows[:, 64, :, 0], rows[:, 64:80, :, 1:] = 450.0, 1.0
    rows[:, 80:96] = -0.0
    rows[:, 96:112] = torch.randint(-255, 256, (1, 16, H, d), generator=g).float() * 2.0 ** -9
    rows[:, 112:128] *= 1e-38
    rows = rows.clamp(-3.3e38, 3.3e38).to(BF)
    cache, mp = _make(1, H, d, 32, 160, False, g)
    want = ref.BlockCache(1, H, d, 160)
    err = _ints([0])
    for lo, hi in ((0, 50), (50, 75), (75, 160)):
        kvq.append(cache, _ints([lo]), rows[:, lo:hi].cuda().contiguous(), rows[:, lo:hi].cuda().contiguous(), err=err)
        want.append([lo], rows[:, lo:hi], rows[:, lo:hi])
    _same(cache, mp, want, [160])
    assert err.item() == 0
    k, v = kvq.dequant(cache, _ints([160]), 160, err=err)
    assert torch.equal(k[0].cpu().double(), want.values(0, 0, 160)) and torch.equal(v[0].cpu().double(), want.values(1, 0, 160))


@pytest.mark.parametrize("d,page", [(64, 16), (128, 256)])
def test_dequant_and_what_lies_behind_the_end(d, page):
    B, H, cap = 2, 3, 300
    g = _gen(9)
    cache, mp = _make(B, H, d, page, cap, True, g)
    cache.pool.random_(0, 256)
    before = cache.pool.clone()
    want = ref.BlockCache(B, H, d, 320)
    k, v = _tokens(g, B, 70, H, d), _tokens(g, B, 70, H, d)
    kvq.append(cache, _ints([0, 0]), k.cuda(), v.cuda(), new_lens=_ints([70, 33]))
    want.append([0, 0], k, v, [70, 33])
    kd, vd = kvq.dequant(cache, _ints([70, 33]), 80)
    assert kd.shape == (B, 80, H, d)
    for b, n in enumerate([70, 33]):
        assert torch.equal(kd[b, :n].cpu().double(), want.values(0, b, n))
        assert torch.equal(vd[b, :n].cpu().double(), want.values(1, b, n))
        assert not kd[b, n:].any() and not vd[b, n:].any()
    kb, vb = kvq.dequant(cache, _ints([70, 33]), 80, dtype=BF)
    assert torch.equal(kb, kd.to(BF)) and torch.equal(vb, vd.to(BF))
    # bytes of tokens behind the last new one are as they were
    for b, n in enumerate([70, 33]):
        m = -(-n // 16) * 16
        old, _ = ref.read_pool(before, cache.page_table, mp, b, m, page, d)
        new, _ = ref.read_pool(cache.pool, cache.page_table, mp, b, m, page, d)
        a, o = new[:, n:m], old[:, n:m]
        assert torch.equal(a.nan_to_num(1e9), o.nan_to_num(1e9))


@pytest.mark.parametrize("base,rd", [(10000.0, 128), (500000.0, 64), (10000.0, 16)])
def test_rope_table(base, rd):
    t = kvq.rope_table(70000, rd, base).cpu().double()
    pos = torch.arange(70000, dtype=torch.float64)[:, None]
    ang = pos * base ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd)
    # fp32 rounding of a value <= 1 (half a step 2^-25) and the fp64 angle's own error, far below
    assert (t[:, :rd // 2] - ang.cos()).abs().max() <= 2.0 ** -24
    assert (t[:, rd // 2:] - ang.sin()).abs().max() <= 2.0 ** -24


def test_a_table_on_an_explicit_stream():
    """Memory that was freed for the current stream while a kernel on it still
    writes there does not become the table of a call on another stream."""
    want = kvq.rope_table(40000, 128)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        busy = torch.empty((40000, 128), device="cuda")
        for _ in range(50):
            busy.fill_(7.0)
        del busy
        got = kvq.rope_table(40000, 128, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        side.synchronize()
        del got


CASES = [  # d, rotary, interleaved, heads, group, n, starts
    (128, 128, False, 2, 8, 5, [0, 77, 1000]),
    (128, 128, True, 1, 3, 17, [3, 0, 30]),
    (128, 32, False, 3, 1, 33, [16, 15, 1]),
    (128, 48, True, 2, 5, 1, [7, 8, 9]),
    (64, 64, False, 2, 4, 20, [0, 1, 2]),
    (64, 16, False, 5, 7, 3, [100, 0, 50]),
    (64, 16, True, 8, 8, 1, [500, 0, 31]),
    (64, 48, False, 1, 2, 64, [8, 24, 40]),
]


@pytest.mark.parametrize("d,rd,inter,H,G,n,starts", CASES)
@pytest.mark.parametrize("packed", [False, True])
def test_rotation_and_append_fp8(d, rd, inter, H, G, n, starts, packed):
    B, cap = len(starts), 1040
    g = _gen(rd + n)
    cache, mp = _make(B, H, d, 64, cap, True, g)
    x = _tokens(g, B, n, (G + 2) * H, d).cuda()
    if packed:
        q, k, v = x[:, :, :G * H], x[:, :, G * H:(G + 1) * H], x[:, :, (G + 1) * H:]
    else:
        q, k, v = (t.contiguous() for t in (x[:, :, :G * H], x[:, :, G * H:(G + 1) * H], x[:, :, (G + 1) * H:]))
    table = kvq.rope_table(cap, rd)
    err = _ints([0])
    k_out = torch.empty((B, n, H, d), dtype=BF, device="cuda")
    q_out = kvq.rope_append(cache, _ints(starts), q, k, v, table, interleaved=inter, k_out=k_out, err=err)
    assert err.item() == 0
    tc = table.cpu()
    want_q, want_k = (ref.rotate32(t.cpu(), starts, tc, inter) for t in (q, k))
    assert torch.equal(q_out.cpu(), want_q) and torch.equal(k_out.cpu(), want_k)
    # against float64: three fp32 roundings of the products' size, then half a bf16 step
    pos = torch.tensor(starts)[:, None] + torch.arange(n)
    cs = tc.double()[pos][:, :, None]
    a = k.cpu().double()
    i = torch.arange(rd // 2)
    p0, p1 = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
    y0 = a[..., p0] * cs[..., :rd // 2] - a[..., p1] * cs[..., rd // 2:]
    size = (a[..., p0] * cs[..., :rd // 2]).abs() + (a[..., p1] * cs[..., rd // 2:]).abs()
    tol = 2.0 ** -8 * y0.abs() + 4 * 2.0 ** -24 * size + 2.0 ** -133
    assert ((k_out.cpu().double()[..., p0] - y0).abs() <= tol).all()
    # the cache holds what the plain append writes for the rotated keys
    twin = kvq.Fp8BlockCache(H, d, 64, cache.num_pages, mp, page_table=cache.page_table)
    kvq.append(twin, _ints(starts), k_out, v.contiguous())
    assert torch.equal(twin.pool, cache.pool)
    want = ref.BlockCache(B, H, d, 1056)
    want.append(starts, want_k, v.cpu())
    for b, s in enumerate(starts):
        codes, _ = ref.read_pool(cache.pool, cache.page_table, mp, b, s + n, 64, d)
        assert torch.equal(codes[:, s:], want.codes[:, b, s:s + n])


@pytest.mark.parametrize("nvfp4", [False, True])
@pytest.mark.parametrize("d,rd,inter,page,n,starts", [
    (64, 64, False, 16, 5, [0, 3]), (128, 128, False, 64, 33, [1, 64]), (128, 32, True, 128, 1, [9, 200]),
    (256, 256, False, 256, 18, [0, 7]), (256, 64, True, 32, 2, [5, 6])])
def test_rotation_and_append_fp4(nvfp4, d, rd, inter, page, n, starts):
    """Into the FP4 and NVFP4 caches: the bytes kvq_append writes for keys
    rotated beforehand, a padded batch and Inf/NaN inputs included."""
    B, H, hq, cap = 2, 2, 4, 300
    g = _gen(d + n + page)
    mp = -(-cap // page)
    table_pages = torch.randperm(B * mp, generator=g).to(torch.int32).view(B, mp).cuda()
    mk = lambda: kvq.Fp4Cache(H, d, page, B * mp, mp, page_table=table_pages, nvfp4=nvfp4)  # noqa: E731
    a, b = mk(), mk()
    x = _tokens(g, B, n, hq + 2 * H, d).cuda()
    if n > 4:
        x[0, 2, hq, 3] = float("inf")
        x[1, 1, hq + H, 5] = float("nan")
    q, k, v = x[:, :, :hq], x[:, :, hq:hq + H], x[:, :, hq + H:]
    if nvfp4:
        for c in (a, b):
            c.k_gscale.copy_(torch.tensor([3e-4, 2e-3]))
            c.v_gscale.copy_(torch.tensor([1e-3, 5e-4]))
    lens = [n, max(0, n - 3)]
    table = kvq.rope_table(cap, rd)
    ea, eb = _ints([0]), _ints([0])
    k_out = torch.zeros((B, n, H, d), dtype=BF, device="cuda")
    kvq.rope_append(a, _ints(starts), q, k, v, table, interleaved=inter, new_lens=_ints(lens), k_out=k_out, err=ea)
    for i, m in enumerate(lens):
        if m:
            kvq.append(b, _ints(starts[i:i + 1]), k_out[i:i + 1, :m].contiguous(), v[i:i + 1, :m].contiguous(), err=eb,
                       page_table=table_pages[i:i + 1].contiguous())
    assert torch.equal(a.pool, b.pool) and ea.item() == eb.item()
    assert (ea.item() == kvq.FLAG_NONFINITE) == (n > 4)
    fin = torch.isfinite(k.float()).all(-1)
    want = ref.rotate32(k.cpu(), starts, table.cpu(), inter)
    for i, m in enumerate(lens):
        ok = fin[i, :m].cpu()
        assert torch.equal(k_out[i, :m].cpu()[ok], want[i, :m][ok])
        assert not k_out[i, m:].any()


def test_in_place_no_queries_no_rotation_and_padding():
    d, H, hq, B, n = 128, 2, 6, 3, 21
    g = _gen(11)
    q, k, v = _tokens(g, B, n, hq, d).cuda(), _tokens(g, B, n, H, d).cuda(), _tokens(g, B, n, H, d).cuda()
    table = kvq.rope_table(200, d)
    lens, starts = [21, 0, 10], [4, 90, 0]
    cache, mp = _make(B, H, d, 16, 128, True, g)
    sentinel = torch.full_like(q, 7.0)
    out = kvq.rope_append(cache, _ints(starts), q, k, v, table, new_lens=_ints(lens), q_out=sentinel)
    assert out is sentinel
    for b, m in enumerate(lens):
        assert (out[b, m:] == 7.0).all()
    q2, k2 = q.clone(), k.clone()
    twin, _ = _make(B, H, d, 16, 128, True, _gen(11))
    twin.page_table = cache.page_table
    kvq.rope_append(twin, _ints(starts), q2, k2, v, table, new_lens=_ints(lens), q_out=q2, k_out=k2)
    assert torch.equal(twin.pool, cache.pool)
    for b, m in enumerate(lens):
        assert torch.equal(q2[b, :m], out[b, :m]) and torch.equal(q2[b, m:], q[b, m:]) and torch.equal(k2[b, m:], k[b, m:])
    # without queries, and without a table (the plain append)
    one, _ = _make(B, H, d, 16, 128, True, _gen(11))
    one.page_table = cache.page_table
    assert kvq.rope_append(one, _ints(starts), None, k, v, table, new_lens=_ints(lens)) is None
    assert torch.equal(one.pool, cache.pool)
    a, _ = _make(B, H, d, 16, 128, True, _gen(11))
    b_, _ = _make(B, H, d, 16, 128, True, _gen(11))
    qa = kvq.rope_append(a, _ints(starts), q, k, v, None, new_lens=_ints(lens))
    kvq.append(b_, _ints(starts), k, v, new_lens=_ints(lens))
    assert torch.equal(a.pool, b_.pool) and torch.equal(qa[0], q[0])


def test_flags():
    d, H, B, n = 64, 2, 4, 5
    g = _gen(12)
    q, k, v = _tokens(g, B, n, 4, d).cuda(), _tokens(g, B, n, H, d).cuda(), _tokens(g, B, n, H, d).cuda()

    def call(starts, lens=None, rows=64, kk=k, vv=v, pages=None):
        cache, mp = _make(B, H, d, 16, 64, True, _gen(12))
        if pages:
            cache.page_table[pages[0], pages[1]] = pages[2]
        err = _ints([0])
        qo = torch.full_like(q, 7.0)
        kvq.rope_append(cache, _ints(starts), q, kk, vv, kvq.rope_table(rows, d),
                        new_lens=None if lens is None else _ints(lens), q_out=qo, err=err)
        return err.item(), cache, qo

    flag, cache, qo = call([0, -1, 3, 10])
    assert flag == kvq.FLAG_BAD_LENGTH and (qo[1] == 7.0).all() and not (qo[0] == 7.0).all()
    assert not cache.pool[cache.page_table[1].long()].any()
    for bad in (-2, 6):
        flag, cache, qo = call([0, 1, 3, 10], [5, bad, 5, 5])
        assert flag == kvq.FLAG_BAD_LENGTH and (qo[1] == 7.0).all()
    flag, cache, qo = call([0, 60, 3, 10], rows=62)   # positions 62, 63, 64 have no row
    assert flag == kvq.FLAG_POSITION and (qo[1, 2:] == 7.0).all() and not (qo[1, 1] == 7.0).all()
    assert call([0, 60, 3, 10], [5, 2, 5, 5], rows=62)[0] == 0
    flag, cache, qo = call([0, 62, 3, 10], rows=80)   # positions 64.. have no page
    assert flag == kvq.FLAG_PAGE_OOB and not (qo[1, 4] == 7.0).all()
    for page in (-1, 1 << 20):
        flag, cache, _ = call([0, 14, 3, 10], pages=(1, 1, page))
        assert flag == kvq.FLAG_PAGE_OOB
        codes, _ = ref.read_pool(cache.pool, cache.page_table, 4, 1, 16, 16, d)
        assert codes[:, 14:].any()                    # the tokens before it are written
    kk = k.clone()
    kk[2, 1, 0, 3] = float("nan")
    flag, cache, _ = call([0, 1, 3, 10], kk=kk)
    assert flag == kvq.FLAG_NONFINITE
    vv = v.clone()
    vv[2, 1, 0, 3] = float("-inf")
    assert call([0, 1, 3, 10], vv=vv)[0] == kvq.FLAG_NONFINITE
    # a block behind a non-finite one is not touched by it, and a page used again forgets it
    cache, mp = _make(1, H, d, 16, 64, False, g)
    kvq.append(cache, _ints([0]), kk[2:3], v[2:3])
    kvq.append(cache, _ints([0]), k[2:3], v[2:3])
    want = ref.BlockCache(1, H, d, 64)
    want.append([0], k[2:3].cpu(), v[2:3].cpu())
    _same(cache, mp, want, [5])


def test_python_refusals():
    d, H, B, n = 64, 2, 2, 3
    g = _gen(13)
    cache, _ = _make(B, H, d, 16, 64, True, g)
    q, k, v = _tokens(g, B, n, 4, d).cuda(), _tokens(g, B, n, H, d).cuda(), _tokens(g, B, n, H, d).cuda()
    t, s = kvq.rope_table(64, d), _ints([0, 0])
    bad = [dict(q=q.float()), dict(k=k[:, :, :1]), dict(v=v[:, :2]), dict(q=q[:1]), dict(s=_ints([0])), dict(t=t.double()),
           dict(s=s.long()), dict(q=q.transpose(1, 2)), dict(q=q[..., ::2]), dict(q_out=q[:, :2].contiguous()),
           dict(new_lens=_ints([1])), dict(err=torch.zeros(1, device="cuda")), dict(k_out=q), dict(k=k.cpu())]
    for kw in bad:
        a = dict(s=s, q=q, k=k, v=v, t=t)
        a.update({x: kw[x] for x in kw if x in a})
        rest = {x: kw[x] for x in kw if x not in a}
        with pytest.raises(ValueError):
            kvq.rope_append(cache, a["s"], a["q"], a["k"], a["v"], a["t"], **rest)
    with pytest.raises(kvq.KvqError):
        kvq.rope_append(cache, s, q, k, v, kvq.rope_table(64, 40))
    with pytest.raises(ValueError):
        kvq.rope_append(kvq.Fp8WindowCache(2, H, d, 16), s, q, k, v, t)
    with pytest.raises(ValueError):
        kvq.append(kvq.Fp4Cache(H, d, 16, 8, 4), s, k, v, new_lens=s)
    with pytest.raises(ValueError):
        kvq.Fp8BlockCache(H, d, 16, 4, 2, pool=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        kvq.Fp8BlockCache(H, 256, 16, 4, 2)


def test_far_positions_and_wide_offsets():
    """A pool of more than 2^31 bytes: pages whose byte offsets pass 32 bits,
    positions past 100,000 (the table's rows too)."""
    d, H, page = 128, 8, 256
    mp = 520
    pages = 4300                                       # 4300 x 8 x 4 x 16416 bytes = 2.26 GB
    cache = kvq.Fp8BlockCache(H, d, page, pages, mp, page_table=torch.zeros((2, mp), dtype=torch.int32, device="cuda"))
    pos = 131070
    cache.page_table[0, pos // page], cache.page_table[0, pos // page + 1] = 4299, 4298
    g = _gen(14)
    n = 9
    q, k, v = (_tokens(g, 1, n, h, d).cuda() for h in (8, H, H))
    table = kvq.rope_table(pos + n, d)
    err = _ints([0])
    k_out = torch.empty_like(k)
    kvq.rope_append(cache, _ints([pos]), q, k, v, table, k_out=k_out, err=err)
    assert err.item() == 0
    assert torch.equal(k_out.cpu(), ref.rotate32(k.cpu(), [pos], table.cpu(), False))
    want = ref.BlockCache(1, H, d, 131328)
    want.append([pos], k_out.cpu(), v.cpu())
    lo = pos // page * page
    small = kvq.Fp8BlockCache(H, d, page, 2, 2, pool=cache.pool[[4299, 4298]].contiguous())
    codes, _ = ref.read_pool(small.pool, None, 2, 0, pos + n - lo, page, d)
    assert torch.equal(codes[:, pos - lo:], want.codes[:, 0, pos:pos + n])


def test_c_entry_with_padded_strides():
    """The C entry takes any token stride that is a multiple of 8."""
    d, H, hq, B, n = 64, 2, 3, 2, 4
    g = _gen(15)
    wide = torch.zeros((B * n, 640), dtype=BF)
    wide[:, :hq * d] = torch.randn((B * n, hq * d), generator=g).to(BF)
    wide[:, 200:200 + H * d] = torch.randn((B * n, H * d), generator=g).to(BF)
    wide[:, 400:400 + H * d] = torch.randn((B * n, H * d), generator=g).to(BF)
    w = wide.cuda()
    cache, mp = _make(B, H, d, 32, 64, False, g)
    table = kvq.rope_table(64, d)
    q_out = torch.empty((B, n, hq, d), dtype=BF, device="cuda")
    s = cache.struct()
    starts = _ints([0, 9])
    st = kvq.load().kvq_rope_append(ctypes.byref(s), B, n, starts.data_ptr(), None, hq, w.data_ptr(), 640,
                                    w.data_ptr() + 400, 640, w.data_ptr() + 800, 640, table.data_ptr(), 64, d, 0,
                                    q_out.data_ptr(), None, None, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    parts = [wide[:, o:o + h * d].reshape(B, n, h, d).cuda() for o, h in ((0, hq), (200, H), (400, H))]
    twin, _ = _make(B, H, d, 32, 64, False, g)
    q2 = kvq.rope_append(twin, starts, *parts, table)
    assert torch.equal(q_out, q2) and torch.equal(twin.pool, cache.pool)
