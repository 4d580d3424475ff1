"""Values of extreme scales in the 8-bit block cache's attention, against float64
with each row's own bound (tests/attn_bounds.py)."""
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


def scales(cache):
    """The scales' view [pages][heads][groups][G / 16][2] of the pool."""
    g, d = cache.group, cache.head_dim
    s = cache.pool[..., 2 * g * d:2 * g * d + max(16, g // 2)].view(torch.float32)
    return s.view(*s.shape[:-1], -1, 2)[..., :g // 16, :]


def filled(T, H, d, page, seed=0):
    """A contiguous cache of one sequence of T random tokens."""
    mp = -(-T // page)
    cache = kvq.Fp8BlockCache(H, d, page, mp, mp)
    k, v = (torch.randn((1, T, H, d), generator=_gen(seed + i), device="cuda").to(BF) for i in range(2))
    kvq.append(cache, _ints([0]), k, v)
    return cache


def value_scales(cache, T):
    """[T][H] of a contiguous cache of one sequence."""
    s = scales(cache)[..., 1]                              # [pages][H][groups][G/16]
    return s.permute(0, 2, 3, 1).reshape(-1, s.shape[1]).repeat_interleave(16, 0)[:T]


def check(cache, T, q, out, last, v_rel=0.0, floor=0.0, prefill=True):
    """out, q [n][Hq][d]: within the bound of the row, or `floor`."""
    n, hq, d = q.shape
    g, scale = hq // cache.num_kv_heads, 1.0 / math.sqrt(d)
    K, V = kvq.dequant(cache, _ints([T]), T)
    vs = value_scales(cache, T)
    for h in range(cache.num_kv_heads):
        rows = slice(h * g, (h + 1) * g)
        want, p = attn_bounds.attend(q[:, rows], K[0, :, h], V[0, :, h], scale, last)
        tol = attn_bounds.bound(q[:, rows], K[0, :, h], V[0, :, h], p, scale, vs[:, h] if prefill else None,
                                out.dtype, want, v_rel) + floor
        off = (out[:, rows].double() - want).abs()
        assert (off <= tol).all(), (h, (off / tol).nan_to_num(math.inf).max().item())


@pytest.mark.parametrize("d,n", [(64, 5), (128, 5), (128, 150)])
@pytest.mark.parametrize("exponent", [-126, -128, -130, -140])
def test_tiny_value_scales(d, n, exponent):
    """The readers take any finite scale: all values of a cache next to and among
    fp32's subnormals."""
    T, H = 300, 2
    cache = filled(T, H, d, 64, seed=1)
    scales(cache)[..., 1] = 2.0 ** exponent
    q = torch.randn((1, n, 4 * H, d), generator=_gen(3), device="cuda").to(BF)
    out = kvq.prefill_attn(cache, _ints([T]), q)
    # half steps of fp32's subnormals: of a value, of each of the T / 16 sums, of a join and the result
    floor = (T / 16 + 3) * 2.0 ** -150
    check(cache, T, q[0], out[0], torch.arange(T - n, T), floor=floor)
    dec = kvq.decode_attn(cache, _ints([T]), q[:, -1].contiguous())
    check(cache, T, q[0, -1:], dec, torch.tensor([T - 1]), floor=floor, prefill=False)


@pytest.mark.parametrize("d,page,T,n", [(128, 64, 300, 5), (64, 16, 129, 40), (128, 32, 1000, 150), (64, 64, 700, 300)])
@pytest.mark.parametrize("larger", [2.0 ** 30, 2.0 ** 100])
def test_larger_values_later_in_a_chunk(d, page, T, n, larger):
    """The values of the chunk's last token, far above all others, leave the rows
    before it as they are; the last row is theirs.  (The 15 tokens that share its
    block of 16 are held at its scale: what the cache holds of them is what counts.)"""
    H, G = 2, 4
    cache = filled(T, H, d, page, seed=5)
    k, v = (torch.randn((1, 1, H, d), generator=_gen(8 + i), device="cuda") for i in range(2))
    kvq.append(cache, _ints([T - 1]), k.to(BF), (v * larger).to(BF))
    q = torch.randn((1, n, H * G, d), generator=_gen(7), device="cuda").to(BF)
    last = torch.arange(T - n, T)
    out = kvq.prefill_attn(cache, _ints([T]), q)
    check(cache, T, q[0], out[0], last)
    for i in (0, n - 2, n - 1):  # one row at its own length
        dec = kvq.decode_attn(cache, _ints([T - n + i + 1]), q[:, i].contiguous())
        check(cache, T, q[0, i:i + 1], dec, last[i:i + 1], prefill=False)


@pytest.mark.parametrize("d,n", [(64, 3), (128, 70), (128, 200)])
def test_values_of_every_scale(d, n):
    """Blocks from 2^-120 to 2^110, each row's weight on a block of its own, the
    blocks in falling and in rising order of their values."""
    T, H = 640, 1
    blocks = T // 16
    for order in (1, -1):
        cache = filled(T, H, d, 64, seed=11)
        at = torch.linspace(-120, 110, blocks, device="cuda").round()[::1]
        e = at if order == 1 else at.flip(0)
        s = scales(cache)[..., 1]                              # [pages][1][1][4]
        s.copy_(torch.ldexp(torch.ones(blocks, device="cuda"), e.int()).view(s.shape))
        # keys: block i answers channel i alone
        k = torch.zeros((1, T, H, d), device="cuda")
        k[0, torch.arange(T), 0, (torch.arange(T) // 16) % d] = 1.0
        codes = cache.pool.clone()
        kvq.append(cache, _ints([0]), k.to(BF), torch.zeros_like(k).to(BF))
        g = cache.group
        cache.pool[..., g * d:2 * g * d] = codes[..., g * d:2 * g * d]
        scales(cache)[..., 1].copy_(torch.ldexp(torch.ones(blocks, device="cuda"), e.int()).view(s.shape))
        q = torch.zeros((1, n, blocks, d), device="cuda")      # head i looks at block i
        q[..., torch.arange(blocks), torch.arange(blocks) % d] = 60.0 * math.sqrt(d)
        H8 = blocks // 8                                       # (eight query heads a call)
        for h in range(H8):
            x = q[:, :, 8 * h:8 * h + 8].to(BF).contiguous()
            out = kvq.prefill_attn(cache, _ints([T]), x)
            assert torch.isfinite(out).all()
            check(cache, T, x[0], out[0], torch.arange(T - n, T))


@pytest.mark.parametrize("d,page,T,n", [(128, 64, 300, 5), (64, 16, 135, 40), (128, 32, 1000, 150), (64, 64, 700, 300),
                                        (128, 64, 20, 7)])
@pytest.mark.parametrize("larger", [2.0 ** 12, 2.0 ** 16, 2.0 ** 30, 2.0 ** 100])
@pytest.mark.parametrize("behind", [0, 3])
def test_a_larger_value_in_the_same_block(d, page, T, n, larger, behind):
    """A row that sees a part of a block whose scale a later token has set: the block
    is what the cache holds of it (its codes may all be 0 there), the row's other
    blocks count as ever.  behind: tokens of the chunk after the large one."""
    H, G = 2, 4
    cache = filled(T, H, d, page, seed=5)
    at = T - 1 - behind
    k, v = (torch.randn((1, 1 + behind, H, d), generator=_gen(8 + i), device="cuda") for i in range(2))
    v[:, 0] *= larger
    kvq.append(cache, _ints([at]), k.to(BF), v.to(BF))
    q = torch.randn((1, n, H * G, d), generator=_gen(7), device="cuda").to(BF)
    last = torch.arange(T - n, T)
    out = kvq.prefill_attn(cache, _ints([T]), q)
    K, V = kvq.dequant(cache, _ints([T]), T)
    t = torch.arange(T)
    part = ((t // 16)[None] == (last // 16)[:, None]) & ((last + 1) % 16 != 0)[:, None]   # the row's own block, in part
    for h in range(H):
        rows = slice(h * G, (h + 1) * G)
        x, vmax = q[0, :, rows], V[0, :, h].abs().amax(-1).double()
        own = vmax / 2.0 ** 5                                  # a token's own exponent: at most this, and over half of it
        block = value_scales(cache, T)[:, h].double()
        vs, least = torch.where(part.cuda(), own, torch.maximum(block, own)), torch.minimum(block, own / 2)
        want, p = attn_bounds.attend(x, K[0, :, h], V[0, :, h], 1 / math.sqrt(d), last)
        for i in range(n):
            tol = attn_bounds.bound(x[i:i + 1], K[0, :, h], V[0, :, h], p[i:i + 1], 1 / math.sqrt(d), vs[i], v_least=least)
            off = (out[0, i:i + 1, rows].double() - want[i:i + 1]).abs()
            assert (off <= tol).all(), (h, i, (off / tol).max().item())
            dec_tol = attn_bounds.bound(x[i:i + 1], K[0, :, h], V[0, :, h], p[i:i + 1], 1 / math.sqrt(d))
            if T - n + i < at:  # and within eight times what a decode of the row may be off
                assert (off <= 8 * dec_tol).all(), (h, i, (off / dec_tol).max().item())


@pytest.mark.parametrize("d,page,T,n,at", [
    (128, 64, 300, 5, 297), (64, 16, 135, 40, 120), (128, 32, 1000, 150, 900), (64, 64, 700, 300, 500),
    (128, 64, 20, 7, 16), (128, 256, 2600, 128, 2495), (64, 32, 900, 33, 100), (128, 64, 300, 200, 299)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_nan_values_reach_the_rows_that_see_them(d, page, T, n, at, dtype):
    """A NaN value of one token and channel: NaN in that channel for the rows from the
    token on, no change for those before it."""
    H, G, ch = 2, 4, d // 2 + 3
    cache = filled(T, H, d, page, seed=5)
    m = 16 - at % 16 if at + 16 <= T else 1                 # and the rest of its block again, so that it is as appended
    k, v = (torch.randn((1, min(m, T - at), H, d), generator=_gen(8 + i), device="cuda") for i in range(2))
    v[0, 0, 1, ch] = float("nan")
    err = _ints([0])
    kvq.append(cache, _ints([at]), k.to(BF), v.to(BF), err=err)
    assert err.item() == kvq.FLAG_NONFINITE
    q = torch.randn((1, n, H * G, d), generator=_gen(7), device="cuda").to(BF)
    out = torch.empty(q.shape, dtype=dtype, device="cuda")
    kvq.prefill_attn(cache, _ints([T]), q, out=out)
    last = torch.arange(T - n, T)
    sees = (last >= at).cuda()
    nan = out[0].isnan()
    want = torch.zeros_like(nan)
    want[sees, G:, ch] = True
    assert torch.equal(nan, want)
    # the rows before it, and the other kv head's, within their bounds
    K, V = kvq.dequant(cache, _ints([T]), T)
    V = V.nan_to_num(0.0)
    for h in range(H):
        rows = slice(h * G, (h + 1) * G)
        own = V[0, :, h].abs().amax(-1).double() / 2 ** 5      # a token's own exponent, as above
        block = value_scales(cache, T)[:, h].double()
        most = torch.maximum(block, own)
        most[at // 16 * 16:at // 16 * 16 + 16] = own[at // 16 * 16:at // 16 * 16 + 16]
        for i in range(n):
            if h == 1 and sees[i]:
                continue
            ref, p = attn_bounds.attend(q[0, i:i + 1, rows], K[0, :, h], V[0, :, h], 1 / math.sqrt(d), last[i:i + 1])
            tol = attn_bounds.bound(q[0, i:i + 1, rows], K[0, :, h], V[0, :, h], p, 1 / math.sqrt(d), most, dtype, ref,
                                    v_least=torch.minimum(block, own / 2))
            off = (out[0, i:i + 1, rows].double() - ref).abs()
            assert (off <= tol).all(), (h, i, (off / tol).max().item())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("small", [2.0 ** -10, 2.0 ** -14, 2.0 ** -33])
def test_small_query_elements(d, small):
    """Elements next to the last bit that a query keeps beside its row's largest, 1
    (which meets zeros): scores of +-1 and +-4 come from them alone, so what they lose
    shows.  small (1 + 2^-7) is off by 2^-17 of the largest in the prefill."""
    T, H, G, n = 40, 1, 4, 6
    cache = kvq.Fp8BlockCache(H, d, 64, 1, 1)
    k = torch.zeros((1, T, H, d), device="cuda")
    k[..., 5] = (torch.arange(T, device="cuda") % 2 * 2.0 - 1.0)[:, None] * math.sqrt(d) / small
    v = torch.randn((1, T, H, d), generator=_gen(4), device="cuda")
    kvq.append(cache, _ints([0]), k.to(BF), v.to(BF))
    q = torch.zeros((1, n, H * G, d), device="cuda")
    q[..., 0] = 1.0
    q[..., 5] = small * torch.tensor([1 + 2.0 ** -7, 1 - 2.0 ** -8, 4 + 2.0 ** -5, -1 - 2.0 ** -6], device="cuda")
    q = q.to(BF)
    last = torch.arange(T - n, T)
    out = kvq.prefill_attn(cache, _ints([T]), q)
    check(cache, T, q[0], out[0], last)
    dec = kvq.decode_attn(cache, _ints([T]), q[:, -1].contiguous())
    check(cache, T, q[0, -1:], dec, last[-1:], prefill=False)


@pytest.mark.parametrize("d,T,n", [(128, 2569, 10), (64, 1290, 12), (128, 3 * 128 + 9, 10), (64, 5 * 128 + 40, 40)])
def test_token_exponents_repeat(d, T, n):
    """A pair whose half meets a tile with exponents of single tokens as its second or a
    later one, in many CTAs at once: every call gives the first one's bits."""
    B, H, G, page = 5, 3, 3, 64
    mp = -(-T // page)
    cache = kvq.Fp8BlockCache(H, d, page, B * mp, mp)
    k, v = (torch.randn((B, T, H, d), generator=_gen(20 + i), device="cuda") for i in range(2))
    v *= torch.exp2(25 * torch.randn((B, -(-T // 16), H, 1), generator=_gen(22), device="cuda")).repeat_interleave(16, 1)[:, :T]
    v = v.clamp(-1e30, 1e30)
    kvq.append(cache, _ints([0] * B), k.to(BF), v.to(BF))
    q = torch.randn((B, n, H * G, d), generator=_gen(23), device="cuda").to(BF)
    lens = _ints([T - 3 * b for b in range(B)])
    first = kvq.prefill_attn(cache, lens, q)
    noise = torch.empty(1 << 26, device="cuda")
    for i in range(200):
        if i % 2:
            noise.fill_(float(i))  # the caches out of L2, so that copies come late
        assert torch.equal(kvq.prefill_attn(cache, lens, q), first)
    K, V = kvq.dequant(cache, lens, T)
    for b in range(B):
        L = T - 3 * b
        for i in (0, n - 1):
            want, p = attn_bounds.attend(q[b, i:i + 1, :G], K[b, :L, 0], V[b, :L, 0], 1 / math.sqrt(d), torch.tensor([L - n + i]))
            off = (first[b, i, :G].double() - want[0]).norm(dim=-1) / want[0].norm(dim=-1)
            assert (off < 0.02).all()
