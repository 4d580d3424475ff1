"""Absorbed latent attention over tokens whose scales lie further apart than 2^80: one token's
exponent far above all others', in each tile of a range, against float64.

Bound: latent_reference.attn_bound with the queries' own rounding left out (they are 0, or one
power of two, which E4M3 holds), and for scores that are taken out of the sum of score and
exponent, y = (y + e) - e: half a step of fp32 under 2^8, 2^-17, in the weight and in the sum of
weights."""
import math

import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests import latent_reference as ref
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
L, R = 128, 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fill(B, T, far, low, high, seed, cap=None):
    """A contiguous cache: sequence b's token far[b] has scale 2^high and the key part 0, all
    others 2^low."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randn((B, T, L), generator=g, device="cuda").clamp(-3.5, 3.5) * 64
    c[..., 0] = 256.0                                   # 224 < 256 <= 448: the scale is the factor
    k = torch.randn((B, T, R), generator=g, device="cuda").clamp(-3.5, 3.5) * 64
    s = torch.full((B, T, 1), 2.0 ** low, device="cuda")
    for b, t in enumerate(far):
        s[b, t], k[b, t] = 2.0 ** high, 0.0
    mp = -(-T // 64)
    cache = kvq.LatentCache(L, R, 64, B * mp, mp)
    kvq.latent_append(cache, _ints([0] * B), None, (c * s).to(BF), (k * s).to(BF), None)
    return cache


def check(out, q, cache, b, T, first, scale):
    """out, q [n][H][...] of sequence b, its row i at position first + i."""
    n, H = out.shape[:2]
    codes, e = ref.read_pool(cache.pool, None, cache.max_pages_per_seq, b, T, 64, L, R)
    assert set(e.tolist()) <= {int(e.min()), int(e.max())} and int(e.max()) - int(e.min()) > 80
    c, k = ref.decode(codes, e, L)
    s, x = ref.power(e - 127), q.reshape(-1, L + R)
    p = ref.weights(x, torch.cat([c, k], -1), scale, (first + torch.arange(n)).repeat_interleave(H))
    want = p @ c
    score = ref._scores_off(x, torch.cat([c, k], -1), p > 0, scale, False)
    prod = p * s
    top = prod.amax(-1, keepdim=True)
    tol = (p @ c.abs()) * (2.0 ** -8 + 2.0 ** -11 + (2 * math.log(2) * (score + 2.0 ** -17) + T / 16 * 2.0 ** -24 +
                                                     2.0 ** -20)[:, None])
    small = (p > 0) & (prod < 2.0 ** -9 * top)
    tol = tol + 2.0 ** -17 * top * (small.double() @ (c.abs() / s[:, None]))
    off = (out.reshape(-1, L).double() - want).abs()
    assert (off <= tol).all(), (off / tol).amax().item()


def queries(n, H, low):
    """Half the heads 0 (equal weights), half a key channel, which weighs the low tokens by it."""
    q = torch.zeros((n, H, L + R), dtype=BF, device="cuda")
    q[:, H // 2:, L + 5] = 2.0 ** (-low - 7)
    return q


@pytest.mark.parametrize("low,high", [(-40, 100), (-16, 119), (-12, 119), (-100, 0)])
@pytest.mark.parametrize("tiles", [3, 4, 9])
@pytest.mark.parametrize("tile", [0, 1, 2, -1])
def test_one_far_token_in_a_unit(low, high, tiles, tile):
    """Whole units of one CTA (more row tiles than half the SMs)."""
    n, H, T = 77, 64, 64 * tiles
    at = 64 * (tile % tiles) + 9
    cache = fill(1, T, [at], low, high, seed=tiles)
    q = queries(n, H, low)
    out = kvq.prefill_attn(cache, _ints([T]), q[None], 1.0)
    check(out[0], q, cache, 0, T, T - n, 1.0)


@pytest.mark.parametrize("low,high", [(-40, 100), (-16, 119)])
def test_one_far_token_in_split_ranges(low, high):
    """Positions shared by several CTAs, the far token in another tile of each sequence."""
    B, H, T = 24, 16, 1300
    cache = fill(B, T, [64 * (3 * b % 20) + b for b in range(B)], low, high, seed=7)
    q = queries(1, H, low).expand(B, H, L + R).contiguous()
    out = kvq.decode_attn(cache, _ints([T] * B), q, 1.0)
    for b in range(B):
        check(out[b][None], q[b][None], cache, b, T, T - 1, 1.0)


def test_several_far_tokens():
    """Scales that rise by 2^60 from tile to tile."""
    n, H, T = 77, 64, 64 * 4
    g = torch.Generator(device="cuda").manual_seed(3)
    c = torch.randn((1, T, L), generator=g, device="cuda").clamp(-3.5, 3.5) * 64
    c[..., 0] = 256.0
    s = 2.0 ** (torch.arange(T, device="cuda") // 64 * 60.0 - 100.0)[None, :, None]
    cache = kvq.LatentCache(L, R, 64, 4, 4)
    kvq.latent_append(cache, _ints([0]), None, (c * s).to(BF), torch.zeros((1, T, R), dtype=BF, device="cuda"), None)
    q = torch.zeros((1, n, H, L + R), dtype=BF, device="cuda")
    out = kvq.prefill_attn(cache, _ints([T]), q, 1.0)
    codes, e = ref.read_pool(cache.pool, None, 4, 0, T, 64, L, R)
    lat = ref.decode(codes, e, L)[0]
    for i in range(n):
        p = T - n + i + 1
        want, size = lat[:p].mean(0), lat[:p].abs().mean(0)
        # tokens 2^60 under the largest: 2^-17 of its product each, at most 448 a code
        tol = size * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16) + 2.0 ** -17 * 448 * ref.power(e[:p].max() - 127)
        assert ((out[0, i].double() - want).abs() <= tol).all(), i
