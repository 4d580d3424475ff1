"""Absorbed latent attention at scores whose fp32 steps are large beside the exponents that stand
next to them: one token outweighs all others by far more than any rounding, so the row is that
token's latent, whatever the score's size.

Bound: the weight's own rounding, 2^-8 + 2^-11 (its factors cancel: the same score stands in the
sum and in the sum of weights), and 2^-20 for exponentials, division and joins."""
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


def fill(T, picked, exps, seed):
    """Key channel i of token picked[i] holds 256, of the other picked ones 0, of the rest at most 64
    (times the scales 2^exps[t])."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randn((1, T, L), generator=g, device="cuda").clamp(-3.5, 3.5) * 64
    c[..., 0] = 256.0
    k = torch.randn((1, T, R), generator=g, device="cuda").clamp(-1, 1) * 64
    k[0, picked] = 0.0
    for i, t in enumerate(picked):
        k[0, t, i] = 256.0
    s = 2.0 ** torch.tensor(exps, dtype=torch.float32, device="cuda")[None, :, None]
    cache = kvq.LatentCache(L, R, 64, -(-T // 64), -(-T // 64))
    kvq.latent_append(cache, _ints([0]), None, (c * s).to(BF), (k * s).to(BF), None)
    codes, e = ref.read_pool(cache.pool, None, cache.max_pages_per_seq, 0, T, 64, L, R)
    assert (e - 127).tolist() == list(exps)
    return cache, ref.decode(codes, e, L)[0]


def check(out, want):
    assert torch.isfinite(out).all()
    off = (out.double() - want).abs()
    assert (off <= want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20)).all(), \
        (out.double().norm(dim=-1) / want.norm(dim=-1)).tolist()


SIZES = [12, 19, 23, 24, 25, 26, 27, 28, 31, 40, 60, 90]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("T", [200, 5000])
def test_near_scales(size, T):
    """Scores of 2^size; scales 2^-3 .. 2^3 (a picked token's 2^3).  T 200: four tiles; 5000: split."""
    picked = [0, 9, 63, 64, 70, 127, 128, 190, 199, T - 1, T // 2, T // 3]
    exps = [(5 * t) % 7 - 3 for t in range(T)]
    for t in picked:
        exps[t] = 3
    cache, lat = fill(T, picked, exps, size)
    q = torch.zeros((1, len(picked), L + R), dtype=BF, device="cuda")
    for i in range(len(picked)):
        q[0, i, L + i] = 2.0 ** (size - 11)
    check(kvq.decode_attn(cache, _ints([T]), q, 1.0)[0], lat[picked])


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("high", [44, 60])
def test_far_scales(size, high):
    """Picked tokens of scales 2^44 and more among tokens of 2^-40 .. 2^3, whole units of one CTA."""
    T, n, H = 320, 77, 64
    picked = [2, 70, 130, 199, 201, 242]  # (row 0 sits at position 243)
    exps = [(5 * t) % 44 - 40 for t in range(T)]
    for i, t in enumerate(picked):
        exps[t] = high + i
    cache, lat = fill(T, picked, exps, size)
    q = torch.zeros((1, n, H, L + R), dtype=BF, device="cuda")
    want = [picked[h % len(picked)] for h in range(H)]
    for h in range(H):
        q[0, :, h, L + h % len(picked)] = 2.0 ** (size - 8 - exps[want[h]])
    out = kvq.prefill_attn(cache, _ints([T]), q, 1.0)
    check(out[0], lat[want][None].expand(n, H, L))
