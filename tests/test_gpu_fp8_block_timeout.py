"""The bounded waits of the 8-bit block cache's attention, exercised without a fault
or a hang: kvq_test_set_wait_limit_ns shortens them, from 1 ns (every wait that is not
met at its first look gives up) to limits that end somewhere inside the kernel.  Each
call returns; it raises KVQ_FLAG_TIMEOUT or gives the normal result bit for bit, and
the calls after it give the normal result."""
import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LIMITS_NS = (1, 500, 1000, 2000, 3000, 5000, 8000, 12000, 20000, 40000)


@pytest.fixture(scope="module")
def lib():
    return ensure_built()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(B, T, H, d, rising=False, uneven=False):
    mp = -(-T // 64)
    cache = kvq.Fp8BlockCache(H, d, 64, B * mp, mp)
    g = torch.Generator(device="cuda").manual_seed(T + d)
    k, v = (torch.randn((B, T, H, d), generator=g, device="cuda") for _ in range(2))
    if rising:    # the running maximum is raised in every tile
        k = k * 0.1
        k[..., 0] = torch.arange(T, device="cuda")[None, :, None] * 0.5
    if uneven:    # the last token's values set the scale of their block
        v[:, -1] *= 2.0 ** 40
    kvq.append(cache, _ints([0] * B), k.to(BF), v.to(BF))
    return cache


def _check(lib, call):
    err = _ints([0])
    ref = call(err)
    torch.cuda.synchronize()
    assert err.item() == 0
    flags = []
    for ns in LIMITS_NS:
        for _ in range(3):
            try:
                lib.kvq_test_set_wait_limit_ns(ns)
                err = _ints([0])
                out = call(err)
                torch.cuda.synchronize()  # the call returned
            finally:
                lib.kvq_test_set_wait_limit_ns(0)
            flags.append(err.item())
            assert err.item() == kvq.FLAG_TIMEOUT or (err.item() == 0 and torch.equal(out, ref))
            err = _ints([0])
            again = call(err)
            assert err.item() == 0 and torch.equal(again, ref)
    assert kvq.FLAG_TIMEOUT in flags


@pytest.mark.parametrize("B,T,H,G,d", [(8, 16384, 8, 8, 128), (4, 8192, 4, 4, 64), (40, 2000, 8, 8, 128), (80, 2000, 8, 3, 64)])
def test_decode(lib, B, T, H, G, d):
    """Ranges of many chunks, whose producers wait for free stages, and one CTA per unit
    (of caches larger than L2, so that the first copies outlast the shortest limit)."""
    cache = _cache(B, T, H, d)
    q = torch.randn((B, H * G, d), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF)
    lens = _ints([T] * B)
    _check(lib, lambda err: kvq.decode_attn(cache, lens, q, err=err))


@pytest.mark.parametrize("B,T,H,G,d,n,kw", [
    (2, 5000, 8, 8, 128, 5, {}), (2, 5000, 8, 8, 64, 5, {}), (1, 3000, 2, 8, 128, 200, {}), (2, 2000, 8, 8, 128, 600, {}),
    (2, 2000, 8, 8, 64, 600, {}), (1, 2000, 2, 8, 128, 100, dict(rising=True)), (1, 900, 2, 4, 64, 300, dict(rising=True)),
    (1, 1000, 2, 8, 128, 90, dict(uneven=True)), (1, 1000, 2, 8, 64, 9, dict(uneven=True))])
def test_prefill(lib, B, T, H, G, d, n, kw):
    """Pairs and single query tiles, split positions and not, O rescaled, tokens with
    exponents of their own."""
    cache = _cache(B, T, H, d, **kw)
    q = torch.randn((B, n, H * G, d), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF)
    lens = _ints([T] * B)
    _check(lib, lambda err: kvq.prefill_attn(cache, lens, q, err=err))
