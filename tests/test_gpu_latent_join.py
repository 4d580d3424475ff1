"""The join of latent attention's ranges: results of the largest latents, split over every CTA."""
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


@pytest.mark.parametrize("T", [200, 5000, 20000])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_the_largest_latents_over_split_ranges(T, dtype):
    """Latents of 1.5e38 .. 2.9e38 in every token: the parts' sum is past fp32, the result is not."""
    g = torch.Generator(device="cuda").manual_seed(T)
    c = ((1.5 + 1.4 * torch.rand((1, T, L), generator=g, device="cuda")) * 1e38).to(BF)
    k = torch.zeros((1, T, R), dtype=BF, device="cuda")
    mp = -(-T // 64)
    cache = kvq.LatentCache(L, R, 64, mp, mp)
    kvq.latent_append(cache, _ints([0]), None, c, k, None)
    q = torch.zeros((1, 4, L + R), dtype=BF, device="cuda")
    out = kvq.decode_attn(cache, _ints([T]), q, 1.0, out=torch.empty((1, 4, L), dtype=dtype, device="cuda"))
    codes, e = ref.read_pool(cache.pool, None, mp, 0, T, 64, L, R)
    lat, key = ref.decode(codes, e, L)
    p = ref.weights(q[0], torch.cat([lat, key], -1), 1.0, torch.full((4,), T - 1))
    want = p @ lat
    tol = ref.attn_bound(q[0], lat, key, ref.power(e - 127), p, 1.0, dtype, want)
    assert torch.isfinite(out).all() and ((out[0].double() - want).abs() <= tol).all()
