"""kvq_expanded_attn at scores whose fp32 steps are large: one token outweighs all others by far more
than any rounding, or stands in two equal copies, so the row is that token's value, whatever the
score's size.  Bound: the weight's rounding to bf16, 2^-8 counted for sum and copies, and 2^-20."""
import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
R = 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [2e3, 3e6, 3e7, 7e7, 5e8, 3e9, 7e11, 3e20, 5e30])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_one_token_or_two_equal_ones(d, size, sign):
    """Scores up to size; sign -1: the dominant token's is the one near 0 among large negative ones."""
    T, n, H = 500, 130, 4
    g = torch.Generator(device="cuda").manual_seed(d)
    v = torch.randn((1, T, H, d), generator=g, device="cuda").to(BF)
    k = torch.zeros((1, T, H, d), dtype=BF, device="cuda")
    kr = torch.zeros((1, T, R), dtype=BF, device="cuda")
    q = torch.zeros((1, n, H, d + R), dtype=BF, device="cuda")
    picked = [(0, 0), (90, 91), (300, 17), (369, 80)]
    level = (0.1 + 0.5 * torch.rand((T, H), generator=g, device="cuda")) if sign > 0 else \
        -(0.5 + 0.4 * torch.rand((T, H), generator=g, device="cuda"))
    for h, (a, b) in enumerate(picked):
        level[[a, b], h] = 1.0 if sign > 0 else -0.01
    k[0, :, :, 3] = level.to(BF)
    unit = size                                                # (the gap is 0.4 of it at least, times 0.7)
    q[..., 3] = torch.tensor(unit).to(BF)
    out = kvq.expanded_attn(q, k, kr, v, torch.tensor([T], dtype=torch.int32, device="cuda"), 0.7)
    want = torch.stack([(v[0, a, h].double() + v[0, b, h].double()) / 2 for h, (a, b) in enumerate(picked)])
    size_of = torch.stack([(v[0, a, h].double().abs() + v[0, b, h].double().abs()) / 2 for h, (a, b) in enumerate(picked)])
    assert torch.isfinite(out).all()
    assert ((out[0].double() - want).abs() <= size_of * (2.0 ** -8 + 2.0 ** -20)).all()


@pytest.mark.parametrize("size", [0.0, 1e4, 1e6, 3e7, 1.2e8])
def test_equal_large_scores_over_the_largest_values(size):
    """5000 equal scores up to 2^27, values of 3.2e38 .. 3.36e38: their mean, not Inf."""
    T, n, d = 5000, 130, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    v = (3.2e38 + 0.16e38 * torch.rand((1, T, 1, d), generator=g, device="cuda")).to(BF)
    k = torch.zeros((1, T, 1, d), dtype=BF, device="cuda")
    k[..., 3] = 1.0
    q = torch.zeros((1, n, 1, d + R), dtype=BF, device="cuda")
    q[..., 3] = size
    kr = torch.zeros((1, T, R), dtype=BF, device="cuda")
    out = kvq.expanded_attn(q, k, kr, v, torch.tensor([T], dtype=torch.int32, device="cuda"), 0.7)
    want = v[0, :, 0].double().cumsum(0)[T - n:] / torch.arange(T - n + 1, T + 1, device="cuda")[:, None]
    assert ((out[0, :, 0].double() - want).abs() <= want * (2.0 ** -8 + T / 16 * 2.0 ** -24 + 2.0 ** -20)).all()
