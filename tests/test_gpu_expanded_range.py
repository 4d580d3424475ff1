"""kvq_expanded_attn at the ends of its values' range, against float64: values up to the largest
bf16 under weights that are equal or rise along the positions, small values, and rows
all of whose scores are -Inf."""
import math

import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests import latent_reference as ref
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
R = 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(n, T, H, d, ramp, v, dtype=torch.float32, extra=0.0):
    """Scores ramp[t] for every row; v [T][H][d].  extra: absolute error allowed beside the bound."""
    q = torch.zeros((1, n, H, d + R), dtype=BF, device="cuda")
    q[..., d] = 1.0
    k = torch.zeros((1, T, H, d), dtype=BF, device="cuda")
    kr = torch.zeros((1, T, R), dtype=BF, device="cuda")
    kr[0, :, 0] = ramp.to(BF)
    v = v.to(BF)[None]
    assert torch.isfinite(v).all()
    out = kvq.expanded_attn(q, k, kr, v, _ints([T]), 1.0, out=torch.empty((1, n, H, d), dtype=dtype, device="cuda"))
    assert torch.isfinite(out).all()
    for h in range(H):
        kk = torch.cat([k[0, :, h], kr[0]], -1)
        p = ref.weights(q[0, :, h], kk, 1.0, torch.arange(T - n, T))
        vv = v[0, :, h].double()
        want = p @ vv
        tol = ref.dense_bound(q[0, :, h], kk, vv, p, 1.0, dtype, want) + extra
        off = (out[0, :, h].double() - want).abs()
        assert (off <= tol).all(), (h, (off / tol).amax().item())


def _values(T, H, d, size, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, H, d), generator=g, device="cuda").clamp(-3.0, 3.0) * (size / 3.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e33, 3e38])
@pytest.mark.parametrize("rise", [5.0, 13.0, 40.0, 200.0])
def test_rising_scores_over_large_values(d, size, rise):
    """The weights rise by up to 2^19 (13), or past it, from the first position to the last."""
    T = 300
    run(T, T, 2, d, torch.linspace(0.0, rise, T, device="cuda"), _values(T, 2, d, size, 1))


def test_a_late_step_over_large_values():
    """Thousands of equal scores, then many 2^k above them."""
    T = 3000
    for step in (0.5, 3.0, 6.0, 13.5):
        ramp = torch.zeros(T, device="cuda")
        ramp[1000:] = step
        run(200, T, 1, 128, ramp, _values(T, 1, 128, 3e38, 2).abs())


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_equal_weights_over_the_largest_values(dtype):
    """Every value at 3.2e38 .. 3.36e38: their sum of 5000 is far past fp32."""
    T = 5000
    g = torch.Generator(device="cuda").manual_seed(3)
    v = 3.2e38 + 0.16e38 * torch.rand((T, 2, 64), generator=g, device="cuda")
    run(130, T, 2, 64, torch.zeros(T, device="cuda"), v, dtype=dtype)


def test_small_values_keep_their_precision():
    """Products of a weight and a value under 2^-126 may count 0.  Weights are at least 2^-17 at a
    row's largest score (8 for the room above it, 9 for 300 positions): under T 2^(17 - 126)."""
    T = 300
    run(T, T, 2, 128, torch.linspace(0.0, 4.0, T, device="cuda"), _values(T, 2, 128, 1e-26, 4), extra=T * 2.0 ** -109)


def test_rows_whose_scores_are_all_minus_inf():
    """0 / 0 by the definition: NaN, not 0; rows that see one finite score take its weight."""
    T, d, H = 200, 64, 2
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.zeros((1, T, H, d + R), dtype=BF, device="cuda")
    q[..., 0] = 1.0
    k = torch.zeros((1, T, H, d), dtype=BF, device="cuda")
    k[0, :90, 1, 0] = -math.inf
    kr = torch.zeros((1, T, R), dtype=BF, device="cuda")
    v = torch.randn((1, T, H, d), generator=g, device="cuda").to(BF)
    out = kvq.expanded_attn(q, k, kr, v, _ints([T]), 1.0)[0]
    assert torch.isnan(out[:90, 1]).all()
    assert torch.isfinite(out[:, 0]).all() and torch.isfinite(out[90:, 1]).all()
    vv = v[0, :, 1].double()
    for i in range(90, T):
        want, size = vv[90:i + 1].mean(0), vv[90:i + 1].abs().mean(0)
        assert ((out[i, 1].double() - want).abs() <= size * (2.0 ** -8 + 2.0 ** -18)).all(), i
