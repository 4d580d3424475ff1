"""The NVFP4 rotary append at block maxima whose sixth lies next to a border
between two E4M3 scales.  With the second-level scale a little above amax / 2688
(1.2 times, as a program that leaves headroom sets it) the maxima of a head land
there for some significands; a sixth taken as a product with the rounded 1 / 6
instead of a quotient then moves the whole block's scale by a step of E4M3."""
import numpy as np
import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests import block8_reference as ref
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def nvfp4_values(x, S):
    """(E2M1 code value * block scale, block scales) in float64 of x, bf16
    [B][n][H][d], by the definition: y = fp32(x / S), scale the E4M3 value nearest
    to y's block maximum / 6, code the E2M1 value nearest to fp32(y / scale)."""
    y = x.float().numpy() / S.numpy()[:, None]
    y = torch.from_numpy(y.reshape(*y.shape[:-1], -1, 16))
    s = ref.e4m3_round(y.abs().amax(-1, keepdim=True).double() / 6.0).clamp(min=2.0 ** -9)
    a = torch.from_numpy(np.abs(y.numpy()) / s.float().numpy()).double().clamp(max=6.0)
    hi = torch.searchsorted(GRID, a.contiguous()).clamp(1, 7)
    up, dn = GRID[hi], GRID[hi - 1]
    m = torch.where((up - a < a - dn) | ((up - a == a - dn) & (hi % 2 == 0)), up, dn)
    return (torch.copysign(m * s, y.double())).reshape(x.shape), s[..., 0]


@pytest.mark.parametrize("rotate", [False, True])
def test_scales_next_to_a_border(rotate):
    """One kv head per bf16 significand of the head's maximum, 128 blocks by the
    significand of their own, each at three magnitudes."""
    H, d, n, mp = 128, 64, 96, 6
    g = torch.Generator().manual_seed(3)
    sig = 1.0 + torch.arange(128) / 128.0
    top = sig * 2.0 ** (torch.arange(H) % 7 - 3)
    block = (sig * torch.tensor([2.0 ** -2, 2.0 ** -5, 2.0 ** -9])[:, None]).reshape(1, n, 1, d // 16, 1)
    sides = []
    for _ in range(2):
        x = (torch.rand((1, n, H, d // 16, 16), generator=g) * 2 - 1) * block
        x[..., 0] = block[..., 0]
        sides.append(x.reshape(1, n, H, d).to(BF))
    k, v = sides
    S = (1.2 * top) * torch.tensor(1.0 / 2688.0, dtype=torch.float32)
    cache = kvq.Fp4Cache(H, d, 16, mp, mp, nvfp4=True)
    cache.k_gscale.copy_(S)
    cache.v_gscale.copy_(S)
    # (positions 0: the rotation is the identity there, so that the maxima stay)
    table = torch.zeros((n, 64), device="cuda")
    table[:, :32] = 1.0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.rope_append(cache, start, None, k.cuda(), v.cuda(), table if rotate else None, err=err)
    got = kvq.dequant(cache, start + n, n)
    assert err.item() == 0
    quotient_differs = 0
    for x, out in ((k, got[0]), (v, got[1])):
        want, s = nvfp4_values(x, S)
        out = out.cpu().double() / S.double()[:, None]
        # the read-back rounds value * S to fp32: half a step, 2^-24 of it
        assert ((out - want).abs() <= 2.0 ** -24 * want.abs()).all()
        y = torch.from_numpy(x.float().numpy() / S.numpy()[:, None]).reshape(1, n, H, -1, 16).abs().amax(-1)
        product = ref.e4m3_round((y * torch.tensor(1.0 / 6.0, dtype=torch.float32)).double()).clamp(min=2.0 ** -9)
        quotient_differs += int((product != s).sum())
    assert quotient_differs > 0  # the case does tell the two apart
