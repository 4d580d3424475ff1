"""kvq_expanded_attn against float64 attention, row by row against
latent_reference.dense_bound."""
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


def draw(B, n, T, H, d, seed, packed, q_scale=1.0, v_scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, s=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * s).to(BF)

    q = rnd(B, n, H, d + R, s=q_scale)
    if packed:
        kv = rnd(B, T, H, 2 * d)
        kv[..., d:] *= v_scale
        return q, kv[..., :d], rnd(B, T, R + 32)[..., 32:], kv[..., d:]
    return q, rnd(B, T, H, d), rnd(B, T, R), rnd(B, T, H, d, s=v_scale)


def check(out, q, k, kr, v, lens, n_of, scale):
    worst = 0.0
    for b, T in enumerate(lens):
        n = n_of[b]
        if n == 0 or T == 0:
            continue
        for h in range(q.shape[2]):
            kk = torch.cat([k[b, :T, h], kr[b, :T]], -1)
            x, vv = q[b, :n, h], v[b, :T, h].double()
            p = ref.weights(x, kk, scale, torch.arange(T - n, T))
            want = p @ vv
            tol = ref.dense_bound(x, kk, vv, p, scale, out.dtype, want)
            off = (out[b, :n, h].double() - want).abs()
            assert (off <= tol).all(), (b, h, (off / tol).nan_to_num(9e9).max().item())
            worst = max(worst, (off / tol).nan_to_num(0.0).max().item())
    return worst


def run(lens, n, H, d, n_of=None, seed=0, packed=True, dtype=torch.float32, scale=None, T=None, dirty=True, **kw):
    B, T = len(lens), max(max(lens), 1) if T is None else T
    q, k, kr, v = draw(B, n, T, H, d, seed, packed, **kw)
    if dirty:  # what lies behind a sequence's end is not used
        for b, m in enumerate(lens):
            for x in (k, kr, v):
                x[b, m:] = float("nan")
    err = _ints([0])
    out = torch.full((B, n, H, d), 3.0, dtype=dtype, device="cuda")
    pad = None if n_of is None else _ints(n_of)
    n_of = [n] * B if n_of is None else n_of
    scale = 1.0 / math.sqrt(d + R) if scale is None else scale
    assert kvq.expanded_attn(q, k, kr, v, _ints(lens), scale, out=out, chunk_lens=pad, err=err) is out
    assert err.item() == 0
    for b in range(B):
        assert (out[b, n_of[b]:] == 3.0).all()
    return check(out, q, k, kr, v, lens, n_of, scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [1, 3, 8])
@pytest.mark.parametrize("packed", [False, True])
def test_prompts(d, H, packed):
    run([200, 200], 200, H, d, seed=H, packed=packed, dtype=BF if packed else torch.float32)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 63, 64, 65, 127, 128, 129, 255, 256, 257, 600])
def test_chunk_lengths(d, n):
    run([n, n + 1, n + 127, n + 300], n, 2, d, seed=n)


def test_padded_batches():
    run([500, 64, 17, 300, 5], 64, 3, 128, n_of=[40, 64, 0, 1, 5], seed=1)
    run([1000, 700], 700, 2, 64, n_of=[513, 700], seed=2, dtype=BF, T=1111)


def test_long_contexts():
    run([20011, 900], 5, 2, 128, seed=3)
    run([3001], 3001, 2, 64, seed=4, dtype=BF)


@pytest.mark.parametrize("scale,q_scale,v_scale", [(0.003, 1.0, 1.0), (2.0, 1.0, 1.0), (1e-18, 1e18, 1e-20), (0.1, 1.0, 1e30)])
def test_ranges(scale, q_scale, v_scale):
    run([300, 129], 129, 2, 128, seed=5, scale=scale, q_scale=q_scale, v_scale=v_scale)


def test_each_position_counts():
    T, d = 700, 128
    q, k, kr, v = draw(1, T, T, 1, d, 6, False)
    at = torch.tensor([0, 1, 63, 64, 65, 127, 128, 300, 511, 512, 640, 698, 699], device="cuda")
    q[0, at, 0] = torch.cat([k[0, at, 0], kr[0, at]], -1)
    out = kvq.expanded_attn(q, k, kr, v, _ints([T]), 1.0)
    assert ((out[0, at, 0] - v[0, at, 0].float()).abs().amax() < 0.2)
    check(out, q, k, kr, v, [T], [T], 1.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_later_values_do_not_reach_earlier_rows(bad):
    """Inf and NaN among keys and values: rows before their position stay as they were, bit for
    bit; the rows from a value's position on are not finite in its channel."""
    T, d = 300, 128
    q, k, kr, v = draw(1, T, T, 2, d, 10, True)
    want = kvq.expanded_attn(q, k, kr, v, _ints([T]))
    for pos, ch in ((0, 0), (77, 5), (150, 64), (299, 127)):
        w = v.clone()
        w[0, pos, 1, ch] = bad
        got = kvq.expanded_attn(q, k, kr, w, _ints([T]))
        hit = torch.zeros_like(want, dtype=torch.bool)
        hit[0, pos:, 1, ch] = True
        assert torch.equal(got[~hit], want[~hit]) and not torch.isfinite(got[hit]).any()
        kk = k.clone()
        kk[0, pos, 0, ch] = float("nan")
        got = kvq.expanded_attn(q, kk, kr, v, _ints([T]))
        assert torch.equal(got[:, :pos], want[:, :pos]) and torch.isnan(got[:, pos:, 0]).all()
        assert torch.equal(got[:, :, 1], want[:, :, 1])


def test_flags_and_skipped_sequences():
    q, k, kr, v = draw(5, 6, 50, 2, 64, 7, True)
    err = _ints([0])
    out = torch.full((5, 6, 2, 64), 3.0, device="cuda")
    kvq.expanded_attn(q, k, kr, v, _ints([50, 51, 3, 40, -1]), out=out, chunk_lens=_ints([6, 6, 5, 7, 2]), err=err)
    assert err.item() == kvq.FLAG_BAD_LENGTH
    assert (out[1] == 3.0).all() and (out[3] == 3.0).all()
    assert not out[2, :5].any() and (out[2, 5:] == 3.0).all() and not out[4, :2].any() and (out[4, 2:] == 3.0).all()
    check(out[:1], q[:1], k[:1], kr[:1], v[:1], [50], [6], 1.0 / math.sqrt(128))


def test_an_empty_context():
    q, k, kr, v = draw(2, 3, 0, 2, 64, 8, False)
    err = _ints([0])
    out = kvq.expanded_attn(q, k, kr, v, _ints([0, 0]), chunk_lens=_ints([0, 2]), err=err)
    assert err.item() == kvq.FLAG_BAD_LENGTH and not out.any()


def test_refusals():
    q, k, kr, v = draw(2, 3, 9, 2, 64, 9, False)
    lens = _ints([9, 9])
    for bad in (dict(q=q.float()), dict(q=q[:, :, :1]), dict(q=q.transpose(1, 2)), dict(k=k[:, :8]), dict(kr=kr[..., :32]),
                dict(v=v.cpu()), dict(lens=lens.long()), dict(lens=_ints([9])), dict(chunk_lens=_ints([3])),
                dict(out=torch.empty((2, 3, 2, 64), dtype=torch.float16, device="cuda"))):
        a = dict(q=q, k=k, kr=kr, v=v, lens=lens) | bad
        with pytest.raises(ValueError):
            kvq.expanded_attn(a.pop("q"), a.pop("k"), a.pop("kr"), a.pop("v"), a.pop("lens"), **a)
