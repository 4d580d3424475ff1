"""The join of latent attention's ranges: results of the largest latents, split over every CTA, and
the records that it goes by, after calls whose waits gave up, too."""
import ctypes

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


def _plan(lens, rows, sms):
    """First CTA and number of parts of each unit, where the positions are shared."""
    tpb = -(-rows // 64)
    tiles = [max(1, -(-t // 64)) for t in lens]
    groups = sms // tpb
    per = max(2, -(-sum(tiles) // groups))
    recs, at = [], 0
    for n in tiles:
        a, b = at // per, (at + n - 1) // per
        recs += [[a * tpb + r, b - a + 1] for r in range(tpb)]
        at += n
    return recs


@pytest.mark.parametrize("ns", [0, 1, 3000, 10000, 30000])
@pytest.mark.parametrize("lens,H,n", [([300, 90, 131], 12, 1), ([64, 0, 1000, 5, 700], 40, 3), ([2000] * 9, 16, 1)])
def test_records_are_the_plan_also_when_waits_give_up(lens, H, n, ns):
    """A CTA that gave up in one sequence's range still writes the next one's record, and marks
    its parts as empty: the join reads only what this call has written."""
    B, T, pages = len(lens), max(lens), -(-max(lens) // 64)
    g = torch.Generator(device="cuda").manual_seed(1)
    c, k, q = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((B, T, L), (B, T, R), (B, n, H, L + R)))
    cache = kvq.LatentCache(L, R, 64, B * pages, pages)
    kvq.latent_append(cache, _ints([0] * B), None, c, k, None)
    n_of = [min(n, t) for t in lens]

    def call(ws, err):
        out = torch.zeros((B, n, H, L), device="cuda")
        if n == 1:
            kvq.decode_attn(cache, _ints(lens), q[:, 0].contiguous(), 0.05, out=out[:, 0], workspace=ws, err=err)
        else:
            kvq.prefill_attn(cache, _ints(lens), q, 0.05, out=out, chunk_lens=_ints(n_of), workspace=ws, err=err)
        return out

    ws = torch.zeros(kvq.latent_workspace_bytes(B, H, L, n), dtype=torch.uint8, device="cuda")
    err, lib = _ints([0]), kvq.load()
    want = call(ws.clone(), err)
    assert err.item() == 0
    lib.kvq_test_set_wait_limit_ns(ctypes.c_uint64(ns))
    try:
        got = call(ws, err)
    finally:
        lib.kvq_test_set_wait_limit_ns(ctypes.c_uint64(0))
    torch.cuda.synchronize()
    assert err.item() in {0: (0,), 1: (kvq.FLAG_TIMEOUT,)}.get(ns, (0, kvq.FLAG_TIMEOUT))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    recs, tpb = _plan(lens, n * H, sms), -(-n * H // 64)
    assert ws[:B * tpb * 8].view(torch.int32).view(-1, 2).tolist() == recs
    lse = ws[-(-B * tpb * 8 // 256) * 256:][:sms // tpb * tpb * 512].view(torch.float32).view(-1, 2, 64)
    for u, (first, parts) in enumerate(recs):
        b, r = u // tpb, u % tpb
        rows = min(64, n_of[b] * H - 64 * r)
        for i in range(parts if parts > 1 and rows > 0 else 0):
            x = lse[first + i * tpb, 1 if i == 0 else 0, :rows]
            assert (x != 0.0).all()                        # written: -Inf, or a sum of weights
            if ns == 1:
                assert (x == -float("inf")).all()
    if err.item() == 0:
        assert torch.equal(got, want)
    assert torch.equal(call(ws, None), want)               # the next call is as the first
