"""The latent operators together, as a serving loop runs them: prompts appended with
the rotation and attended in chunks (absorbed, and expanded over the read-back), then
tokens decoded one by one -- eager, captured and replayed, on other streams, beside one
another, with waits that give up -- against float64 over latents quantised on the host."""
import ctypes
import math

import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests import latent_reference as ref
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
L, R, H, D, B, CAP, PAGE = 512, 64, 12, 128, 3, 320, 32
SCALE = 1.0 / math.sqrt(D + R)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _draw(seed, n):
    """A packed down-projection, query position parts behind 128 other channels, absorbed queries."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, n, L + R), generator=g) * torch.exp(0.3 * torch.randn((B, n, 1), generator=g))
    return (x.to(BF).cuda(), torch.randn((B, n, H, D + R), generator=g).to(BF).cuda(),
            (0.3 * torch.randn((B, n, H, L + R), generator=g)).to(BF).cuda())


class Loop:
    """A program's state: one layer's cache, its buffers and workspaces."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        mp = CAP // PAGE
        self.cache = kvq.LatentCache(L, R, PAGE, B * mp, mp,
                                     page_table=torch.randperm(B * mp, generator=g).to(torch.int32).view(B, mp).cuda())
        self.cache.pool.random_(0, 256)
        self.table = kvq.rope_table(CAP, R)
        self.err, self.lens, self.start = _ints([0]), _ints([0] * B), _ints([0] * B)
        self.down, self.qp, self.q = (torch.zeros_like(x) for x in _draw(0, 1))
        self.out = torch.empty((B, H, L), dtype=BF, device="cuda")
        self.ws = torch.empty(kvq.latent_workspace_bytes(B, H, L), dtype=torch.uint8, device="cuda")

    def append(self, x, lens):
        down, qp, q = x
        n = _ints(lens)
        kvq.latent_append(self.cache, self.lens, qp[..., D:], down[..., :L], down[..., L:], self.table, new_lens=n,
                          q_out=q[..., L:], err=self.err)
        self.lens += n
        return q, n

    def prompt(self, x, lens):
        q, n = self.append(x, lens)
        return kvq.prefill_attn(self.cache, self.lens, q, SCALE, chunk_lens=n, err=self.err)

    def step(self):
        """One token per sequence from down, qp and q, at position lens - 1 after the increment."""
        self.start.copy_(self.lens)
        self.lens += 1
        kvq.latent_append(self.cache, self.start, self.qp[..., D:], self.down[..., :L], self.down[..., L:], self.table,
                          q_out=self.q[..., L:], err=self.err)
        kvq.decode_attn(self.cache, self.lens, self.q[:, 0], SCALE, out=self.out, workspace=self.ws, err=self.err)

    def feed(self, x):
        for a, b in zip((self.down, self.qp, self.q), x):
            a.copy_(b)


class Host:
    def __init__(self, table):
        self.table, self.lens = table, [0] * B
        self.codes = torch.zeros((B, CAP, L + 2 * R), dtype=torch.float64, device="cuda")
        self.e = torch.ones((B, CAP), dtype=torch.int64, device="cuda")

    def append(self, x, lens):
        down, qp, q = x
        kr = ref.rotate32(down[..., L:], self.lens, self.table, False)
        q = torch.cat([q[..., :L], ref.rotate32(qp[..., D:], self.lens, self.table, False)], -1)
        codes, e = ref.encode(down[..., :L], kr)
        for b in range(B):
            a, n = self.lens[b], lens[b]
            self.codes[b, a:a + n], self.e[b, a:a + n] = codes[b, :n], e[b, :n].long()
            self.lens[b] = a + n
        return q

    def check(self, out, q, lens):
        """out [B][n][H][L], q [B][n][H][L + R]."""
        for b in range(B):
            n, T = lens[b], self.lens[b]
            if n == 0:
                continue
            c, k = ref.decode(self.codes[b, :T], self.e[b, :T], L)
            x = q[b, :n].reshape(-1, L + R)
            p = ref.weights(x, torch.cat([c, k], -1), SCALE, torch.arange(T - n, T).repeat_interleave(H))
            want = p @ c
            tol = ref.attn_bound(x, c, k, ref.power(self.e[b, :T] - 127), p, SCALE, out.dtype, want)
            assert ((out[b, :n].reshape(-1, L).double() - want).abs() <= tol).all(), b


def test_a_serving_loop():
    loop = Loop(0)
    host = Host(loop.table)
    for seed, lens in ((1, [70, 33, 0]), (2, [5, 64, 40])):
        x = _draw(seed, max(lens))
        want = host.append(tuple(t.clone() for t in x), lens)
        host.check(loop.prompt(x, lens), want, lens)
    for s in range(20):                                       # past page and tile borders
        x = _draw(100 + s, 1)
        want = host.append(tuple(t.clone() for t in x), [1] * B)
        loop.feed(x)
        loop.step()
        host.check(loop.out[:, None], want, [1] * B)
    assert loop.err.item() == 0 and loop.lens.tolist() == host.lens


def test_the_expanded_form_agrees_with_the_absorbed_one():
    """Cached latents read back, multiplied out per head and attended as dense keys and values,
    against the absorbed form of the same weights: both within the bounds of their roundings
    (the multiplied keys, values, queries and results are rounded to bf16 on the way)."""
    loop = Loop(1)
    x = _draw(3, 200)
    lens = [200, 77, 130]
    _, n = loop.append(x, lens)
    g = torch.Generator().manual_seed(4)
    wk, wv = (torch.randn((H, L, D), generator=g).to(BF).cuda() / math.sqrt(L) for _ in range(2))
    c, kr = kvq.dequant(loop.cache, loop.lens, 200, dtype=BF)
    kv = torch.stack([torch.einsum("btl,hld->bthd", c.float(), w.float()) for w in (wk, wv)], 3).to(BF).flatten(3)
    qn = x[1][..., :D]
    qe = torch.cat([qn, x[2][..., L:]], -1).contiguous()
    dense = kvq.expanded_attn(qe, kv[..., :D], kr, kv[..., D:], loop.lens, SCALE, chunk_lens=n)
    qa = torch.cat([torch.einsum("bthd,hld->bthl", qn.float(), wk.float()).to(BF), x[2][..., L:]], -1).contiguous()
    lat = kvq.prefill_attn(loop.cache, loop.lens, qa, SCALE, chunk_lens=n)
    got = torch.einsum("bthl,hld->bthd", lat, wv.float())
    for b, m in enumerate(lens):
        a, d = got[b, :m], dense[b, :m]
        assert ((a - d).norm() / d.norm()).item() < 0.02  # a dozen bf16 roundings of 2^-9 each


def _replays(loop, step, eager):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        saved = loop.cache.pool.clone(), loop.lens.clone()
        step()                                                # warm-up (module load, attributes)
        loop.cache.pool.copy_(saved[0])
        loop.lens.copy_(saved[1])
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    return g


def test_a_captured_step_replays():
    eager, graph = Loop(3), Loop(3)
    eager.cache.pool.copy_(graph.cache.pool)
    for loop in (eager, graph):
        loop.prompt(_draw(4, 50), [50, 1, 31])
    g = _replays(graph, graph.step, eager)
    for s in range(20):
        x = _draw(200 + s, 1)
        eager.feed(x)
        eager.step()
        graph.feed(x)
        g.replay()
        assert torch.equal(eager.out, graph.out), s
    assert torch.equal(eager.cache.pool, graph.cache.pool) and torch.equal(eager.lens, graph.lens)
    assert eager.err.item() == graph.err.item() == 0


def test_captured_chunks_replay():
    """A chunk over the cache and one over dense keys, captured; the workspace and the output
    are overwritten between replays."""
    loop = Loop(5)
    loop.prompt(_draw(6, 60), [60, 60, 60])
    q = _draw(7, 9)[2]
    want = kvq.prefill_attn(loop.cache, loop.lens, q, SCALE)
    ws = torch.empty(kvq.latent_workspace_bytes(B, H, L, 9), dtype=torch.uint8, device="cuda")
    out = torch.zeros((B, 9, H, L), device="cuda")
    kv, kr, qe = (torch.randn(s, device="cuda").to(BF) for s in ((B, 60, H, 2 * D), (B, 60, R), (B, 9, H, D + R)))
    dense = kvq.expanded_attn(qe, kv[..., :D], kr, kv[..., D:], loop.lens)
    out2 = torch.zeros_like(dense)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.prefill_attn(loop.cache, loop.lens, q, SCALE, out=out, workspace=ws)
        kvq.expanded_attn(qe, kv[..., :D], kr, kv[..., D:], loop.lens, out=out2)
    for _ in range(3):
        out.zero_()
        out2.zero_()
        ws.random_(0, 256)
        g.replay()
        assert torch.equal(out, want) and torch.equal(out2, dense)


def test_two_loops_on_two_streams():
    loops, hosts, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    xs = [[_draw(10 * i + s, 30 if s == 0 else 1) for s in range(9)] for i in range(2)]
    wants = [[], []]
    for i in range(2):
        loops.append(Loop(20 + i))
        hosts.append(Host(loops[i].table))
        hosts[i].append(tuple(t.clone() for t in xs[i][0]), [30, 7, 16])
    torch.cuda.synchronize()
    outs = [[], []]
    for s in range(9):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                if s == 0:
                    loops[i].prompt(xs[i][0], [30, 7, 16])
                else:
                    loops[i].feed(xs[i][s])
                    loops[i].step()
                    outs[i].append(loops[i].out.clone())
    torch.cuda.synchronize()
    for i in range(2):
        for s in range(1, 9):
            hosts[i].check(outs[i][s - 1][:, None], hosts[i].append(xs[i][s], [1] * B), [1] * B)
        assert loops[i].err.item() == 0


def test_an_explicit_stream():
    """A stream argument: buffers made by the call come from that stream's memory."""
    loop = Loop(30)
    x = _draw(31, 40)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    n = _ints([40, 40, 40])
    q = x[2].clone()
    s.wait_stream(torch.cuda.current_stream())
    kvq.latent_append(loop.cache, loop.lens, x[1][..., D:], x[0][..., :L], x[0][..., L:], loop.table, q_out=q[..., L:], stream=s)
    out = kvq.prefill_attn(loop.cache, n, q, SCALE, stream=s)
    c, k = kvq.dequant(loop.cache, n, 40, stream=s)
    s.synchronize()
    host = Host(loop.table)
    host.check(out, host.append(x, [40] * B), [40] * B)
    assert torch.equal(c[1].double(), ref.decode(host.codes[1, :40], host.e[1, :40], L)[0])


def test_back_to_back_decodes_share_a_workspace():
    loop = Loop(32)
    loop.prompt(_draw(33, 300), [300, 90, 131])
    qs = [_draw(34 + i, 1)[2][:, 0].contiguous() for i in range(12)]
    want = [kvq.decode_attn(loop.cache, loop.lens, q, SCALE) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [kvq.decode_attn(loop.cache, loop.lens, q, SCALE, workspace=loop.ws, out=None) for q in qs]
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("ns", [1, 2000, 20000, 100000])
def test_waits_that_give_up(ns):
    """With the wait limit shortened the attention returns with the TIMEOUT flag (or in time) and
    the next call at the default limit gives what it gave before."""
    loop = Loop(40)
    loop.prompt(_draw(41, 300), [300, 90, 131])
    q = _draw(42, 1)[2][:, 0].contiguous()
    kv, kr, qe = (torch.randn(s, device="cuda").to(BF) for s in ((B, 300, H, 2 * D), (B, 300, R), (B, 200, H, D + R)))
    lens = _ints([300, 200, 250])

    def both(err=None):
        return (kvq.decode_attn(loop.cache, loop.lens, q, SCALE, err=err),
                kvq.expanded_attn(qe, kv[..., :D], kr, kv[..., D:], lens, err=err))

    want = both()
    L_ = kvq.load()
    for which in range(2):
        err = _ints([0])
        L_.kvq_test_set_wait_limit_ns(ctypes.c_uint64(ns))
        try:
            if which:
                kvq.decode_attn(loop.cache, loop.lens, q, SCALE, err=err)
            else:
                kvq.expanded_attn(qe, kv[..., :D], kr, kv[..., D:], lens, err=err)
        finally:
            L_.kvq_test_set_wait_limit_ns(ctypes.c_uint64(0))
        torch.cuda.synchronize()
        assert err.item() in ((kvq.FLAG_TIMEOUT,) if ns == 1 else (0, kvq.FLAG_TIMEOUT))
    for a, b in zip(both(), want):
        assert torch.equal(a, b)
