"""The operators together, as a serving loop runs them: prompts appended with
the rotation and attended in chunks, then tokens decoded one by one -- eager,
captured into a graph and replayed, on other streams, beside one another --
against float64 attention over keys rotated and quantised on the host."""
import math

import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests import block8_reference as ref
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
H, G, D, B, CAP, PAGE = 2, 4, 128, 3, 288, 32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Loop:
    """A program's state: one layer's cache, its buffers and workspaces."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        mp = CAP // PAGE
        self.cache = kvq.Fp8BlockCache(H, D, PAGE, B * mp, mp,
                                       page_table=torch.randperm(B * mp, generator=g).to(torch.int32).view(B, mp).cuda())
        self.table = kvq.rope_table(CAP, D)
        self.err = _ints([0])
        self.lens = _ints([0] * B)
        self.start = _ints([0] * B)
        self.qkv = torch.zeros((B, 1, (G + 2) * H, D), dtype=BF, device="cuda")
        self.q = torch.empty((B, 1, G * H, D), dtype=BF, device="cuda")
        self.out = torch.empty((B, G * H, D), dtype=BF, device="cuda")
        self.ws = torch.empty(kvq.decode_workspace_bytes(B, G * H, H, D), dtype=torch.uint8, device="cuda")

    def prompt(self, x, lens):
        """x [B][n][(G + 2) H][D], lens[b] of its tokens."""
        q, k, v = x[:, :, :G * H], x[:, :, G * H:(G + 1) * H], x[:, :, (G + 1) * H:]
        n = _ints(lens)
        qr = kvq.rope_append(self.cache, self.lens, q, k, v, self.table, new_lens=n, err=self.err)
        self.lens += n
        return kvq.prefill_attn(self.cache, self.lens, qr, chunk_lens=n, err=self.err)

    def step(self):
        """One token per sequence from self.qkv, at position lens - 1 after the increment."""
        self.start.copy_(self.lens)
        self.lens += 1
        x = self.qkv
        kvq.rope_append(self.cache, self.start, x[:, :, :G * H], x[:, :, G * H:(G + 1) * H], x[:, :, (G + 1) * H:],
                        self.table, q_out=self.q, err=self.err)
        kvq.decode_attn(self.cache, self.lens, self.q[:, 0], out=self.out, workspace=self.ws, err=self.err)


class Host:
    def __init__(self, table):
        self.cache, self.table, self.lens = ref.BlockCache(B, H, D, CAP), table.cpu(), [0] * B

    def append(self, x, lens):
        x = x.cpu()
        kr = ref.rotate32(x[:, :, G * H:(G + 1) * H], self.lens, self.table, False)
        qr = ref.rotate32(x[:, :, :G * H], self.lens, self.table, False)
        self.cache.append(self.lens, kr, x[:, :, (G + 1) * H:], lens)
        self.lens = [a + n for a, n in zip(self.lens, lens)]
        return qr

    def check(self, out, qr, lens, prefill):
        """out, qr [B][n][G H][D]."""
        for b in range(B):
            n, T = lens[b], self.lens[b]
            if n == 0:
                continue
            for h in range(H):
                k, v = self.cache.values(0, b, T)[:, h], self.cache.values(1, b, T)[:, h]
                want, A, bq = ref.attend(qr[b, :n, h * G:(h + 1) * G], k, v, 1 / math.sqrt(D), torch.arange(T - n, T))
                tol = ref.tolerance(D, T, float(v.abs().max()), A, bq if prefill else None, out.dtype, want.abs())
                assert ((out[b, :n, h * G:(h + 1) * G].cpu().double() - want).abs() <= tol).all(), (b, h)


def _draw(seed, n):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((B, n, (G + 2) * H, D), generator=g).to(BF).cuda()


def test_a_serving_loop():
    loop = Loop(0)
    host = Host(loop.table)
    for seed, lens in ((1, [70, 33, 0]), (2, [5, 64, 40])):   # two rounds of ragged prompts
        x = _draw(seed, max(lens))
        host.check(loop.prompt(x, lens), host.append(x, lens), lens, True)
    for s in range(20):                                       # past block and page borders
        x = _draw(100 + s, 1)
        loop.qkv.copy_(x)
        loop.step()
        host.check(loop.out[:, None], host.append(x, [1] * B), [1] * B, False)
    assert loop.err.item() == 0 and loop.lens.tolist() == host.lens


def test_a_captured_step_replays():
    """The step captured into a graph and replayed gives the eager steps' bytes."""
    eager, graph = Loop(3), Loop(3)
    x = _draw(4, 50)
    for loop in (eager, graph):
        loop.prompt(x, [50, 1, 31])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        saved = graph.cache.pool.clone(), graph.lens.clone()
        graph.step()                                          # warm-up (module load, attributes)
        graph.cache.pool.copy_(saved[0])
        graph.lens.copy_(saved[1])
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.step()
    for s in range(20):
        x = _draw(200 + s, 1)
        eager.qkv.copy_(x)
        eager.step()
        graph.qkv.copy_(x)
        g.replay()
        assert torch.equal(eager.out, graph.out), s
    assert torch.equal(eager.cache.pool, graph.cache.pool) and torch.equal(eager.lens, graph.lens)
    assert eager.err.item() == graph.err.item() == 0


def test_a_captured_prefill_replays():
    loop = Loop(5)
    x = _draw(6, 60)
    loop.prompt(x, [60, 60, 60])
    q = _draw(7, 9)[:, :, :G * H].contiguous()
    want = kvq.prefill_attn(loop.cache, loop.lens, q)
    ws = torch.empty(kvq.prefill_workspace_bytes(B, G * H, H, D, 9), dtype=torch.uint8, device="cuda")
    out = torch.zeros(q.shape, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.prefill_attn(loop.cache, loop.lens, q, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        ws.random_(0, 256)
        g.replay()
        assert torch.equal(out, want)


def test_two_loops_on_two_streams():
    """Calls on different streams with buffers of their own do not meet."""
    loops, hosts, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    xs = [[_draw(10 * i + s, 30 if s == 0 else 1) for s in range(9)] for i in range(2)]
    for i in range(2):
        loops.append(Loop(20 + i))
        hosts.append(Host(loops[i].table))
    torch.cuda.synchronize()
    outs = [[], []]
    for s in range(9):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                if s == 0:
                    loops[i].prompt(xs[i][0], [30, 7, 16])
                else:
                    loops[i].qkv.copy_(xs[i][s])
                    loops[i].step()
                    outs[i].append(loops[i].out.clone())
    torch.cuda.synchronize()
    for i in range(2):
        hosts[i].append(xs[i][0], [30, 7, 16])
        for s in range(1, 9):
            hosts[i].check(outs[i][s - 1][:, None], hosts[i].append(xs[i][s], [1] * B), [1] * B, False)
        assert loops[i].err.item() == 0


def test_back_to_back_decodes_share_a_workspace():
    """Steps in a row on one stream with one workspace, nothing waited for."""
    loop = Loop(30)
    loop.prompt(_draw(31, 200), [200, 90, 131])
    qs = [_draw(32 + i, 1)[:, 0, :G * H].contiguous() for i in range(12)]
    want = [kvq.decode_attn(loop.cache, loop.lens, q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [kvq.decode_attn(loop.cache, loop.lens, q, workspace=loop.ws) for q in qs]
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_queries_rotated_in_place_reach_the_attention():
    """q rotated in place, the decode launched behind the append at once."""
    loop = Loop(40)
    loop.prompt(_draw(41, 100), [100, 3, 64])
    for s in range(30):
        x = _draw(42 + s, 1)
        q, k, v = (t.contiguous() for t in (x[:, :, :G * H], x[:, :, G * H:(G + 1) * H], x[:, :, (G + 1) * H:]))
        want = ref.rotate32(q.cpu(), loop.lens.tolist(), loop.table.cpu(), False)
        start = loop.lens.clone()
        loop.lens += 1
        kvq.rope_append(loop.cache, start, q, k, v, loop.table, q_out=q)
        out = kvq.decode_attn(loop.cache, loop.lens, q[:, 0])
        again = kvq.decode_attn(loop.cache, loop.lens, want[:, 0].cuda().contiguous())
        assert torch.equal(out, again), s
