"""Plain references of the 8-bit block cache, the rotation and attention over
dense values, in float64 on the host (torch CPU tensors), written from the
definitions in include/kvq_fp8_block.h.  Nothing here uses the CUDA library."""
from __future__ import annotations

import math

import torch

ORDER = [0, 1, 8, 9, 2, 3, 10, 11, 4, 5, 12, 13, 6, 7, 14, 15]  # token of a block at byte i of a V row


def e4m3_round(x: torch.Tensor) -> torch.Tensor:
    """Nearest E4M3 value of float64 x, ties to even, saturating at 448."""
    a = x.abs().clamp(max=448.0)
    _, e = torch.frexp(torch.where(a > 0, a, torch.ones_like(a)))
    step = torch.ldexp(torch.ones_like(a), (e - 1).clamp(min=-6) - 3)
    return torch.copysign(torch.round(a / step) * step, x).clamp(-448.0, 448.0)


def block_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    if amax > 448.0 * s:
        s = 2.0 ** (math.frexp(amax / 448.0)[1] - 1)
        if amax > 448.0 * s:
            s *= 2.0
    return s


class BlockCache:
    """Codes (as values) and scales of one layer's cache by position."""

    def __init__(self, batch, heads, d, capacity):
        self.codes = torch.zeros((2, batch, capacity, heads, d), dtype=torch.float64)
        self.scales = torch.zeros((2, batch, capacity // 16, heads), dtype=torch.float64)

    def append(self, start, k, v, new_lens=None):
        B, n = k.shape[:2]
        for side, x in enumerate((k.double(), v.double())):
            for b in range(B):
                sp, m = int(start[b]), n if new_lens is None else int(new_lens[b])
                for blk in range(sp // 16, (sp + m + 15) // 16 if m else 0):
                    lo, hi = max(sp, 16 * blk), min(sp + m, 16 * blk + 16)
                    for h in range(x.shape[2]):
                        new = x[b, lo - sp:hi - sp, h]
                        s, old = block_scale(float(new.abs().max())), float(self.scales[side, b, blk, h])
                        if lo > 16 * blk:
                            s = max(s, old)
                            if s > old:
                                kept = self.codes[side, b, 16 * blk:lo, h]
                                self.codes[side, b, 16 * blk:lo, h] = e4m3_round(kept * (old / s))
                        self.codes[side, b, lo:hi, h] = e4m3_round(new / s)
                        self.scales[side, b, blk, h] = s

    def values(self, side, b, n):
        s = self.scales[side, b].repeat_interleave(16, 0)[:n]
        return self.codes[side, b, :n] * s[..., None]


def read_pool(pool, page_table, max_pages, b, n, page, d):
    """(codes as float64 [2][n][heads][d], scales [2][ceil(n/16)][heads]) of
    positions 0 .. n-1 of sequence b, by byte arithmetic on a host copy."""
    pool = pool.cpu()
    P, H = page, pool.shape[1]
    G = min(P, 64)
    t = torch.arange(n)
    pg = t // P
    phys = (b * max_pages + pg) if page_table is None else page_table.cpu()[b].long()[pg]
    slot = t % P
    block = pool[phys, :, slot // G]                       # [n][H][bytes]
    lt, c = (slot % G)[:, None], torch.arange(d)[None]
    koff = (lt // 8) * (8 * d) + (c // 16) * 128 + (lt % 8) * 16 + c % 16
    byte = torch.tensor([ORDER.index(u) for u in range(16)])[lt % 16]
    voff = G * d + (lt // 16) * (16 * d) + c * 16 + byte
    codes = torch.stack([block.gather(2, off[:, None].expand(n, H, d)) for off in (koff, voff)])
    codes = codes.view(torch.float8_e4m3fn).double()
    sc = []
    for side in range(2):
        first = t[::16]
        o = 2 * G * d + 8 * ((first % G) // 16) + 4 * side
        raw = torch.stack([pool[phys[first], :, slot[first] // G].gather(2, (o + i)[:, None, None].expand(-1, H, 1))[..., 0]
                           for i in range(4)], -1).contiguous()
        sc.append(raw.view(torch.float32)[..., 0].double())
    return codes, torch.stack(sc)


def rotate32(x: torch.Tensor, start, table: torch.Tensor, interleaved: bool) -> torch.Tensor:
    """The rotation as defined: each product and sum rounded to fp32, the
    result to bf16 (x bf16 [B][n][H][d] on the host)."""
    r = table.shape[1]
    pos = torch.as_tensor(start).long()[:, None] + torch.arange(x.shape[1])
    cs = table[pos][:, :, None]
    c, s = cs[..., :r // 2], cs[..., r // 2:]
    y = x.float().clone()
    if interleaved:
        x0, x1 = x.float()[..., 0:r:2], x.float()[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = x0 * c - x1 * s, x1 * c + x0 * s
    else:
        x0, x1 = x.float()[..., :r // 2], x.float()[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = x0 * c - x1 * s, x1 * c + x0 * s
    return y.to(torch.bfloat16)


def attend(q, k, v, scale, last):
    """float64 attention on q's device: q [rows][g][d], k, v [T][d]; row i
    attends positions 0 .. last[i].  Returns (out [rows][g][d], A, B): A the
    largest sum_c |q_c k_c| and B the largest max|q| sum_c |k_c| of any pair, in
    the log2 domain (what score errors scale with)."""
    rows, g, d = q.shape
    if k.shape[0] == 0:
        return torch.zeros_like(q, dtype=torch.float64), 0.0, 0.0
    x, k, v = q.double().reshape(-1, d), k.double(), v.double()
    s = x @ k.T * scale
    hide = torch.arange(k.shape[0], device=q.device) > last.to(q.device).repeat_interleave(g)[:, None]
    s = s.masked_fill(hide, -math.inf)
    p = torch.softmax(s, -1).nan_to_num(0.0)
    l2e = scale * math.log2(math.e)
    A = float((x.abs() @ k.abs().T).max()) * l2e
    Bq = float(x.abs().max() * k.abs().sum(1).max()) * l2e
    return (p @ v).view(rows, g, d), A, Bq


def tolerance(d, T, vmax, A, bq=None, out=torch.float32, ref=0.0):
    """Largest |error| the kernels' roundings can make, by their definition.
    The weights are rounded to f16 for the second product: 2^-11 relative
    (2^-25 absolute under 2^-14, of a largest weight >= 1 that the sum holds);
    a score's fp32 sum of d products and the few roundings behind it move it
    by (d + 8) 2^-24 A in the log2 domain, and the weights, above and below
    the fraction, by ln 2 times that each; 2^-20 covers the exponentials and
    the joins.  With bq (the prefill): q is held in two E4M3 parts, off by at
    most 2^-18 of the row's largest value, and a weight may be rounded twice.
    A bf16 output adds half a step, 2^-8 of the value."""
    score = (d + 8) * 2.0 ** -24 * A + (2.0 ** -18 * bq if bq is not None else 0.0)
    w = 2.0 ** -11 * (1 if bq is None else 2)
    tol = vmax * (w + T * 2.0 ** -25 + 2 * math.log(2) * score + 2.0 ** -20)
    return tol + (2.0 ** -8 * (ref + tol) if out == torch.bfloat16 else 0.0)
