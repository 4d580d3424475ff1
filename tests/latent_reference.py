"""Plain references of the latent cache and of attention over it, in float64
(torch, on the tensors' device), written from the definitions in
include/kvq_latent.h.  Nothing here uses the CUDA library.

Bounds count the roundings of the attention kernels, row by row.
  latent (attn_bound)
    weights  x = weight * value scale over a power of two, the row's largest x between
             2^3 and 2^11, rounded to f16 (2^-11 relative), then held as an E4M3 and an
             E5M2 value, one the rounding of x, the other of the rest: off by half a step of
             the rest's rounding, 2^-8 of x (of x in [1, 2) the rest behind E4M3 is at most
             2^-4 and E5M2's half step there 2^-8; behind E5M2, over 448, 2^-3 and 2^-8),
             or 2^-14 where x is under 2^-6 (E4M3's steps end at 2^-9), which is 2^-17 of
             the row's largest.  It reaches the result times the value's code.
    scores   q is scaled to 2^7 .. 2^8 and held in two E4M3 parts: off by at most
             2^-17 of the row's largest element; (w + 8) half steps of fp32 of the
             sum of |q_c k_c| for w products, which counts twice (numerator and
             denominator), times ln 2 in the log2 domain.
    sums     one half step of fp32 for each of the T / 16 products' sums, 2^-20
             for exponentials and joins.
  expanded (dense_bound)
    weights  bf16: 2^-8 of a weight.  q, k and v enter as they are; scores and sums
             as above, without q's parts.
A bf16 output adds half a step, 2^-8 of the value.
"""
from __future__ import annotations

import math

import torch

LOG2E = math.log2(math.e)
E4M3_MAX = 448.0


def power(e: torch.Tensor) -> torch.Tensor:
    """2^e in float64, of whole e from -1022 (from the bits: ldexp takes a float32 power)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def e4m3_round(x: torch.Tensor) -> torch.Tensor:
    """Nearest E4M3 value of float64 x, ties to even, saturating at 448."""
    a = x.abs().clamp(max=E4M3_MAX)
    _, e = torch.frexp(torch.where(a > 0, a, torch.ones_like(a)))
    step = power((e - 1).clamp(min=-6) - 3)
    return torch.copysign(torch.round(a / step) * step, x).clamp(-E4M3_MAX, E4M3_MAX)


def token_scale(amax: torch.Tensor) -> torch.Tensor:
    """The smallest power of two s >= 2^-126 with amax <= 448 s (float64)."""
    e = torch.full(amax.shape, -126, dtype=torch.int64, device=amax.device)
    for _ in range(256):
        e = torch.where(amax > E4M3_MAX * power(e), e + 1, e)
    return power(e)


def encode(c: torch.Tensor, k: torch.Tensor):
    """bf16 latents [..., L] and rotated key parts [..., R] -> (code values float64
    [..., L + 2 R], exponent bytes [...])."""
    x, y = c.double(), k.double()
    amax = torch.maximum(x.abs().amax(-1), y.abs().amax(-1))
    bad = ~torch.isfinite(x).all(-1) | ~torch.isfinite(y).all(-1)
    s = token_scale(torch.where(bad, torch.zeros_like(amax), amax))
    hi = e4m3_round(y / s[..., None])
    codes = torch.cat([e4m3_round(x / s[..., None]), hi, e4m3_round(y / s[..., None] - hi)], -1)
    codes = torch.where(bad[..., None], torch.zeros_like(codes), codes)
    e = torch.frexp(s)[1] - 1 + 127
    return codes, torch.where(bad, torch.full_like(e, 255), e)


def decode(codes: torch.Tensor, e: torch.Tensor, L: int):
    """(latents, key parts) of code values and exponent bytes, float64."""
    R = (codes.shape[-1] - L) // 2
    s = torch.where(e == 255, torch.full(e.shape, float("nan"), dtype=torch.float64, device=e.device),
                    power(e.long() - 127))[..., None]
    return codes[..., :L] * s, (codes[..., L:L + R] + codes[..., L + R:]) * s


def read_pool(pool, page_table, max_pages, b, n, page, L, R):
    """(code values float64 [n][L + 2 R], exponent bytes [n]) of positions 0 .. n - 1
    of sequence b, by byte arithmetic."""
    G, row = min(page, 64), L + 2 * R
    t = torch.arange(n, device=pool.device)
    phys = (b * max_pages + t // page) if page_table is None else page_table[b].long()[t // page]
    block = pool[phys, (t % page) // G]
    lt, c = (t % G)[:, None], torch.arange(row, device=pool.device)[None]
    off = (lt // 8) * (8 * row) + (c // 16) * 128 + (lt % 8) * 16 + c % 16
    codes = block.gather(1, off).view(torch.float8_e4m3fn).double()
    return codes, block.gather(1, G * row + lt)[:, 0].long()


def rotate32(x: torch.Tensor, start, table: torch.Tensor, interleaved: bool) -> torch.Tensor:
    """bf16 [B][n][..., R], every product and sum rounded to fp32, the result to bf16."""
    r = table.shape[1]
    pos = torch.as_tensor(start).long().to(table.device)[:, None] + torch.arange(x.shape[1], device=table.device)
    cs = table[pos]
    cs = cs[:, :, None] if x.dim() == 4 else cs
    c, s = cs[..., :r // 2], cs[..., r // 2:]
    f = x.float()
    y = f.clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[..., a] = f[..., a] * c - f[..., b] * s
    y[..., b] = f[..., b] * c + f[..., a] * s
    return y.to(torch.bfloat16)


def weights(q, k, scale, last):
    """float64 softmax weights [rows][T]; q [rows][w], k [T][w], row i attends 0 .. last[i]."""
    s = q.double() @ k.double().T * scale
    hide = torch.arange(k.shape[0], device=q.device) > last.to(q.device)[:, None]
    return torch.softmax(s.masked_fill(hide, -math.inf), -1).nan_to_num(0.0)


def _scores_off(q, k, seen, scale, parts):
    x, kk = q.double().abs(), k.double().abs()
    w = k.shape[1]
    off = (w + 8) * 2.0 ** -24 * ((x @ kk.T) * seen).amax(-1)
    if parts:
        off = off + 2.0 ** -17 * x.amax(-1) * (kk.sum(1) * seen).amax(-1)
    return off * scale * LOG2E


def _finish(e, out, ref):
    return e + 2.0 ** -8 * (ref.abs() + e) if out == torch.bfloat16 else e


def attn_bound(q, c, k, s, p, scale, out=torch.float32, ref=None):
    """Largest |error| [rows][L] of the latent attention: q [rows][L + R], c and k the
    tokens' values, s [T] their scales, p [rows][T] the weights."""
    T = c.shape[0]
    seen = p > 0
    score = _scores_off(q, torch.cat([c, k], -1), seen, scale, True)
    prod = p * s
    top = prod.amax(-1, keepdim=True)
    total = p @ c.abs()
    e = total * (2.0 ** -8 + 2.0 ** -11 + (2 * math.log(2) * score + T / 16 * 2.0 ** -24 + 2.0 ** -20)[..., None])
    small = seen & (prod < 2.0 ** -9 * top)
    e = e + 2.0 ** -17 * top * (small.double() @ (c.abs() / s[:, None]))
    return _finish(e, out, ref)


def dense_bound(q, k, v, p, scale, out=torch.float32, ref=None):
    T = k.shape[0]
    score = _scores_off(q, k, p > 0, scale, False)
    e = (p @ v.double().abs()) * (2.0 ** -8 + (2 * math.log(2) * score + T / 16 * 2.0 ** -24 + 2.0 ** -20)[..., None])
    return _finish(e, out, ref)
