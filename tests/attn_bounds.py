"""Attention in float64 with an error bound of each row's own.

The bound counts the roundings of the 8-bit block cache's attention against
what the row sums up, not against the largest value of the cache:
  weights   f16, half a step: 2^-11 of a weight, or 2^-25 of the reference where
            that is more (weights under 2^-14 of it).  The decode's reference is
            at most the row's largest weight.  The prefill rounds weight * value
            scale against a power of two that is at most twice the largest such
            product that the row attends; what a product loses reaches the result
            times the value's code, |v| over the scale.
  scores    (d + 8) half steps of fp32 of sum |q_c k_c|, in the log2 domain; the
            prefill holds q in two E4M3 parts, off by at most 2^-17 of the
            row's largest element (scaled to 2^7 .. 2^8, half of a smallest step
            of 2^-9), the decode in f16, 2^-39 (2^14 .. 2^15, 2^-24).  A score
            off by e changes numerator and denominator by ln 2 * e each.
  sums      one half step of fp32 for each of the T / 16 products' sums, and
            2^-20 for the exponentials and the joins.
"""
from __future__ import annotations

import math

import torch

LOG2E = math.log2(math.e)


def attend(q, k, v, scale, last):
    """q [rows][g][d], k, v [T][d] (any float type, one device); row i attends
    positions 0 .. last[i].  (out [rows][g][d], p [rows][g][T]) in float64."""
    rows, g, d = q.shape
    s = torch.einsum("rgd,td->rgt", q.double(), k.double()) * scale
    hide = torch.arange(k.shape[0], device=q.device) > last.to(q.device)[:, None]
    p = torch.softmax(s.masked_fill(hide[:, None], -math.inf), -1).nan_to_num(0.0)
    return torch.einsum("rgt,td->rgd", p, v.double()), p


def bound(q, k, v, p, scale, v_scale=None, out=torch.float32, ref=None, v_rel=0.0, v_least=None):
    """Largest |error| of each output element [rows][g][d]; v_scale [T]: the value
    scales, given for the prefill, or the most that they can be (v_least: the least;
    v_scale when not given); v_rel: a relative rounding of its values."""
    d, T = k.shape[1], k.shape[0]
    seen = p > 0
    x, kk, vv = q.double().abs(), k.double().abs(), v.double().abs()
    reach = (torch.einsum("rgd,td->rgt", x, kk) * seen).amax(-1)
    score = (d + 8) * 2.0 ** -24 * scale * LOG2E * reach
    score = score + 2.0 ** (-39 if v_scale is None else -17) * scale * LOG2E * x.amax(-1) * (kk.sum(1) * seen).amax(-1)
    if v_scale is None:
        most, code, top = p, vv, p.amax(-1, keepdim=True)
        least = p
    else:
        v_least = v_scale if v_least is None else v_least
        most, least = p * v_scale.double(), p * v_least.double()
        code = torch.where(v_least[:, None] > 0, vv / v_least.double().clamp(min=2.0 ** -149)[:, None], 0.0)
        top = 2 * most.amax(-1, keepdim=True)
    small = seen & (least < 2.0 ** -14 * top)
    total = torch.einsum("rgt,td->rgd", p, vv)
    e = total * (2.0 ** -11 + v_rel + (2 * math.log(2) * score + T / 16 * 2.0 ** -24 + 2.0 ** -20)[..., None])
    e = e + 2.0 ** -25 * top * torch.einsum("rgt,td->rgd", small.double(), code)
    if out == torch.bfloat16:
        e = e + 2.0 ** -8 * (ref.abs() + e)
    return e
