"""Measured cases of the latent-attention operators: keys and values of a token come from one latent vector that
all heads share, and a rotated key part beside it.

``append``    rotates the queries' and the key's position part and writes latent and key part to a paged 8-bit cache
``decode``    attention of one token per sequence over that cache, queries and results in the latent space (absorbed)
``chunk``     the same for a chunk of new tokens, causal
``step``      append and decode of one token, as a serving loop runs them
``read``      the cache read back as dense rows (what the expanded form multiplies out)
``expanded``  attention of a chunk over keys and values multiplied out per head, the key's position part shared

``own`` selects who computes: False is the plain form (elementary torch operations in fp32, rounded once at the
end), True the framework's calls.

The pool is uint8 [pages][page / G][bytes], G = min(page, 64) tokens: their codes [G/8][row/16][8][16], row = latent
+ 2 rope bytes, then one exponent byte per token [G].  A token's row is E4M3(latent / s), hi = E4M3(key / s) and lo =
E4M3(key / s - hi) with s = 2^(exponent - 127), the smallest power of two with max|latent, key| <= 448 s.
"""
from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0


def _cache_case(name, op, batch, heads, latent, rope, page, lo, hi, n=1, ragged=False, interleaved=False):
    """lo..hi: cached positions (of append and step: the positions before the new ones); n: new tokens."""
    return {"name": name, "op": op, "batch": batch, "heads": heads, "latent": latent, "rope": rope, "page": page,
            "lo": lo, "hi": hi, "n": n, "ragged": ragged, "interleaved": interleaved}


def _expanded_case(name, batch, heads, d, lo, hi, n, ragged=False, packed=True):
    return {"name": name, "op": "expanded", "batch": batch, "heads": heads, "d": d, "rope": 64, "lo": lo, "hi": hi,
            "n": n, "ragged": ragged, "packed": packed}


def listed():
    return [
        # the new token of every running sequence of a decode batch
        _cache_case("append_step", "append", 64, 16, 512, 64, 64, 1000, 4000),
        # a padded batch of odd prompts, the position part in adjacent pairs
        _cache_case("append_prompt", "append", 12, 16, 512, 64, 64, 0, 300, n=3001, ragged=True, interleaved=True),
        # one short sequence, a small latent: latency
        _cache_case("decode_tiny", "decode", 1, 4, 128, 32, 64, 256, 256),
        # one GPU's share of the heads over a large batch: the cache is streamed
        _cache_case("decode_batch", "decode", 64, 16, 512, 64, 64, 8192, 8192),
        # all heads of a large layer over long contexts: bound by the products
        _cache_case("decode_long", "decode", 16, 128, 512, 64, 128, 32768, 32768),
        # ragged lengths over small pages, an odd number of heads
        _cache_case("decode_ragged", "decode", 24, 40, 512, 64, 16, 1, 20001),
        # a prompt's chunk over what is cached already
        _cache_case("chunk_prompt", "chunk", 2, 64, 512, 64, 64, 8192, 8192, n=1024),
        # a few drafted tokens over ragged contexts, as a padded batch
        _cache_case("chunk_draft", "chunk", 6, 20, 256, 64, 32, 3000, 9001, n=5, ragged=True),
        # cached prefixes read back to be multiplied out
        _cache_case("read_prefix", "read", 8, 1, 512, 64, 64, 8192, 8192),
        # short ragged prefixes on small pages
        _cache_case("read_ragged", "read", 5, 1, 256, 32, 16, 1, 1501),
        # whole prompts, keys and values straight from the packed up-projection
        _expanded_case("expanded_prompt", 2, 32, 128, 4096, 4096, 4096),
        # odd chunks of a padded batch behind cached prefixes, small heads
        _expanded_case("expanded_ragged", 3, 12, 64, 700, 2900, 515, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "step", "decode", "decode", "chunk", "chunk", "read", "expanded", "expanded"])
    batch = _log_int(rng, 1, 64)
    if kind == "expanded":
        heads = rng.choice([1, 2, 3, 5, 8, 12, 16, 32])
        hi = _log_int(rng, 1, 4200)
        n = _log_int(rng, 1, hi)
        batch = max(1, min(batch, 6, 300_000_000 // (heads * n * hi)))
        c = _expanded_case("", batch, heads, rng.choice([64, 128]), rng.randint(n, hi), hi, n,
                           ragged=n > 1 and rng.random() < 0.5, packed=rng.random() < 0.5)
        del c["name"]
        return c
    heads = rng.choice([1, 2, 3, 7, 8, 12, 16, 16, 20, 32, 40, 64, 128])
    latent, rope = rng.choice([128, 256, 512, 512]), rng.choice([32, 64, 64])
    page = rng.choice([16, 32, 64, 128, 256])
    n, ragged = 1, False
    if kind == "append":
        n, hi = _log_int(rng, 1, 4096), _log_int(rng, 1, 4000)
        batch = max(1, min(batch, 16000 // n))
        lo = rng.randint(0, hi)
    elif kind == "chunk":
        hi = _log_int(rng, 1, 16000)
        n = _log_int(rng, 1, min(1200, hi))
        batch = max(1, min(batch, 16, 800_000_000 // (heads * n * hi)))
        lo = rng.randint(n, hi)
    else:
        hi = _log_int(rng, 1, 30000)
        batch = max(1, min(batch, (65_536 if kind == "read" else 500_000) // hi))
        lo = rng.randint(1, hi)
    if n > 1:
        ragged = rng.random() < 0.5
    c = _cache_case("", kind, batch, heads, latent, rope, page, lo, hi, n, ragged, rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _scale_exponent(amax):
    """The exponent byte of each token: 127 + the smallest e in -126..120 with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-126, 120)
    return torch.where(amax > 0, e, torch.full_like(e, -126)) + 127


def _power(e):
    """2^(e - 127) in fp32 of exponent bytes."""
    return torch.ldexp(torch.ones(e.shape, device=e.device), e.int() - 127)


def _encode(c, k):
    """Rows of codes uint8 [..., latent + 2 rope] and exponent bytes [...] of latents and key parts (fp32)."""
    e = _scale_exponent(torch.maximum(c.abs().amax(-1), k.abs().amax(-1)))
    s = _power(e)[..., None]
    y = k / s
    hi = y.to(torch.float8_e4m3fn)
    lo = (y - hi.float()).to(torch.float8_e4m3fn)
    row = torch.cat([x.view(torch.uint8) for x in ((c / s).to(torch.float8_e4m3fn), hi, lo)], dim=-1)
    return row, e.to(torch.uint8)


def _token_rows(part, g, row):
    """Codes of groups in the pool's order, [..., g * row], as [..., g, row]."""
    lead = part.shape[:-1]
    return part.reshape(*lead, g // 8, row // 16, 8, 16).transpose(-3, -2).reshape(*lead, g, row)


def _pool_order(rows):
    *lead, g, row = rows.shape
    return rows.reshape(*lead, g // 8, 8, row // 16, 16).transpose(-3, -2).reshape(*lead, g * row)


def _latents(shape, gen):
    """Latents with a few larger channels and tokens of differing magnitude."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp(0.3 * torch.randn(shape[:-1], generator=gen, device="cuda"))[..., None]
    x[..., [1, 9, shape[-1] // 2, shape[-1] - 3]] *= 5.0
    return x


def _random_pool(pages, page, latent, rope, gen):
    g, row = min(page, 64), latent + 2 * rope
    pool = torch.zeros((pages, page // g, g * (row + 1)), dtype=torch.uint8, device="cuda")
    per = max(1, (1 << 25) // (page * row))
    for p0 in range(0, pages, per):
        part = pool[p0:p0 + per]
        c = _latents((part.shape[0], page // g, g, latent), gen).to(torch.bfloat16).float()
        k = (2.0 * torch.randn((part.shape[0], page // g, g, rope), generator=gen, device="cuda")).to(torch.bfloat16)
        codes, e = _encode(c, k.float())
        part[..., :g * row], part[..., g * row:] = _pool_order(codes), e
    return pool


def _paging(rows, page, gen, most):
    """A page table over a shuffled pool for `most` positions a sequence: rows[b] positions, -1 behind them."""
    pages = -(-most // page)
    table = torch.full((len(rows), pages), -1, dtype=torch.int32)
    perm = torch.randperm(len(rows) * pages, generator=gen).to(torch.int32)
    at = 0
    for b, r in enumerate(rows):
        m = -(-r // page)
        table[b, :m] = perm[at:at + m]
        at += m
    return table.cuda(), len(rows) * pages


def _lens(case, gen):
    if case["lo"] == case["hi"]:
        return [case["hi"]] * case["batch"]
    lens = torch.randint(case["lo"], case["hi"] + 1, (case["batch"],), generator=gen).tolist()
    lens[0] = case["hi"]
    return lens


def _new_lens(case, gen, least):
    if not case["ragged"]:
        return None
    n = torch.randint(least, case["n"] + 1, (case["batch"],), generator=gen).to(torch.int32)
    n[0] = case["n"]
    return n.cuda()


def _randn(shape, gen, scale=1.0):
    return (scale * torch.randn(shape, generator=gen, device="cuda")).to(torch.bfloat16)


def prepare(case, seed):
    dev = torch.Generator(device="cuda")
    dev.manual_seed(seed * 7919 + 5)
    cpu = torch.Generator()
    cpu.manual_seed(seed * 104729 + 11)
    b, h, n, r = case["batch"], case["heads"], case["n"], case["rope"]
    st = dict(case)
    lens = _lens(case, cpu)
    if case["op"] == "expanded":
        d, t = case["d"], max(lens)
        st["q"] = _randn((b, n, h, d + r), dev)
        kv = _randn((b, t, h, 2 * d), dev)
        st["k"], st["v"] = (x if case["packed"] else x.contiguous() for x in (kv[..., :d], kv[..., d:]))
        st["k_rope"] = _randn((b, t, r), dev)
        st["lens"], st["max_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda"), t
        st["new_lens"] = _new_lens(case, cpu, 1)
        st["scale"] = 1.0 / math.sqrt(d + r)
        st["out"] = torch.zeros((b, n, h, d), dtype=torch.bfloat16, device="cuda")
        return st
    latent, page = case["latent"], case["page"]
    # the scale of heads of 128 channels and the position part: the latent does not show in it
    st["scale"] = 1.0 / math.sqrt(128 + r)
    new = n if case["op"] in ("append", "step") else 0
    table, st["pages"] = _paging([x + new for x in lens], page, cpu, case["hi"] + new)
    st["page_table"] = table
    st["pool"] = _random_pool(st["pages"], page, latent, r, dev)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["max_len"] = max(lens) + new
    g, row = min(page, 64), latent + 2 * r
    st["group"], st["row"] = g, row
    st["codes"] = st["pool"][..., :g * row].view(torch.float8_e4m3fn)
    st["exponents"] = st["pool"][..., g * row:]
    if case["op"] == "read":
        return st
    # absorbed queries: the latent part comes from a product with the up-projection, the position part stands behind it
    st["q"] = _randn((b, n, h, latent + r), dev, 0.5)
    st["new_lens"] = _new_lens(case, cpu, 0 if new else 1)
    if new:
        st["q_rope"] = _randn((b, n, h, 128 + r), dev)[..., 128:]             # a part of the query projection
        x = torch.cat([_latents((b, n, latent), dev), 2.0 * torch.randn((b, n, r), generator=dev, device="cuda")], -1)
        st["down"] = x.to(torch.bfloat16)                                      # the packed down-projection
        pos = torch.arange(st["max_len"] + 1, dtype=torch.float64, device="cuda")
        inv = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
        ang = pos[:, None] * inv[None, :]
        st["table"] = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
        st["lens_after"] = st["lens"] + n
    if case["op"] != "append":
        shape = (b, n, h, latent) if case["op"] == "chunk" else (b, h, latent)
        st["out"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------------ the framework's calls
def _cache(st):
    """The cache object and workspace that a program keeps, made on the first pass."""
    if "cache" not in st:
        from fp4_kv_cache_kvq_gb300 import kvq
        st["kvq"] = kvq
        st["cache"] = kvq.LatentCache(st["latent"], st["rope"], st["page"], st["pages"], st["page_table"].shape[1],
                                      page_table=st["page_table"], pool=st["pool"])
        nbytes = kvq.latent_workspace_bytes(st["batch"], st["heads"], st["latent"], st["n"])
        st["workspace"] = torch.empty(max(16, nbytes), dtype=torch.uint8, device="cuda")
    return st["cache"], st["kvq"]


def _append_own(st, cache, kvq):
    latent = st["latent"]
    kvq.latent_append(cache, st["lens"], st["q_rope"], st["down"][..., :latent], st["down"][..., latent:], st["table"],
                      interleaved=st["interleaved"], new_lens=st["new_lens"], q_out=st["q"][..., latent:])
    return {"q": st["q"][..., latent:], "codes": st["codes"], "exponents": st["exponents"]}


def _run_own(st):
    if st["op"] == "expanded":
        from fp4_kv_cache_kvq_gb300 import kvq
        return kvq.expanded_attn(st["q"], st["k"], st["k_rope"], st["v"], st["lens"], st["scale"], out=st["out"],
                                 chunk_lens=st["new_lens"])
    cache, kvq = _cache(st)
    if st["op"] == "append":
        return _append_own(st, cache, kvq)
    if st["op"] == "step":
        res = _append_own(st, cache, kvq)
        res["out"] = kvq.decode_attn(cache, st["lens_after"], st["q"][:, 0], st["scale"], out=st["out"],
                                     workspace=st["workspace"])
        return res
    if st["op"] == "decode":
        return kvq.decode_attn(cache, st["lens"], st["q"][:, 0], st["scale"], out=st["out"], workspace=st["workspace"])
    if st["op"] == "chunk":
        return kvq.prefill_attn(cache, st["lens"], st["q"], st["scale"], out=st["out"], chunk_lens=st["new_lens"],
                                workspace=st["workspace"])
    return kvq.dequant(cache, st["lens"], st["max_len"], dtype=torch.bfloat16)


# ------------------------------------------------------------------ the plain form
def _rotate(x, st):
    """bf16 [b][n][..., rope] rotated by the table's rows lens + t, in fp32, rounded to bf16."""
    r = st["rope"]
    pos = st["lens"].long()[:, None] + torch.arange(x.shape[1], device=x.device)
    cs = st["table"][pos]
    if x.dim() == 4:
        cs = cs[:, :, None]
    c, s = cs[..., :r // 2], cs[..., r // 2:]
    x = x.float()
    if st["interleaved"]:
        x0, x1 = x[..., 0::2], x[..., 1::2]
        y = torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], dim=-1).flatten(-2)
    else:
        x0, x1 = x[..., :r // 2], x[..., r // 2:]
        y = torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], dim=-1)
    return y.to(torch.bfloat16)


def _valid(st):
    t = torch.arange(st["n"], device="cuda")
    if st["new_lens"] is None:
        return torch.ones((st["batch"], st["n"]), dtype=torch.bool, device="cuda")
    return t[None] < st["new_lens"][:, None]


def _append_plain(st):
    latent, page, g = st["latent"], st["page"], st["group"]
    ok = _valid(st)
    q_out = st["q"][..., latent:]
    q_out.copy_(torch.where(ok[..., None, None], _rotate(st["q_rope"], st), q_out))
    k = _rotate(st["down"][..., latent:], st)
    rows, e = _encode(st["down"][..., :latent].float(), k.float())
    seq, t = ok.nonzero(as_tuple=True)
    pos = st["lens"].long()[seq] + t
    phys, grp, slot = st["page_table"].long()[seq, pos // page], (pos % page) // g, pos % g
    whole = st["pool"][..., :g * st["row"]].view(st["pages"], page // g, g // 8, st["row"] // 16, 8, 16)
    whole[phys, grp, slot // 8, :, slot % 8] = rows[seq, t].view(-1, st["row"] // 16, 16)
    st["exponents"][phys, grp, slot] = e[seq, t]
    return {"q": q_out, "codes": st["codes"], "exponents": st["exponents"]}


def _dense(st, max_len):
    """Latents [b][positions][latent] and key parts [b][positions][rope] in fp32."""
    b, latent, g, row, r = st["batch"], st["latent"], st["group"], st["row"], st["rope"]
    idx = st["page_table"][:, :-(-max_len // st["page"])].long().clamp(min=0)
    raw = st["pool"][idx]                                                        # [b][pages][groups][bytes]
    codes = _token_rows(raw[..., :g * row], g, row).reshape(b, -1, row)[:, :max_len]
    s = _power(raw[..., g * row:].reshape(b, -1)[:, :max_len])[..., None]
    x = codes.contiguous().view(torch.float8_e4m3fn).float()
    return x[..., :latent] * s, (x[..., latent:latent + r] + x[..., latent + r:]) * s


def _softmax_product(s, last, v):
    """Scores s [b][rows][positions], row i attending 0 .. last[b][i] (none if < 0), times v [b][positions][d]."""
    t = torch.arange(s.shape[-1], device=s.device)
    s.masked_fill_(t > last[..., None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / l.clamp(min=1e-30)


def _attend(st, q, last, max_len):
    """q bf16 [b][n][h][latent + rope] over the cache; token i of sequence b attends 0 .. last[b][i]."""
    b, n, h, w = q.shape
    c, k = _dense(st, max_len)
    s = torch.matmul(q.reshape(b, n * h, w).float(), torch.cat([c, k], -1).transpose(-1, -2)).mul_(st["scale"])
    o = _softmax_product(s, last.repeat_interleave(h, 1), c)
    return o.view(b, n, h, -1).to(torch.bfloat16)


def _last(st):
    """Last position that token i of each sequence attends, [b][n]."""
    n = st["new_lens"].long() if st["new_lens"] is not None else torch.full_like(st["lens"], st["n"]).long()
    return (st["lens"].long() - n)[:, None] + torch.arange(st["n"], device="cuda")


def _run_plain(st):
    op = st["op"]
    if op == "append":
        return _append_plain(st)
    if op == "step":
        res = _append_plain(st)
        res["out"] = _attend(st, st["q"], st["lens_after"].long()[:, None] - 1, st["max_len"])[:, 0]
        return res
    if op == "decode":
        return _attend(st, st["q"], st["lens"].long()[:, None] - 1, st["max_len"])[:, 0]
    if op == "chunk":
        o = _attend(st, st["q"], _last(st), st["max_len"])
        return torch.where(_valid(st)[..., None, None], o, st["out"])
    if op == "read":
        keep = (torch.arange(st["max_len"], device="cuda") < st["lens"][:, None])[..., None]
        return tuple(torch.where(keep, x, 0.0).to(torch.bfloat16) for x in _dense(st, st["max_len"]))
    b, n, h, d = st["out"].shape
    k = torch.cat([st["k"].float(), st["k_rope"].float()[:, :, None].expand(-1, -1, h, -1)], -1)
    s = torch.matmul(st["q"].float().transpose(1, 2), k.permute(0, 2, 3, 1)).mul_(st["scale"])
    o = _softmax_product(s, _last(st)[:, None], st["v"].float().transpose(1, 2))
    return torch.where(_valid(st)[..., None, None], o.transpose(1, 2).to(torch.bfloat16), st["out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    b, h, r = case["batch"], case["heads"], case["rope"]
    n = 0.5 * (case["n"] + 1) if case["ragged"] else case["n"]
    mean = 0.5 * (case["lo"] + case["hi"])
    if case["op"] == "expanded":
        d = case["d"]
        nbytes = 2.0 * b * (n * h * (2 * d + r) + mean * (2 * h * d + r))
        return {"bytes": nbytes, "flops": 2.0 * b * h * (2 * d + r) * n * (mean - 0.5 * (n - 1))}
    latent = case["latent"]
    token = latent + 2 * r + 1
    new = b * n
    append = new * (2 * (latent + r) + token + 4 * h * r) + (case["n"] + min(b, case["hi"] + 1)) * r * 4
    append_flops = new * (h + 1) * r * 3
    if case["op"] == "append":
        return {"bytes": append, "flops": append_flops}
    if case["op"] == "read":
        return {"bytes": b * (mean * token + case["hi"] * 2 * (latent + r)), "flops": b * mean * (latent + 2 * r)}
    if case["op"] == "step":
        mean += 1
    nbytes = b * (mean * token + n * h * 2 * (2 * latent + r))
    flops = 2.0 * b * h * (2 * latent + r) * n * (mean - 0.5 * (n - 1))
    if case["op"] == "step":
        return {"bytes": nbytes + append - new * h * r * 2, "flops": flops + append_flops}
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3(x):
    """x (float64, |x| <= 448) to the nearest E4M3 value, ties to the even code."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.round(x / step) * step


def _exact_rotate(x, st):
    r = st["rope"]
    i = torch.arange(r // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if st["interleaved"] else (i, i + r // 2)
    out = x.double().clone()
    for j in range(x.shape[0]):
        at = int(st["lens"][j])
        cs = st["table"][at:at + x.shape[1]].double()
        cs = cs[:, None] if x.dim() == 4 else cs
        z = torch.complex(out[j][..., first], out[j][..., second])
        z = z * torch.complex(cs[..., :r // 2].contiguous(), cs[..., r // 2:].contiguous())
        out[j][..., first], out[j][..., second] = z.real, z.imag
    return out.to(torch.bfloat16).double()


def _places(st, b, pos):
    """Pages, groups and byte offsets [tokens][row] of positions of sequence b."""
    g, row, page = st["group"], st["row"], st["page"]
    phys = st["page_table"][b].long()[pos // page]
    t, c = (pos % g)[:, None], torch.arange(row, device="cuda")[None]
    return phys, (pos % page) // g, (t // 8) * (8 * row) + (c // 16) * 128 + (t % 8) * 16 + c % 16


def _exact_append(st):
    latent, r = st["latent"], st["rope"]
    codes, exps = st["codes"].double(), st["exponents"].clone()
    q = _exact_rotate(st["q_rope"], st)
    key = _exact_rotate(st["down"][..., latent:], st)
    ok = _valid(st)
    for b in range(st["batch"]):
        m = int(ok[b].sum())
        if not m:
            continue
        c, k = st["down"][b, :m, :latent].double(), key[b, :m]
        amax = torch.cat([c, k], -1).abs().amax(-1)
        e = torch.ceil(torch.log2((amax / E4M3_MAX).clamp(min=2.0 ** -140)))
        e = torch.where(amax <= E4M3_MAX * torch.exp2(e - 1.0), e - 1.0, e).clamp(-126, 120)  # log2 may be off at a power
        s = torch.exp2(e)[:, None]
        hi = _e4m3(k / s)
        pos = int(st["lens"][b]) + torch.arange(m, device="cuda")
        phys, grp, at = _places(st, b, pos)
        codes[phys[:, None], grp[:, None], at] = torch.cat([_e4m3(c / s), hi, _e4m3(k / s - hi)], -1)
        exps[phys, grp, pos % st["group"]] = (e + 127).to(torch.uint8)
    q = torch.where(ok[..., None, None], q, st["q"][..., latent:].double())
    return {"q": q, "codes": codes, "exponents": exps}


def _exact_rows(st, b, n):
    """float64 latents [n][latent] and key parts [n][rope] of sequence b."""
    latent, r = st["latent"], st["rope"]
    pos = torch.arange(n, device="cuda")
    phys, grp, at = _places(st, b, pos)
    x = st["codes"][phys, grp].view(torch.uint8).gather(1, at).view(torch.float8_e4m3fn).double()
    x = x * torch.exp2(st["exponents"][phys, grp, pos % st["group"]].double() - 127.0)[:, None]
    return x[:, :latent], x[:, latent:latent + r] + x[:, latent + r:]


def _exact_softmax(s, last):
    s[torch.arange(s.shape[-1], device="cuda") > last[:, None]] = -math.inf
    return torch.softmax(s, -1)


def _exact_attend(st, q, last, lens):
    """float64 attention, one sequence at a time and rows by blocks; q bf16 [b][n][h][w], last [b][n]."""
    b, n, h, w = q.shape
    out = torch.zeros((b, n, h, st["latent"]), dtype=torch.float64, device="cuda")
    for j in range(b):
        c, k = _exact_rows(st, j, int(lens[j]))
        ck = torch.cat([c, k], -1).T.contiguous()
        per = max(1, (1 << 28) // (h * ck.shape[1]))
        for i in range(0, n, per):
            x = q[j, i:i + per].double().reshape(-1, w)
            p = _exact_softmax(x @ ck * st["scale"], last[j, i:i + per].clamp(0, int(lens[j]) - 1).repeat_interleave(h))
            out[j, i:i + per] = (p @ c).view(-1, h, st["latent"])
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(st)
    if op == "step":
        res = _exact_append(st)
        st["codes"].copy_(res["codes"].to(torch.float8_e4m3fn))
        st["exponents"].copy_(res["exponents"])
        q = torch.cat([st["q"][..., :case["latent"]], res["q"].to(torch.bfloat16)], -1)
        last = st["lens_after"].long()[:, None] - 1
        res["out"] = _exact_attend(st, q, last, st["lens_after"])[:, 0]
        return res
    if op == "decode":
        return _exact_attend(st, st["q"], st["lens"].long()[:, None] - 1, st["lens"])[:, 0]
    if op == "chunk":
        o = _exact_attend(st, st["q"], _last(st), st["lens"])
        return torch.where(_valid(st)[..., None, None], o, 0.0)
    if op == "read":
        outs = [torch.zeros((case["batch"], st["max_len"], w), dtype=torch.float64, device="cuda")
                for w in (case["latent"], case["rope"])]
        for b in range(case["batch"]):
            n = int(st["lens"][b])
            for o, x in zip(outs, _exact_rows(st, b, n)):
                o[b, :n] = x
        return tuple(outs)
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    last = _last(st)
    for b in range(case["batch"]):
        t = int(st["lens"][b])
        for h in range(case["heads"]):
            q, kr = st["q"][b, :, h].double(), st["k_rope"][b, :t].double()
            s = q[:, :case["d"]] @ st["k"][b, :t, h].double().T + q[:, case["d"]:] @ kr.T
            out[b, :, h] = _exact_softmax(s * st["scale"], last[b].clamp(0, t - 1)) @ st["v"][b, :t, h].double()
    return torch.where(_valid(st)[..., None, None], out, 0.0)
