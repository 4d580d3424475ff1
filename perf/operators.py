"""Measured cases of the serving operators on a paged cache: the append with the
position rotation on the way (``rope_append``) into 8-bit block-scaled, FP4 and
NVFP4 caches, and attention over the 8-bit block-scaled cache, one token per
sequence (``decode``) or a chunk of them (``prefill``); ``step`` is the append
and the decode of one token as a serving loop runs them.

``own`` selects who computes: False is the plain form (elementary torch
operations in fp32, rounded once at the end), True the framework's calls.

The 8-bit pool is uint8 [pages][kv heads][page / G][bytes], G = min(page, 64):
the K codes of G tokens [G/8][d/16][8][16], their V codes [G/16][d][16] with the
16 tokens of a block in the order ``ORDER``, then (K scale, V scale) fp32 pairs
[G/16][2].  A value is E4M3(code) * scale of its 16 tokens and head.
"""
from __future__ import annotations

import math

import torch

own = False

ORDER = [0, 1, 8, 9, 2, 3, 10, 11, 4, 5, 12, 13, 6, 7, 14, 15]  # token of a 16-token block at byte i
E4M3_MAX = 448.0


def _append(name, fmt, batch, n_new, hq, hkv, d, rotary, page, context=0, ragged=False, packed=False,
            interleaved=False, op="rope_append"):
    return {"name": name, "op": op, "format": fmt, "batch": batch, "n_new": n_new, "q_heads": hq, "kv_heads": hkv,
            "d": d, "rotary": rotary, "page": page, "context": context, "ragged": ragged, "packed": packed,
            "interleaved": interleaved}


def _attn(name, op, batch, hq, hkv, d, page, lo, hi, chunk=0, ragged=False):
    return {"name": name, "op": op, "batch": batch, "q_heads": hq, "kv_heads": hkv, "d": d, "page": page, "lo": lo,
            "hi": hi, "chunk": chunk, "ragged": ragged}


def listed():
    return [
        # the new token of every running sequence of a decode batch
        _append("append_step", "fp8", 32, 1, 64, 8, 128, 128, 64, context=2000),
        # prompts of equal length straight from the packed projection
        _append("append_prompt", "fp8", 8, 4096, 64, 8, 128, 128, 64, packed=True),
        # a padded batch of odd prompts behind earlier turns, a quarter of the channels rotated in adjacent pairs
        _append("append_ragged_d64", "fp8", 5, 777, 12, 4, 64, 16, 16, context=300, ragged=True, interleaved=True),
        # prompts into the 4-bit caches
        _append("append_prompt_fp4", "fp4", 2, 2048, 32, 8, 128, 128, 64),
        _append("append_prompt_nvfp4", "nvfp4", 3, 1001, 32, 8, 128, 64, 128, ragged=True),
        # one short sequence, two heads: latency
        _attn("decode_tiny", "decode", 1, 2, 2, 64, 64, 256, 256),
        # a small batch of medium contexts
        _attn("decode_gqa", "decode", 8, 32, 8, 128, 64, 4096, 4096),
        # a large batch of long contexts: the whole cache is streamed
        _attn("decode_long", "decode", 32, 64, 8, 128, 64, 32768, 32768),
        # ragged lengths over small pages, an odd group of query heads
        _attn("decode_ragged", "decode", 24, 15, 5, 128, 16, 1, 20001),
        # a few new tokens (a drafted continuation) over a long context
        _attn("prefill_draft", "prefill", 2, 64, 8, 128, 64, 9001, 12345, chunk=5),
        # a prompt's chunk over what is cached already
        _attn("prefill_chunk", "prefill", 4, 64, 8, 128, 64, 16384, 16384, chunk=1024),
        # a padded batch of odd chunks, head size 64
        _attn("prefill_ragged_d64", "prefill", 3, 32, 8, 64, 32, 700, 2900, chunk=515, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    g = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    kind = rng.choice(["rope_append", "rope_append", "step", "decode", "decode", "prefill", "prefill"])
    batch = _log_int(rng, 1, 64)
    if kind in ("rope_append", "step"):
        fmt = rng.choice(["fp8", "fp8", "fp4", "nvfp4"]) if kind == "rope_append" else "fp8"
        n_new = _log_int(rng, 1, 4096) if kind == "rope_append" else 1
        batch = max(1, min(batch, 16000 // n_new))
        c = _append("", fmt, batch, n_new, g * hkv, hkv, d, rng.choice([16, 32, d // 2, d]), page,
                    context=_log_int(rng, 1, 3000) if fmt == "fp8" else 0,
                    ragged=kind == "rope_append" and rng.random() < 0.5, packed=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, op=kind)
    else:
        hi = _log_int(rng, 1, 30000)
        chunk = _log_int(rng, 1, min(1200, hi)) if kind == "prefill" else 0
        limit = 6_000_000 if kind == "decode" else max(1, 30_000_000 // max(1, chunk))
        batch = max(1, min(batch, limit // (hi * hkv)))
        lo = rng.randint(max(1, chunk), hi)
        c = _attn("", kind, batch, g * hkv, hkv, d, page, lo, hi, chunk=chunk, ragged=chunk > 1 and rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _group(page):
    return min(page, 64)


def _group_bytes(page, d):
    g = _group(page)
    return 2 * g * d + max(16, g // 16 * 8)


def _scale_of(amax):
    """The smallest 2^e with amax <= 448 * 2^e (e >= -126), elementwise on fp32."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-126, 120)
    e = torch.where(amax > 0, e, torch.full_like(e, -126))
    return torch.ldexp(torch.ones_like(amax), e)


def _k_layout(codes):
    """[..., G, d] codes -> [..., G * d] in the pool's order of K."""
    *lead, g, d = codes.shape
    return codes.view(*lead, g // 8, 8, d // 16, 16).transpose(-3, -2).reshape(*lead, g * d)


def _v_layout(codes):
    *lead, g, d = codes.shape
    order = torch.tensor(ORDER, device=codes.device)
    return codes.view(*lead, g // 16, 16, d).index_select(-2, order).transpose(-2, -1).reshape(*lead, g * d)


def _random_pool(pages, hkv, page, d, gen):
    """A pool of quantised tokens: N(0, 1) values, token magnitudes that differ, four larger K channels."""
    g, nbytes = _group(page), _group_bytes(page, d)
    pool = torch.zeros((pages, hkv, page // g, nbytes), dtype=torch.uint8, device="cuda")
    per = max(1, (1 << 26) // (hkv * page * d))
    for p0 in range(0, pages, per):
        part = pool[p0:p0 + per]
        n = part.shape[0]
        for side in range(2):
            x = torch.randn((n, hkv, page // g, g, d), generator=gen, device="cuda")
            x *= torch.exp(0.4 * torch.randn(x.shape[:-1], generator=gen, device="cuda"))[..., None]
            if side == 0:
                x[..., [1, 7, d // 2, d - 3]] *= 8.0
            x = x.view(n, hkv, page // g, g // 16, 16 * d)
            s = _scale_of(x.abs().amax(-1))
            codes = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(n, hkv, page // g, g, d)
            part[..., side * g * d:(side + 1) * g * d] = (_v_layout if side else _k_layout)(codes)
            part[..., 2 * g * d:2 * g * d + g // 2].view(torch.float32)[..., side::2] = s
    return pool


def _paging(batch, rows, page, gen, most):
    """A page table over a shuffled pool of pages for `most` positions a sequence: rows[b] positions, -1 behind them."""
    need = [-(-r // page) for r in rows]
    pages = -(-most // page)
    table = torch.full((batch, pages), -1, dtype=torch.int32)
    perm = torch.randperm(batch * pages, generator=gen).to(torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.cuda(), batch * pages


def _lens(case, gen):
    if case["lo"] == case["hi"]:
        return [case["hi"]] * case["batch"]
    lens = torch.randint(case["lo"], case["hi"] + 1, (case["batch"],), generator=gen).tolist()
    lens[0] = case["hi"]
    return lens


def _pool_views(st):
    g, d = st["group"], st["d"]
    st["codes"] = st["pool"][..., :2 * g * d].view(torch.float8_e4m3fn)
    st["scales"] = st["pool"][..., 2 * g * d:2 * g * d + g // 2].view(torch.float32)


def prepare(case, seed):
    dev = torch.Generator(device="cuda")
    dev.manual_seed(seed * 7919 + 1)
    cpu = torch.Generator()
    cpu.manual_seed(seed * 104729 + 3)
    b, hq, hkv, d, page = case["batch"], case["q_heads"], case["kv_heads"], case["d"], case["page"]
    st = dict(case)
    st["group"] = _group(page)
    st["scale"] = 1.0 / math.sqrt(d)
    if case["op"] in ("rope_append", "step"):
        n, ctx, r = case["n_new"], case["context"], case["rotary"]
        start = [0] * b if ctx == 0 else torch.randint(max(1, ctx // 2), ctx + 1, (b,), generator=cpu).tolist()
        table, pages = _paging(b, [s + n + 16 for s in start], page, cpu, ctx + n + 16)
        st["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        st["new_lens"] = None
        if case["ragged"]:
            lens = torch.randint(0, n + 1, (b,), generator=cpu).to(torch.int32)
            lens[0] = n
            st["new_lens"] = lens.cuda()
        x = torch.randn((b, n, (hq + 2 * hkv) * d), generator=dev, device="cuda")
        x.view(b, n, hq + 2 * hkv, d)[:, :, hq:hq + hkv, [1, d // 2 + 1]] *= 6.0  # keys with two large channels
        x = x.to(torch.bfloat16)
        parts = (x[..., :hq * d], x[..., hq * d:(hq + hkv) * d], x[..., (hq + hkv) * d:])
        st["q"], st["k"], st["v"] = ((p if case["packed"] else p.contiguous()).view(b, n, -1, d) for p in parts)
        pos = torch.arange(ctx + n + 1, dtype=torch.float64, device="cuda")
        inv = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
        ang = pos[:, None] * inv[None, :]
        st["table"] = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
        st["q_out"] = torch.zeros((b, n, hq, d), dtype=torch.bfloat16, device="cuda")
        if case["format"] == "fp8":
            st["pool"] = _random_pool(pages, hkv, page, d, dev)
            _pool_views(st)
        else:
            st["lens"] = st["start"] + (st["new_lens"] if case["ragged"] else n)
            amax = [t.float().abs().amax((0, 1, 3)) for t in (st["k"], st["v"])]
            st["gscale"] = [(1.2 * a / 2688.0).contiguous() for a in amax]
        st["lens_after"] = (st["start"] + 1) if case["op"] == "step" else None
        st["max_len"] = max(start) + n
    else:
        lens = _lens(case, cpu)
        table, pages = _paging(b, lens, page, cpu, case["hi"])
        st["pool"] = _random_pool(pages, hkv, page, d, dev)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["max_len"] = max(lens)
        c = case["chunk"]
        shape = (b, c, hq, d) if c else (b, hq, d)
        st["q"] = torch.randn(shape, generator=dev, device="cuda").to(torch.bfloat16)
        st["chunk_lens"] = None
        if case["ragged"]:
            n = torch.randint(1, c + 1, (b,), generator=cpu).to(torch.int32)
            n[0] = c
            st["chunk_lens"] = n.cuda()
    st["page_table"], st["pages"] = table, pages
    if case["op"] != "rope_append":
        shape = st["q"].shape if case["op"] != "step" else (b, hq, d)
        st["out"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------------ the framework's calls
def _cache(st):
    """The cache object and workspace that a program keeps, made on the first pass."""
    if "cache" not in st:
        from fp4_kv_cache_kvq_gb300 import kvq
        if "pool" in st:
            st["cache"] = kvq.Fp8BlockCache(st["kv_heads"], st["d"], st["page"], st["pages"], st["page_table"].shape[1],
                                            page_table=st["page_table"], pool=st["pool"])
        else:
            st["cache"] = kvq.Fp4Cache(st["kv_heads"], st["d"], st["page"], st["pages"], st["page_table"].shape[1],
                                       page_table=st["page_table"], nvfp4=st["format"] == "nvfp4")
            if st["format"] == "nvfp4":
                st["cache"].k_gscale, st["cache"].v_gscale = st["gscale"]
        nbytes = 16
        if st["op"] in ("decode", "step"):
            nbytes = kvq.decode_workspace_bytes(st["batch"], st["q_heads"], st["kv_heads"], st["d"])
        elif st["op"] == "prefill":
            nbytes = kvq.prefill_workspace_bytes(st["batch"], st["q_heads"], st["kv_heads"], st["d"], st["chunk"])
        st["workspace"] = torch.empty(max(16, nbytes), dtype=torch.uint8, device="cuda")
        st["kvq"] = kvq
    return st["cache"], st["kvq"]


def _run_own(st):
    cache, kvq = _cache(st)
    if st["op"] == "decode":
        return kvq.decode_attn(cache, st["lens"], st["q"], st["scale"], out=st["out"], workspace=st["workspace"])
    if st["op"] == "prefill":
        return kvq.prefill_attn(cache, st["lens"], st["q"], st["scale"], out=st["out"], chunk_lens=st["chunk_lens"],
                                workspace=st["workspace"])
    kvq.rope_append(cache, st["start"], st["q"], st["k"], st["v"], st["table"], interleaved=st["interleaved"],
                    new_lens=st["new_lens"], q_out=st["q_out"])
    if st["op"] == "step":
        out = kvq.decode_attn(cache, st["lens_after"], st["q_out"][:, 0], st["scale"], out=st["out"],
                              workspace=st["workspace"])
        return {"out": out, "codes": st["codes"], "scales": st["scales"]}
    if st["format"] == "fp8":
        return {"q": st["q_out"], "codes": st["codes"], "scales": st["scales"]}
    k, v = kvq.dequant(cache, st["lens"], st["n_new"], dtype=torch.bfloat16)
    return {"q": st["q_out"], "k": k, "v": v}


# ------------------------------------------------------------------ the plain form
def _rotate(x, st):
    """bf16 [b][n][h][d] rotated by the table's rows start + t, in fp32, rounded to bf16."""
    b, n, h, d = x.shape
    r = st["rotary"]
    pos = st["start"].long()[:, None] + torch.arange(n, device=x.device)
    cs = st["table"][pos][:, :, None]
    c, s = cs[..., :r // 2], cs[..., r // 2:]
    x = x.float()
    if st["interleaved"]:
        x0, x1 = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], dim=-1).flatten(-2)
    else:
        x0, x1 = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], dim=-1)
    return torch.cat([y, x[..., r:]], dim=-1).to(torch.bfloat16)


def _new_mask(st):
    t = torch.arange(st["n_new"], device="cuda")
    if st["new_lens"] is None:
        return torch.ones((st["batch"], st["n_new"]), dtype=torch.bool, device="cuda")
    return t[None] < st["new_lens"][:, None]


def _blocks_of(st, side):
    """The pool's codes of one side by 16-token blocks: [pages][heads][groups][G/16][16 d] (a view)."""
    g, d = st["group"], st["d"]
    part = st["pool"][..., side * g * d:(side + 1) * g * d]
    return part.view(*part.shape[:-1], g // 16, 16 * d)


def _tokens(raw, side, d):
    """[..., 16 d] bytes of blocks -> [..., 16, d] in token order."""
    lead = raw.shape[:-1]
    if side == 0:
        return raw.reshape(*lead, 2, d // 16, 8, 16).transpose(-3, -2).reshape(*lead, 16, d)
    inv = torch.tensor(ORDER, device=raw.device).argsort()
    return raw.reshape(*lead, d, 16).transpose(-2, -1).index_select(-2, inv)


def _append_fp8(st, x, side):
    """Append x [b][n][h][d] (bf16) to one side of the 8-bit pool, block by block."""
    b, n, h, d = x.shape
    page, g = st["page"], st["group"]
    nblk = (n + 30) // 16
    start = st["start"].long()
    off = start % 16
    grid = torch.zeros((b, nblk * 16, h, d), dtype=torch.float32, device=x.device)
    fresh = torch.zeros((b, nblk * 16), dtype=torch.bool, device=x.device)
    at = off[:, None] + torch.arange(n, device=x.device)
    valid = _new_mask(st)
    rows = torch.arange(b, device=x.device)[:, None]
    grid[rows, at] = torch.where(valid[..., None, None], x.float(), torch.zeros((), device=x.device))
    fresh[rows, at] = valid
    grid = grid.view(b, nblk, 16, h, d).permute(0, 1, 3, 2, 4)                   # [b][blk][h][16][d]
    fresh = fresh.view(b, nblk, 1, 16)
    slot = torch.arange(16, device=x.device)
    kept = (torch.arange(nblk, device=x.device)[None, :, None] == 0) & (slot < off[:, None, None])  # [b][blk][16]
    kept = kept[:, :, None] & fresh.any(-1, keepdim=True)
    block = start[:, None] // 16 + torch.arange(nblk, device=x.device)
    pg = (block * 16 // page).clamp(max=st["page_table"].shape[1] - 1)
    phys = st["page_table"].long().gather(1, pg).clamp(min=0)
    grp, sub = (block * 16 % page) // g, (block * 16 % g) // 16
    pool = _blocks_of(st, side)
    scales = st["scales"].view(*st["scales"].shape[:-1], g // 16, 2)
    old = _tokens(pool[phys, :, grp, sub], side, d)                               # [b][blk][h][16][d]
    s_old = scales[phys, :, grp, sub, side]                                       # [b][blk][h]
    s_new = _scale_of(grid.abs().amax((-1, -2)))
    s = torch.where(kept.any(-1), torch.maximum(s_old, s_new), s_new)
    touched = fresh.any(-1).expand_as(s)
    s = torch.where(touched, s, s_old)
    again = (old.view(torch.float8_e4m3fn).float() * (s_old / s)[..., None, None]).to(torch.float8_e4m3fn)
    codes = (grid / s[..., None, None]).to(torch.float8_e4m3fn)
    merged = torch.where(fresh[..., None], codes.view(torch.uint8),
                         torch.where(kept[..., None], again.view(torch.uint8), old))
    # blocks behind the last new token keep their bytes; a sequence's row always holds one more block
    keep = ~touched[:, :, 0]
    merged = torch.where(keep[:, :, None, None, None], old, merged)
    pool[phys, :, grp, sub] = (_v_layout if side else _k_layout)(merged.contiguous())
    scales[phys, :, grp, sub, side] = s


def _fp4_values(x, gscale):
    """The values that x (bf16 [b][n][h][d]) reads back as from the 4-bit cache."""
    b, n, h, d = x.shape
    x = x.float()
    if gscale is not None:
        x = x / gscale[:, None]
    y = x.view(b, n, h, d // 16, 16)
    s = (y.abs().amax(-1, keepdim=True) / 6.0).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn).float()
    s = s.clamp(min=2.0 ** -9)
    a = (y / s).abs()
    m = (0.5 * ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float())
         + (a > 2.5).float() + (a >= 3.5).float() + 2.0 * (a > 5.0).float())
    out = (m * s * torch.where(torch.signbit(y), -1.0, 1.0)).view(b, n, h, d)
    return out * gscale[:, None] if gscale is not None else out


def _dense(st):
    """K and V in fp32, [b][heads][positions][d], of every cached position."""
    b, hkv, d, page, g = st["batch"], st["kv_heads"], st["d"], st["page"], st["group"]
    idx = st["page_table"][:, :-(-st["max_len"] // page)].long().clamp(min=0)
    raw = st["pool"][idx].transpose(1, 2)                                        # [b][h][pages][P/G][bytes]
    sc = raw[..., 2 * g * d:2 * g * d + g // 2].contiguous().view(torch.float32).view(*raw.shape[:-1], g // 16, 2)
    sides = []
    for side in range(2):
        x = raw[..., side * g * d:(side + 1) * g * d].reshape(*raw.shape[:-1], g // 16, 16 * d)
        x = _tokens(x, side, d).view(torch.float8_e4m3fn).float() * sc[..., side, None, None]
        sides.append(x.reshape(b, hkv, -1, d)[:, :, :st["max_len"]])
    return sides


def _attend(q, last, st):
    """q fp32 [b][hkv][rows][d] over the cache; row r of sequence b attends positions 0 .. last[b][r]."""
    k, v = _dense(st)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"])
    t = torch.arange(st["max_len"], device=q.device)
    s.masked_fill_(t > last[:, None, :, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / l.clamp(min=1e-30)


def _run_plain(st):
    b, hq, hkv, d = st["batch"], st["q_heads"], st["kv_heads"], st["d"]
    g = hq // hkv
    if st["op"] in ("rope_append", "step"):
        qr, kr = _rotate(st["q"], st), _rotate(st["k"], st)
        valid = _new_mask(st)[..., None, None]
        q = torch.where(valid, qr, st["q_out"])
        if st["format"] != "fp8":
            gs = st["gscale"] if st["format"] == "nvfp4" else (None, None)
            k, v = (torch.where(valid, _fp4_values(x, s), 0.0).to(torch.bfloat16)
                    for x, s in ((kr, gs[0]), (st["v"], gs[1])))
            return {"q": q, "k": k, "v": v}
        _append_fp8(st, kr, 0)
        _append_fp8(st, st["v"], 1)
        if st["op"] == "rope_append":
            return {"q": q, "codes": st["codes"], "scales": st["scales"]}
        last = (st["lens_after"].long() - 1)[:, None].expand(b, g)
        o = _attend(q[:, 0].float().view(b, hkv, g, d), last, st)
        return {"out": o.reshape(b, hq, d).to(torch.bfloat16), "codes": st["codes"], "scales": st["scales"]}
    if st["op"] == "decode":
        last = (st["lens"].long() - 1)[:, None].expand(b, g)
        o = _attend(st["q"].float().view(b, hkv, g, d), last, st)
        return o.reshape(b, hq, d).to(torch.bfloat16)
    c = st["chunk"]
    n = st["chunk_lens"].long() if st["chunk_lens"] is not None else torch.full((b,), c, device="cuda")
    i = torch.arange(c, device="cuda")
    last = (st["lens"].long() - n)[:, None] + i
    q = st["q"].float().view(b, c, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, c * g, d)
    o = _attend(q, last.clamp(max=st["max_len"]).repeat_interleave(g, 1), st)
    o = o.view(b, hkv, c, g, d).permute(0, 2, 1, 3, 4).reshape(b, c, hq, d).to(torch.bfloat16)
    return torch.where((i < n[:, None])[..., None, None], o, st["out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    b, hq, hkv, d = case["batch"], case["q_heads"], case["kv_heads"], case["d"]
    if case["op"] in ("rope_append", "step"):
        tokens = b * case["n_new"] * (0.5 if case["ragged"] else 1.0)
        rows = case["n_new"] + case["context"] // 2 if case["n_new"] > 1 else min(b, case["context"] + 1)
        code = 1.0 if case["format"] == "fp8" else 0.5625
        nbytes = tokens * ((2 * hq + 2 * hkv) * d * 2 + 2 * hkv * d * code) + rows * case["rotary"] * 4
        if hq and case["op"] == "step":
            nbytes -= tokens * hq * d * 2
        flops = tokens * (hq + hkv) * case["rotary"] * 3
        if case["format"] != "fp8":  # read back as dense bf16 rows
            nbytes += tokens * 2 * hkv * d * code + b * case["n_new"] * 2 * hkv * d * 2
        if case["op"] == "step":
            t = 0.75 * case["context"] + 1
            nbytes += b * (t * hkv * (2 * d + 0.5) + hq * d * 2)
            flops += 4.0 * b * hq * d * t
        return {"bytes": nbytes, "flops": flops}
    mean = 0.5 * (case["lo"] + case["hi"])
    c = case["chunk"] or 1
    n = 0.5 * (c + 1) if case["ragged"] else c
    nbytes = b * (mean * hkv * (2 * d + 0.5) + n * hq * d * 4)
    return {"bytes": nbytes, "flops": 4.0 * b * hq * d * n * (mean - 0.5 * (n - 1))}


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3_round(x):
    """x (float64, |x| <= 448) to the nearest E4M3 value, ties to the even code."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.round(x / step) * step


def _offsets(t, d, g, side):
    """Byte offsets [t][d] in a group's block of the codes of tokens t of one side."""
    c = torch.arange(d, device=t.device)[None, :]
    t = t[:, None]
    if side == 0:
        return (t // 8) * (8 * d) + (c // 16) * 128 + (t % 8) * 16 + c % 16
    u = t % 16
    byte = torch.where(u < 8, 4 * (u // 2) + u % 2, 4 * ((u - 8) // 2) + 2 + u % 2)
    return g * d + (t // 16) * (16 * d) + c * 16 + byte


def _exact_rows(st, b, h, n, side):
    """Values of positions 0 .. n - 1 of one sequence and head, float64 [n][d]."""
    page, g, d = st["page"], st["group"], st["d"]
    t = torch.arange(n, device="cuda")
    phys = st["page_table"][b].long()[t // page]
    block = st["pool"][phys, h, (t % page) // g]
    code = block.gather(1, _offsets(t % g, d, g, side)).view(torch.float8_e4m3fn).double()
    sc = st["scales"][phys, h, (t % page) // g].gather(1, (2 * ((t % g) // 16) + side)[:, None])
    return code * sc.double()


def _exact_attend(st, q, last_of):
    """float64 attention, one sequence and head at a time; q [b][rows][hq][d] -> the same."""
    b, rows, hq, d = q.shape
    g = hq // st["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lens = (st["lens_after"] if st["op"] == "step" else st["lens"]).tolist()
    for i in range(b):
        last = last_of(i)
        for h in range(st["kv_heads"]):
            k, v = (_exact_rows(st, i, h, lens[i], side) for side in range(2))
            x = q[i, :, h * g:(h + 1) * g].double().reshape(-1, d)
            s = x @ k.T * st["scale"]
            hide = torch.arange(lens[i], device="cuda") > last.repeat_interleave(g)[:, None]
            s[hide] = -math.inf
            out[i, :, h * g:(h + 1) * g] = (torch.softmax(s, -1) @ v).view(rows, g, d)
    return out


def _exact_rotate(x, st):
    b, n, h, d = x.shape
    r = st["rotary"]
    out = x.double().clone()
    i = torch.arange(r // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if st["interleaved"] else (i, i + r // 2)
    for j in range(b):
        at = int(st["start"][j])
        cs = st["table"][at:at + n].double()[:, None]
        z = torch.complex(x[j].double()[..., first], x[j].double()[..., second])
        z = z * torch.complex(cs[..., :r // 2], cs[..., r // 2:])
        out[j][..., first], out[j][..., second] = z.real, z.imag
    return out.to(torch.bfloat16)


def _exact_append(st, kr):
    """The pool's codes (as values) and scales after the append, laid out as the pool."""
    g, d, page = st["group"], st["d"], st["page"]
    codes, scales = st["codes"].double(), st["scales"].double()
    for b in range(st["batch"]):
        sp = int(st["start"][b])
        n = st["n_new"] if st["new_lens"] is None else int(st["new_lens"][b])
        for side, x in ((0, kr), (1, st["v"])):
            for blk in range(sp // 16, (sp + n + 15) // 16 if n else 0):
                lo, hi = max(sp, 16 * blk), min(sp + n, 16 * blk + 16)
                rows = x[b, lo - sp:hi - sp].double().transpose(0, 1)            # [h][tokens][d]
                amax = rows.abs().amax((1, 2))
                e = torch.ceil(torch.log2((amax / E4M3_MAX).clamp(min=2.0 ** -140))).clamp(-126, 120)
                s = torch.exp2(e)
                phys = int(st["page_table"][b, 16 * blk // page])
                grp, idx = (16 * blk % page) // g, 2 * ((16 * blk % g) // 16) + side
                t0 = 16 * blk % g
                if lo > 16 * blk:
                    old = scales[phys, :, grp, idx].clone()
                    s = torch.maximum(s, old)
                    at = _offsets(torch.arange(t0, t0 + lo - 16 * blk, device="cuda"), d, g, side).reshape(-1)
                    codes[phys, :, grp, at] = _e4m3_round(codes[phys, :, grp, at] * (old / s)[:, None])
                at = _offsets(torch.arange(t0 + lo - 16 * blk, t0 + hi - 16 * blk, device="cuda"), d, g, side).reshape(-1)
                codes[phys, :, grp, at] = _e4m3_round(rows.reshape(rows.shape[0], -1) / s[:, None])
                scales[phys, :, grp, idx] = s
    return codes, scales


def _exact_fp4(x, gscale):
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    b, n, h, d = x.shape
    y = x.double()
    if gscale is not None:
        y = (y / gscale.double()[:, None]).float().double()  # x / S is held in fp32
    y = y.view(b, n, h, d // 16, 16)
    s = _e4m3_round((y.abs().amax(-1, keepdim=True) / 6.0).clamp(max=E4M3_MAX)).clamp(min=2.0 ** -9)
    a = (y / s).abs().clamp(max=6.0)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)
    up, dn = grid[hi], grid[hi - 1]
    take = (up - a < a - dn) | ((up - a == a - dn) & (hi % 2 == 0))
    out = (torch.where(take, up, dn) * s * torch.where(torch.signbit(y), -1.0, 1.0)).view(b, n, h, d)
    return out * gscale.double()[:, None] if gscale is not None else out


def exact(case, seed):
    if case["op"] in ("rope_append", "step") and case["format"] == "fp8":
        if case["batch"] * (case["n_new"] + 15) // 16 > 4000:
            return None
    st = prepare(case, seed)
    b, hq, hkv, d = case["batch"], case["q_heads"], case["kv_heads"], case["d"]
    if case["op"] == "decode":
        lens = st["lens"].long()
        _pool_views(st)
        return _exact_attend(st, st["q"][:, None], lambda i: lens[i:i + 1] - 1)[:, 0]
    if case["op"] == "prefill":
        lens = st["lens"].long()
        _pool_views(st)
        c = case["chunk"]
        n = st["chunk_lens"].long() if st["chunk_lens"] is not None else torch.full_like(lens, c)
        i = torch.arange(c, device="cuda")
        o = _exact_attend(st, st["q"], lambda j: (lens[j] - n[j] + i).clamp(max=lens[j] - 1))
        return torch.where((i < n[:, None])[..., None, None], o, 0.0)
    qr, kr = _exact_rotate(st["q"], st), _exact_rotate(st["k"], st)
    valid = _new_mask(st)[..., None, None]
    q = torch.where(valid, qr.double(), 0.0)
    if case["format"] != "fp8":
        gs = st["gscale"] if case["format"] == "nvfp4" else (None, None)
        k, v = (torch.where(valid, _exact_fp4(x, s), 0.0) for x, s in ((kr, gs[0]), (st["v"], gs[1])))
        return {"q": q, "k": k, "v": v}
    codes, scales = _exact_append(st, kr)
    if case["op"] == "rope_append":
        return {"q": q, "codes": codes, "scales": scales}
    st["codes"].copy_(codes.to(torch.float8_e4m3fn))
    st["scales"].copy_(scales.float())
    lens = st["lens_after"].long()
    out = _exact_attend(st, q.to(torch.bfloat16), lambda i: lens[i:i + 1] - 1)[:, 0]
    return {"out": out, "codes": codes, "scales": scales}
