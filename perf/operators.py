"""The operators between the quantized matrix products of a decode or prefill
step, on a paged key / value cache held in Q4_0 (4 bits a value and an fp16
scale per 32 values), as measured cases:

  plan   block tables, slots and positions of a step, from request lengths
  rope   norms of queries and keys per head, the position rotation, and the
         store of keys and values into the cache (read back as values)
  attn   causal attention over the cache: single tokens, chunks, whole
         prompts; optionally a sliding window with first tokens kept visible

`run` computes them in plain torch operations, or, where `own` is true, by the
calls that a user makes.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_EPS = 1e-6


# ---------------------------------------------------------------------------- the cases

def listed():
    return [
        # one new token for each of a few requests: the smallest call of a serving loop
        {"name": "plan, 8 decoding requests", "op": "plan", "requests": 8, "tokens": 8, "ctx": 4096, "page": 16},
        # a large mixed step: many requests, prompts of all lengths among them
        {"name": "plan, 2048 requests", "op": "plan", "requests": 2048, "tokens": 131072, "ctx": 16384, "page": 32},
        # one token of a 24-head layer (latency), fp32 activations, adjacent-pair rotation
        {"name": "qkv, 1 token f32", "op": "rope", "tokens": 1, "heads": 24, "kv_heads": 8, "dim": 128, "rot": 128,
         "neox": False, "norm": True, "type": "f32", "page": 16, "positions": 131072},
        # a small batch of a layer with wide heads, of which a quarter is rotated
        {"name": "qkv, 77 tokens d256 f16", "op": "rope", "tokens": 77, "heads": 16, "kv_heads": 2, "dim": 256,
         "rot": 64, "neox": True, "norm": True, "type": "f16", "page": 32, "positions": 32768},
        # a prompt chunk
        {"name": "qkv, 2048 tokens", "op": "rope", "tokens": 2048, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "neox": True, "norm": True, "type": "bf16", "page": 64, "positions": 32768},
        # one short request, fp32 activations: latency
        {"name": "decode, 1 x 333 f32", "op": "attn", "requests": 1, "singles": 1, "q": 1, "ctx": 332, "heads": 24,
         "kv_heads": 8, "dim": 128, "type": "f32", "page": 16, "window": 0, "sinks": 0},
        # a decoding batch with ragged lengths
        {"name": "decode, 32 x 8192", "op": "attn", "requests": 32, "singles": 32, "q": 1, "ctx": 8191, "heads": 32,
         "kv_heads": 8, "dim": 128, "type": "bf16", "page": 64, "window": 0, "sinks": 0},
        # few requests with long contexts, wide heads shared by eight queries
        {"name": "decode, 4 x 131072 d256", "op": "attn", "requests": 4, "singles": 4, "q": 1, "ctx": 131071,
         "heads": 16, "kv_heads": 2, "dim": 256, "type": "bf16", "page": 128, "window": 0, "sinks": 0},
        # a sliding-window layer of a decoding batch, first tokens kept
        {"name": "decode, window 4096 d64 f16", "op": "attn", "requests": 64, "singles": 64, "q": 1, "ctx": 32767,
         "heads": 32, "kv_heads": 8, "dim": 64, "type": "f16", "page": 32, "window": 4096, "sinks": 4},
        # a mixed step: prompt chunks beside decoding requests
        {"name": "mixed, chunks of 512", "op": "attn", "requests": 12, "singles": 8, "q": 512, "ctx": 3500,
         "heads": 24, "kv_heads": 8, "dim": 128, "type": "bf16", "page": 16, "window": 0, "sinks": 0},
        # a whole long prompt
        {"name": "prefill, 8192", "op": "attn", "requests": 1, "singles": 0, "q": 8192, "ctx": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "type": "bf16", "page": 64, "window": 0, "sinks": 0},
        # prompts of odd lengths in a sliding-window layer
        {"name": "prefill, window 1000 d64 f16", "op": "attn", "requests": 2, "singles": 0, "q": 4093, "ctx": 0,
         "heads": 32, "kv_heads": 8, "dim": 64, "type": "f16", "page": 32, "window": 1000, "sinks": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = ((24, 8), (32, 8), (16, 2), (8, 8), (28, 4), (12, 1))


def draw(rng):
    most = [work(c) for c in listed()]
    while True:   # none larger than the largest listed
        case = _draw(rng)
        w = work(case)
        if all(w[k] <= max(m[k] for m in most) for k in w):
            return case


def _draw(rng):
    kind = rng.choice(("plan", "rope", "rope", "decode", "decode", "decode", "chunk", "prefill"))
    page = rng.choice((16, 32, 64, 128))
    heads, kv_heads = rng.choice(_HEADS)
    dim = rng.choice((64, 128, 128, 256))
    if kind == "plan":
        n = _log(rng, 1, 2048)
        return {"op": "plan", "requests": n, "tokens": max(n, _log(rng, n, 131072)), "ctx": _log(rng, 64, 16384),
                "page": page}
    if kind == "rope":
        return {"op": "rope", "tokens": _log(rng, 1, 2048), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice((dim, dim, dim // 2, dim // 4)), "neox": rng.random() < 0.5,
                "norm": rng.random() < 0.75, "type": rng.choice(("bf16", "bf16", "f16", "f32")), "page": page,
                "positions": 32768}
    window = rng.choice((0, 0, _log(rng, 50, 4096)))
    case = {"op": "attn", "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window,
            "sinks": rng.choice((0, 4, 20)) if window else 0}
    if kind == "decode":
        n = _log(rng, 1, 64)
        q = rng.choice((1, 1, 1, 2, 3))   # a few tokens to check at once now and then
        case.update(requests=n, singles=n if q == 1 else n // 2, q=q, ctx=_log(rng, 30, min(131072, 262144 // n)),
                    type=rng.choice(("bf16", "bf16", "f16", "f32")))
    elif kind == "chunk":
        n = rng.randint(2, 12)
        case.update(requests=n, singles=rng.randint(0, n - 1), q=_log(rng, 17, 1024), ctx=_log(rng, 100, 4000),
                    type=rng.choice(("bf16", "bf16", "f16")))
    else:
        n = rng.randint(1, 3)
        case.update(requests=n, singles=0, q=_log(rng, 300, 4096), ctx=rng.choice((0, 0, 555)),
                    type=rng.choice(("bf16", "bf16", "f16")))
    return case


def _spread(n, total):
    """n whole numbers >= 1 of different sizes with the given sum."""
    extra = total - n
    cum = [extra * i * i // (n * n) for i in range(n + 1)]
    return [1 + cum[i + 1] - cum[i] for i in range(n)]


def _lengths(case):
    """(query tokens, tokens cached before) of each request, the longest first."""
    n, singles = case["requests"], case["singles"]
    q = [max(1, case["q"] * (n - i) // n) for i in range(n - singles)]
    q = q + [1] * singles if case["q"] > 1 else [1] * n
    ctx = [case["ctx"] - case["ctx"] * 3 * i // (4 * n) for i in range(n)]
    return q, ctx


def _visible(case):
    """Over all requests: cache tokens that some query sees, and (query, token) pairs."""
    tokens = pairs = 0
    w, s = case["window"], case["sinks"]
    for q, c in zip(*_lengths(case)):
        pos = np.arange(c, c + q, dtype=np.int64)
        if w:
            first = np.maximum(pos - w + 1, 0)
            pairs += int((pos + 1 - first + np.minimum(first, s)).sum())
            tokens += int(c + q - first[0] + min(int(first[0]), s))
        else:
            pairs += int((pos + 1).sum())
            tokens += c + q
    return tokens, pairs


def work(case):
    if case["op"] == "plan":
        n, t = case["requests"], case["tokens"]
        pages = t // case["page"]   # about that many are new
        return {"bytes": 4 * n * 4 + 12 * t + 8 * pages, "flops": 0}
    e = 4 if case["type"] == "f32" else 2
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        t = case["tokens"]
        # q, k, v and the table's rows in; q and the packed rows out; the rows read back as bf16 values
        row = (2 * h + 2 * hk) * d * e + 4 * case["rot"] + 2 * hk * d * 18 // 32 + 12
        return {"bytes": t * (row + 2 * hk * d * 18 // 32 + 4 * hk * d), "flops": t * (h + hk) * d * 8}
    q, c = _lengths(case)
    tokens, pairs = _visible(case)
    return {"bytes": tokens * hk * d * 36 // 32 + 2 * sum(q) * h * d * e, "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------------------- inputs

_CODES = None


def _codes(device):
    """Bytes of two 4-bit codes, as Q4_0 gives them for normal values, in a table to draw from."""
    global _CODES
    if _CODES is None or _CODES.device != device:
        gen = torch.Generator(device=device).manual_seed(11)
        x = torch.randn(1 << 16, 32, generator=gen, device=device)
        big = x.gather(1, x.abs().argmax(1, keepdim=True))
        c = (x * (-8.0 / big) + 8.5).floor().clamp(0, 15).to(torch.uint8).reshape(-1, 2)
        _CODES = (c[:, 0] | (c[:, 1] << 4)).contiguous()
    return _CODES


def _cache(pages, kv_heads, dim, page, gen, device):
    """Pages of packed keys and values with codes and scales as normal values of different sizes have them."""
    tiles = pages * kv_heads * (page // 16)
    codes = _codes(device)
    out = torch.empty(tiles, 18 * dim, dtype=torch.uint8, device=device)
    for part in range(2):
        at = part * 9 * dim
        step = max(1, (1 << 28) // (8 * dim))
        for a in range(0, tiles, step):
            b = min(tiles, a + step)
            pick = torch.randint(0, codes.numel(), (b - a, 8 * dim), generator=gen, device=device, dtype=torch.int32)
            out[a:b, at:at + 8 * dim] = codes[pick]
            size = torch.randn(b - a, dim // 2, generator=gen, device=device).mul_(0.2).exp_().mul_(0.28)
            sign = torch.randint(0, 2, size.shape, generator=gen, device=device, dtype=torch.int32) * 2 - 1
            out[a:b, at + 8 * dim:at + 9 * dim] = (size * sign).to(torch.float16).view(torch.uint8)
    return out.view(pages, -1)


def _cos_sin(positions, rot, device):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    a = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = np.random.default_rng(seed)
    if case["op"] == "plan":
        n, page = case["requests"], case["page"]
        new = np.array(_spread(n, case["tokens"]))[rnd.permutation(n)]
        ctx = rnd.integers(0, case["ctx"] + 1, n)
        width = -(-(case["ctx"] + int(new.max())) // page)
        had = -(-ctx // page)
        need = int((-(-(ctx + new) // page) - had).sum())
        order = torch.randperm(int(had.sum()) + need + 64, generator=gen, device=dev).to(torch.int32)
        table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
        cols = torch.arange(width, device=dev)[None]
        held = cols < torch.from_numpy(had).to(dev)[:, None]
        table[held] = order[:int(had.sum())]
        as_int = lambda a: torch.from_numpy(a.astype(np.int32)).to(dev)  # noqa: E731
        empty = lambda m, t: torch.empty(m, dtype=t, device=dev)  # noqa: E731
        return {"case": case, "ctx": as_int(ctx), "new": as_int(new), "free": order[int(had.sum()):].contiguous(),
                "table": table,
                "out": (empty(n + 1, torch.int32), empty(n, torch.int32), empty(case["tokens"], torch.int32),
                        empty(case["tokens"], torch.int64), empty(1, torch.int32))}
    typ, d, hk, page = _TYPES[case["type"]], case["dim"], case["kv_heads"], case["page"]
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
    if case["op"] == "rope":
        t, h = case["tokens"], case["heads"]
        qkv = (normal(t, (h + 2 * hk) * d) * 1.5).to(typ)   # one fused projection's rows
        pages = -(-t // page) + 3
        cache = torch.zeros(pages, hk * page * d * 18 // 16, dtype=torch.uint8, device=dev)
        # consecutive slots of pages in any order
        at = torch.randperm(pages, generator=gen, device=dev)
        tok = torch.arange(t, device=dev)
        slots = at[tok // page] * page + tok % page
        first = int(rnd.integers(0, case["positions"] - t))
        weight = lambda: (1 + 0.1 * normal(d)) if case["norm"] else None  # noqa: E731
        return {"case": case, "q": qkv[:, :h * d].view(t, h, d), "k": qkv[:, h * d:(h + hk) * d].view(t, hk, d),
                "v": qkv[:, (h + hk) * d:].view(t, hk, d), "qw": weight(), "kw": weight(),
                "pos": torch.arange(first, first + t, device=dev, dtype=torch.int32), "slots": slots,
                "table": _cos_sin(case["positions"], case["rot"], dev), "cache": cache,
                "out": torch.empty(t, h, d, dtype=typ, device=dev),
                "kv": [torch.empty(t, hk, d, dtype=torch.bfloat16, device=dev) for _ in range(2)]}
    q, ctx = _lengths(case)
    order = rnd.permutation(len(q))
    q, ctx = np.array(q)[order], np.array(ctx)[order]
    kv = q + ctx
    counts = -(-kv // page)
    pages = int(counts.sum()) + 5
    cache = _cache(pages, hk, d, page, gen, dev)
    at = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(q), int(counts.max())), -1, dtype=torch.int32, device=dev)
    table[torch.arange(table.shape[1], device=dev)[None] < torch.from_numpy(counts).to(dev)[:, None]] = \
        at[:int(counts.sum())]
    x = (normal(int(q.sum()), case["heads"], d) * 2).to(typ)
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(q)]).astype(np.int32)).to(dev)
    return {"case": case, "q": x, "cache": cache, "table": table, "start": start, "max_q": int(q.max()),
            "kv_len": torch.from_numpy(kv.astype(np.int32)).to(dev), "out": torch.empty_like(x)}


# ---------------------------------------------------------------------------- the framework's calls

_pkg = None


def _framework():
    global _pkg
    if _pkg is None:
        import gguf_block_quantized_quantize_gb300 as pkg
        _pkg = pkg
    return _pkg


def _own(s):
    g, c = _framework(), s["case"]
    if c["op"] == "plan":
        start, kv_len, pos, slots, used = g.gguf_kv_plan(s["ctx"], s["new"], s["free"], s["table"], c["page"],
                                                         c["tokens"], out=s["out"])
        return {"start": start, "kv_len": kv_len, "pos": pos, "slots": slots, "used": used, "table": s["table"]}
    if c["op"] == "rope":
        q = g.gguf_qk_norm_rope(s["q"], s["k"], s["v"], s["qw"], s["kw"], _EPS, s["pos"], s["table"],
                                g.ROPE_NEOX if c["neox"] else g.ROPE_NORM, cache=s["cache"], slots=s["slots"],
                                page_size=c["page"], q_out=s["out"])
        k, v = g.gguf_kv_get_rows(s["cache"], s["slots"], c["kv_heads"], c["dim"], c["page"], out=s["kv"])
        return {"q": q, "k": k, "v": v}
    return g.gguf_paged_attention(s["q"], s["cache"], s["table"], s["start"], s["kv_len"], c["kv_heads"], c["page"],
                                  s["max_q"], c["dim"] ** -0.5, window=c["window"], sinks=c["sinks"], out=s["out"])


# ---------------------------------------------------------------------------- plain forms

def _plain_plan(s):
    c = s["case"]
    page, dev = c["page"], s["ctx"].device
    ctx, new = s["ctx"].long(), s["new"].long()
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), new.cumsum(0)])
    kv = ctx + new
    had, has = (ctx + page - 1) // page, (kv + page - 1) // page
    before = (has - had).cumsum(0) - (has - had)
    col = torch.arange(s["table"].shape[1], device=dev)[None]
    rank = before[:, None] + col - had[:, None]
    fresh = (col >= had[:, None]) & (col < has[:, None])
    table = torch.where(fresh, s["free"][rank.clamp(0, s["free"].numel() - 1)], s["table"])
    tok = torch.arange(c["tokens"], device=dev)
    req = torch.searchsorted(start, tok, right=True) - 1
    pos = ctx[req] + tok - start[req]
    slots = table[req, pos // page].long() * page + pos % page
    i32 = torch.int32
    return {"start": start.to(i32), "kv_len": kv.to(i32), "pos": pos.to(i32), "slots": slots,
            "used": (has - had).sum().to(i32).reshape(1), "table": table}


def _plain_norm(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w


def _plain_rotate(x, cs, rot, neox):
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    r = x[..., :rot]
    a, b = (r[..., :rot // 2], r[..., rot // 2:]) if neox else (r[..., 0::2], r[..., 1::2])
    y, z = a * cos - b * sin, b * cos + a * sin
    r = torch.cat([y, z], -1) if neox else torch.stack([y, z], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_q4(x):
    """Values as Q4_0 holds them: blocks of 32, scale = the value of largest magnitude / -8, held in fp16;
    codes are the multiples of the held scale, rounded half away from zero."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    d = (b.gather(-1, b.abs().argmax(-1, keepdim=True)) * -0.125).to(torch.float16).float()
    c = torch.where(d == 0, torch.zeros_like(b), b / d)
    whole = c.trunc()
    c = (whole + ((c - whole).abs() >= 0.5) * c.sign()).clamp(-8, 7)
    return (d * c).reshape(x.shape)


def _plain_rope(s):
    c = s["case"]
    cs = s["table"][s["pos"].long()]
    q = _plain_rotate(_plain_norm(s["q"].float(), s["qw"]), cs, c["rot"], c["neox"])
    k = _plain_rotate(_plain_norm(s["k"].float(), s["kw"]), cs, c["rot"], c["neox"])
    return {"q": q.to(s["q"].dtype), "k": _plain_q4(k).to(torch.bfloat16),
            "v": _plain_q4(s["v"].float()).to(torch.bfloat16)}


def _plain_unpack(tiles, d):
    """Keys and values [n, 16, d] (fp32) of packed tiles [n, 18 d]."""
    n, nb = tiles.shape[0], d // 32
    bw = min(nb, 4)
    nc = nb // bw
    nibbles = lambda b: torch.stack([b & 15, b >> 4], -1)  # noqa: E731
    scale = lambda b: b.contiguous().view(torch.float16).float().view(n, 8, nb, 2)  # noqa: E731
    # keys: [token / 8][block chunk][token % 8][quarter][block][half][byte][nibble], value = quarter, byte, nibble, half
    k = nibbles(tiles[:, :8 * d].reshape(n, 2, nc, 8, 4, bw, 2, 2)).to(torch.float32)
    k = k.permute(0, 1, 3, 2, 5, 4, 7, 8, 6).reshape(n, 16, nb, 32)
    ks = scale(tiles[:, 8 * d:9 * d]).permute(0, 1, 3, 2).reshape(n, 16, nb, 1)
    # values: [token / 8][block chunk][eighth][token % 8 / 2][block][token % 2][byte][nibble], value = eighth, byte, nibble
    v = nibbles(tiles[:, 9 * d:17 * d].reshape(n, 2, nc, 8, 4, bw, 2, 2)).to(torch.float32)
    v = v.permute(0, 1, 4, 6, 2, 5, 3, 7, 8).reshape(n, 16, nb, 32)
    vs = scale(tiles[:, 17 * d:]).permute(0, 1, 3, 2).reshape(n, 16, nb, 1)
    return (k.sub_(8) * ks).view(n, 16, d), (v.sub_(8) * vs).view(n, 16, d)


def _plain_attn(s):
    c = s["case"]
    d, hk, h, page = c["dim"], c["kv_heads"], c["heads"], c["page"]
    x, dev = s["q"], s["q"].device
    n, width = s["table"].shape
    t, lq = x.shape[0], s["max_q"]
    start = s["start"].long()
    pages = s["cache"][s["table"].clamp(min=0).long().flatten()]
    k, v = _plain_unpack(pages.view(-1, 18 * d), d)
    # [n, width, hk, page / 16, 16, d] -> [n, hk, d, tokens] and [n, hk, tokens, d]
    k = k.view(n, width, hk, page, d).permute(0, 2, 4, 1, 3).reshape(n, hk, d, width * page)
    v = v.view(n, width, hk, page, d).permute(0, 2, 1, 3, 4).reshape(n, hk, width * page, d)
    i = torch.arange(lq, device=dev)[None]
    length = start[1:] - start[:-1]
    q = x[(start[:-1, None] + i).clamp(max=t - 1)].float().view(n, lq, hk, h // hk, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    score = torch.matmul(q, k).mul_(d ** -0.5)
    del k
    pos = (s["kv_len"].long() - length)[:, None] + i
    j = torch.arange(width * page, device=dev)
    hide = j > pos[..., None]
    if c["window"]:
        hide |= (j <= pos[..., None] - c["window"]) & (j >= c["sinks"])
    hide = hide[:, None, None]
    score = score.view(n, hk, h // hk, lq, -1).masked_fill_(hide, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1)
    v.masked_fill_((j >= s["kv_len"].long()[:, None])[:, None, :, None], 0)
    o = torch.matmul(p.view(n, hk, -1, width * page), v).view(n, hk, h // hk, lq, d)
    o = torch.where(total[..., None] == 0, torch.zeros_like(o), o / total[..., None])
    tok = torch.arange(t, device=dev)
    req = torch.searchsorted(start, tok, right=True) - 1
    return o[req, :, :, tok - start[req]].reshape(t, h, d).to(x.dtype)


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "rope": _plain_rope, "attn": _plain_attn}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- 64 bits

def _exact_rows(cache, rows, head, d, page, hk):
    """Keys and values of one head at the cache slots `rows`, by the place of each value in a page."""
    tile = (rows // page) * (hk * page // 16) + head * (page // 16) + rows % page // 16
    flat = cache.view(-1)
    tok = (rows % 16)[:, None]
    i = torch.arange(d, device=rows.device)[None]
    b, x = i // 32, i % 32
    nb = d // 32
    bw = min(nb, 4)
    base = (tile * (18 * d))[:, None]
    # word and bit of the key: words of 8 values, pairs of values in the two halves
    wk = ((tok // 8 * (nb // bw) + b // bw) * 32 + tok % 8 * 4 + x // 8) * bw + b % bw
    bit = x % 8 // 2 * 4 + x % 2 * 16
    k = (flat[base + 4 * wk + bit // 8].long() >> (bit % 8)) & 15
    # word and bit of the value: words of 4 values of two tokens
    wv = ((tok // 8 * (nb // bw) + b // bw) * 32 + x // 4 * 4 + tok % 8 // 2) * bw + b % bw
    bit = x % 4 * 4 + tok % 2 * 16
    v = (flat[base + 9 * d + 4 * wv + bit // 8].long() >> (bit % 8)) & 15
    at = (tok // 2 * nb + b) * 2 + tok % 2
    half = lambda o: (flat[o].long() | flat[o + 1].long() << 8).to(torch.int32).to(torch.int16)  # noqa: E731
    ks, vs = (half(base + o + 2 * at).view(torch.float16).double() for o in (8 * d, 17 * d))
    return (k - 8).double() * ks, (v - 8).double() * vs


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    d, hk = case["dim"], case["kv_heads"]
    if case["op"] == "rope":
        half = case["rot"] // 2
        cs = s["table"][s["pos"].long()].double()
        first = torch.arange(half, device="cuda") * (1 if case["neox"] else 2)
        second = first + (half if case["neox"] else 1)

        def turned(x, w):
            x = x.double()
            if w is not None:
                x = x / (x.square().sum(-1, keepdim=True) / d + _EPS).sqrt() * w.double()
            y = x.clone()
            cos, sin = cs[:, None, :half], cs[:, None, half:]
            y[..., first] = x[..., first] * cos - x[..., second] * sin
            y[..., second] = x[..., first] * sin + x[..., second] * cos
            return y

        def held(x):
            x = x.unflatten(-1, (-1, 32))
            scale = (torch.take_along_dim(x, x.abs().max(-1, keepdim=True).indices, -1) / -8).half().double()
            steps = x / scale
            return (scale * (steps.sign() * torch.floor(steps.abs() + 0.5)).clamp(-8, 7)).flatten(-2)

        return {"q": turned(s["q"], s["qw"]), "k": held(turned(s["k"], s["kw"])), "v": held(s["v"].double())}
    g, page = case["heads"] // hk, case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, lens = s["start"].tolist(), s["kv_len"].tolist()
    for r, n in enumerate(lens):
        a, e = starts[r], starts[r + 1]
        tok = torch.arange(n, device="cuda")
        rows = s["table"][r].long()[tok // page] * page + tok % page
        for head in range(hk):
            parts = [_exact_rows(s["cache"], c, head, d, page, hk) for c in rows.split(1 << 17)]
            k, v = (torch.cat(p) for p in zip(*parts))
            for c in range(a, e, 1024):
                f = min(e, c + 1024)
                x = s["q"][c:f, head * g:(head + 1) * g].double().transpose(0, 1)
                p = torch.arange(n - e + c, n - e + f, device="cuda")[:, None]
                see = tok <= p
                if case["window"]:
                    see &= (tok > p - case["window"]) | (tok < case["sinks"])
                score = torch.where(see, x @ k.T / math.sqrt(d), -math.inf)
                out[c:f, head * g:(head + 1) * g] = (torch.softmax(score, -1) @ v).transpose(0, 1)
    return out
