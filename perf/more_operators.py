"""The operators around the quantized products of a batch that asks about one
long prompt of text and images, as measured cases:

  norm   the norms before and after a block with its gate, the residual sum,
         and the next product's input as floats and as q8_1 blocks
  rope   norms of queries and keys per head, the rotation by positions on
         several axes (time, height, width), and the store into the Q4_0 cache
  attn   attention of requests that share the pages of a long prefix, group by
         group: the plan from lengths and groups, then the attention

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
        # one new token between two products of a decode step: latency; the next product takes q8_1 rows
        {"name": "norm 1 token", "op": "norm", "tokens": 1, "width": 4096, "type": "bf16", "resid": "bf16",
         "post": "none", "pre": "rms", "gate": "none", "float": False, "q8": True},
        # a decoding batch, norms on both sides and a gate of its own per token, residual stream in fp32
        {"name": "norm 64 tokens gated f16", "op": "norm", "tokens": 64, "width": 2048, "type": "f16", "resid": "f32",
         "post": "rms", "pre": "rms", "gate": "rows", "float": True, "q8": True},
        # fp32 activations with centred norms, biases and one gate row for all tokens, an odd width
        {"name": "norm 777 tokens centred f32", "op": "norm", "tokens": 777, "width": 1111, "type": "f32",
         "resid": "f32", "post": "layer", "pre": "layer", "gate": "row", "float": True, "q8": False},
        # a long prompt, norms on both sides
        {"name": "norm 8192 tokens", "op": "norm", "tokens": 8192, "width": 4096, "type": "bf16", "resid": "bf16",
         "post": "rms", "pre": "rms", "gate": "none", "float": True, "q8": True},
        # one token of a decode step: latency
        {"name": "rope 1 token", "op": "rope", "tokens": 1, "heads": 24, "kv_heads": 8, "dim": 128,
         "sections": "16,24,24", "mixed": False, "neox": True, "norm": True, "type": "bf16", "page": 16},
        # a small image, wide heads of which a quarter is rotated, two axes
        {"name": "rope 333 tokens d256 f16", "op": "rope", "tokens": 333, "heads": 16, "kv_heads": 2, "dim": 256,
         "sections": "16,16", "mixed": False, "neox": False, "norm": True, "type": "f16", "page": 32},
        # a prompt of images and text, axes in turn
        {"name": "rope 4096 tokens", "op": "rope", "tokens": 4096, "heads": 32, "kv_heads": 8, "dim": 128,
         "sections": "24,20,20", "mixed": True, "neox": True, "norm": True, "type": "bf16", "page": 64},
        # two short requests, fp32 activations: latency
        {"name": "attn 2 x (700 + 60) f32", "op": "attn", "groups": 1, "per": 2, "prefix": 700, "tail": 60, "q": 1,
         "heads": 24, "kv_heads": 8, "dim": 128, "type": "f32", "page": 16, "window": 0, "sinks": 0},
        # a decoding batch on one system prompt
        {"name": "attn 32 x (8192 + 512)", "op": "attn", "groups": 1, "per": 32, "prefix": 8192, "tail": 512, "q": 1,
         "heads": 32, "kv_heads": 8, "dim": 128, "type": "bf16", "page": 64, "window": 0, "sinks": 0},
        # several prompts, each with a few requests, wide heads shared by eight queries
        {"name": "attn 6 x 8 x (5000 + 300) d256", "op": "attn", "groups": 6, "per": 8, "prefix": 5000, "tail": 300,
         "q": 1, "heads": 16, "kv_heads": 2, "dim": 256, "type": "bf16", "page": 32, "window": 0, "sinks": 0},
        # a few tokens of each request to check at once, fp16
        {"name": "attn 16 x 4 x (20000 + 400) d64", "op": "attn", "groups": 1, "per": 16, "prefix": 20000,
         "tail": 400, "q": 4, "heads": 32, "kv_heads": 8, "dim": 64, "type": "f16", "page": 16, "window": 0,
         "sinks": 0},
        # many samples from one long document
        {"name": "attn 256 x (32768 + 128)", "op": "attn", "groups": 1, "per": 256, "prefix": 32768, "tail": 128,
         "q": 1, "heads": 32, "kv_heads": 8, "dim": 128, "type": "bf16", "page": 64, "window": 0, "sinks": 0},
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
    kind = rng.choice(("norm", "norm", "rope", "attn", "attn", "attn"))
    page = rng.choice((16, 32, 64, 128))
    typ = rng.choice(("bf16", "bf16", "f16", "f32"))
    if kind == "norm":
        q8 = rng.random() < 0.6
        width = _log(rng, 64, 16384)
        return {"op": "norm", "tokens": _log(rng, 1, 8192), "width": (width + 31) // 32 * 32 if q8 else width,
                "type": typ, "resid": rng.choice((typ, "f32")), "post": rng.choice(("none", "rms", "layer")),
                "pre": rng.choice(("rms", "rms", "layer")), "gate": rng.choice(("none", "rows", "row")),
                "float": not q8 or rng.random() < 0.5, "q8": q8}
    heads, kv_heads = rng.choice(_HEADS)
    dim = rng.choice((64, 128, 128, 256))
    if kind == "rope":
        pairs = rng.choice((dim, dim, dim // 2)) // 2
        n = rng.choice((2, 3, 3, 4))
        cuts = sorted(rng.sample(range(1, pairs), n - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        return {"op": "rope", "tokens": _log(rng, 1, 4096), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "sections": ",".join(map(str, sections)), "mixed": rng.random() < 0.5, "neox": rng.random() < 0.7,
                "norm": rng.random() < 0.75, "type": typ, "page": page}
    window = rng.choice((0, 0, 0, _log(rng, 50, 8192)))
    per = _log(rng, 1, 256)
    return {"op": "attn", "groups": _log(rng, 1, 1 + 64 // per), "per": per, "prefix": _log(rng, 30, 40000),
            "tail": _log(rng, 1, 1500), "q": rng.choice((1, 1, 1, 2, 4)), "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "type": typ if per < 64 else rng.choice(("bf16", "f16")), "page": page, "window": window,
            "sinks": rng.choice((0, 4, 20)) if window else 0}


def _batch(case):
    """Requests per group, prefix tokens of each group; of each request its group, cached tokens of its own, queries."""
    n, per = case["groups"], case["per"]
    size = np.array([max(1, per - per * i // (2 * n)) for i in range(n)])
    prefix = np.array([case["prefix"] - case["prefix"] * i // (2 * n) for i in range(n)])
    group = np.repeat(np.arange(n), size)
    r = np.arange(len(group))
    tail = case["tail"] - case["tail"] * 3 * r // (4 * len(r))
    return size, prefix, group, tail, np.maximum(1, case["q"] - r % 2)


def _visible(case):
    """Cache tokens that some query sees (those of a group's shared pages once), and (query, token) pairs."""
    size, prefix, group, tail, q = _batch(case)
    w, s = case["window"], case["sinks"]
    whole = prefix // case["page"] * case["page"]
    end = prefix[group] + tail + q
    pairs = tokens = 0
    for i in range(case["q"]):
        pos = (prefix[group] + tail + i)[i < q]
        first = np.maximum(pos - w + 1, 0) if w else 0 * pos
        pairs += int((pos + 1 - first + np.minimum(first, s)).sum())
    low = np.maximum(prefix[group] + tail - w + 1, 0) if w else 0 * end   # the first token that a request's queries see
    own_low = np.maximum(low, whole[group])
    tokens += int((end - own_low).sum())
    for g in range(len(size)):
        lo = int(low[group == g].min())
        tokens += max(0, int(whole[g]) - lo) + min(lo, s)
    return tokens, pairs


def work(case):
    if case["op"] == "norm":
        t, k = case["tokens"], case["width"]
        e, r = (4 if case[x] == "f32" else 2 for x in ("type", "resid"))
        rows = e + 2 * r + (e if case["gate"] == "rows" else 0) + (e if case["float"] else 0)
        weights = 4 * k * sum({"none": 0, "rms": 1, "layer": 2}[case[x]] for x in ("post", "pre"))
        # the q8_1 rows are written, and read back as bf16 values
        back = t * k * (36 / 32 + 36 / 32 + 2) if case["q8"] else 0
        return {"bytes": t * k * rows + weights + back, "flops": 16 * t * k}
    e = 4 if case["type"] == "f32" else 2
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        t = case["tokens"]
        axes = [int(x) for x in case["sections"].split(",")]
        # q, k, v and the table's rows in; q and the packed rows out; the rows read back as bf16 values
        row = (2 * h + 2 * hk) * d * e + 8 * sum(axes) + 2 * hk * d * 18 // 32 + 8 + 4 * len(axes)
        return {"bytes": t * (row + 2 * hk * d * 18 // 32 + 4 * hk * d), "flops": t * (h + hk) * d * 8}
    tokens, pairs = _visible(case)
    return {"bytes": tokens * hk * d * 36 // 32 + 2 * int(_batch(case)[4].sum()) * h * d * e, "flops": 4 * d * h * pairs}


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


_POSITIONS = 32768


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = np.random.default_rng(seed)
    typ = _TYPES[case["type"]]
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
    if case["op"] == "norm":
        t, k, resid = case["tokens"], case["width"], _TYPES[case["resid"]]
        weight = lambda kind: (1 + 0.1 * normal(k)) if kind != "none" else None  # noqa: E731
        bias = lambda kind: 0.1 * normal(k) if kind == "layer" else None  # noqa: E731
        gate = {"none": None, "rows": (t, k), "row": (k,)}[case["gate"]]
        empty = lambda on, t_, *shape: torch.empty(*shape, dtype=t_, device=dev) if on else None  # noqa: E731
        return {"case": case, "x": (normal(t, k) * 0.7 + 0.1).to(typ),
                "h": (normal(t, k) * (0.5 + 2 * torch.rand(t, 1, generator=gen, device=dev))).to(resid),
                "gate": normal(*gate).to(typ) if gate else None,
                "post": (weight(case["post"]), bias(case["post"])), "pre": (weight(case["pre"]), bias(case["pre"])),
                "h_out": torch.empty(t, k, dtype=resid, device=dev), "z": empty(case["float"], typ, t, k),
                "zq": empty(case["q8"], torch.uint8, t, k // 32 * 36),
                "values": empty(case["q8"], torch.bfloat16, t, k)}
    d, hk, h, page = case["dim"], case["kv_heads"], case["heads"], case["page"]
    if case["op"] == "rope":
        t = case["tokens"]
        axes = [int(x) for x in case["sections"].split(",")]
        qkv = (normal(t, (h + 2 * hk) * d) * 1.5).to(typ)   # one fused projection's rows
        pages = -(-t // page) + 3
        cache = torch.zeros(pages, hk * page * d * 18 // 16, dtype=torch.uint8, device=dev)
        # consecutive slots of pages in any order
        at = torch.randperm(pages, generator=gen, device=dev)
        tok = torch.arange(t, device=dev)
        slots = at[tok // page] * page + tok % page
        # some text, whose axes are equal, then patches of images of 53 x 37: frame, row and column
        first, text = int(rnd.integers(0, _POSITIONS - 2 * t - 64)), t // 8
        patch = tok - text
        grid = [patch // (53 * 37), patch // 37 % 53, patch % 37, patch % 7]
        pos = torch.stack([torch.where(patch < 0, tok, text + grid[i]) for i in range(len(axes))]) + first
        weight = lambda: (1 + 0.1 * normal(d)) if case["norm"] else None  # noqa: E731
        return {"case": case, "sections": tuple(axes), "q": qkv[:, :h * d].view(t, h, d),
                "k": qkv[:, h * d:(h + hk) * d].view(t, hk, d), "v": qkv[:, (h + hk) * d:].view(t, hk, d),
                "qw": weight(), "kw": weight(), "pos": pos.to(torch.int32), "slots": slots,
                "table": _cos_sin(_POSITIONS, 2 * sum(axes), dev), "cache": cache,
                "out": torch.empty(t, h, d, dtype=typ, device=dev),
                "kv": [torch.empty(t, hk, d, dtype=torch.bfloat16, device=dev) for _ in range(2)]}
    size, prefix, group, tail, q = _batch(case)
    order = rnd.permutation(len(q))   # which request is how long; the groups stay in place
    tail, q = tail[order], q[order]
    kv = prefix[group] + tail + q
    shared, counts = prefix // page, -(-kv // page)
    pages = int(shared.sum() + (counts - shared[group]).sum()) + 5
    cache = _cache(pages, hk, d, page, gen, dev)
    at = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).cpu().numpy()
    table = np.full((len(q), int(counts.max())), -1, dtype=np.int32)
    used = 0
    for g in range(len(size)):   # every request's row lists all its pages
        table[group == g, :shared[g]] = at[used:used + shared[g]]
        used += int(shared[g])
    for r in range(len(q)):
        n = int(counts[r] - shared[group[r]])
        table[r, shared[group[r]]:counts[r]] = at[used:used + n]
        used += n
    ints = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).to(dev)  # noqa: E731
    x = (normal(int(q.sum()), h, d) * 2).to(typ)
    return {"case": case, "q": x, "cache": cache, "table": ints(table), "start": ints(np.r_[0, np.cumsum(q)]),
            "kv_len": ints(kv), "group_start": ints(np.r_[0, np.cumsum(size)]), "prefix": ints(prefix),
            "max_q": int(q.max()), "most": (int(size.max()), int(shared.max()), int((counts - shared[group]).max())),
            "out": torch.empty_like(x)}


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
    if c["op"] == "norm":
        kinds = {"none": g.NORM_NONE, "rms": g.NORM_RMS, "layer": g.NORM_LAYER}
        h, z, zq = g.gguf_block_norm(s["x"], s["h"], gate=s["gate"], gate_act=g.GATE_SIGMOID, branch_scale=0.75,
                                     post_kind=kinds[c["post"]], post_weight=s["post"][0], post_bias=s["post"][1],
                                     pre_kind=kinds[c["pre"]], pre_weight=s["pre"][0], pre_bias=s["pre"][1],
                                     eps=_EPS, residual_out=s["h_out"], out=s["z"], out_q8_1=s["zq"])
        if zq is not None:
            zq = g.gguf_dequantize(zq, g.Q8_1, c["tokens"], c["width"], out=s["values"])
        return {"h": h, "z": z, "q8": zq}
    if c["op"] == "rope":
        q = g.gguf_qk_norm_mrope(s["q"], s["k"], s["v"], s["qw"], s["kw"], _EPS, s["pos"], s["table"], s["sections"],
                                 c["mixed"], g.ROPE_NEOX if c["neox"] else g.ROPE_NORM, cache=s["cache"],
                                 slots=s["slots"], page_size=c["page"], q_out=s["out"])
        k, v = g.gguf_kv_get_rows(s["cache"], s["slots"], c["kv_heads"], c["dim"], c["page"], out=s["kv"])
        return {"q": q, "k": k, "v": v}
    plan = g.gguf_prefix_plan(s["start"], s["kv_len"], s["group_start"], s["prefix"], c["page"], s["q"].shape[0])
    return g.gguf_prefix_attention(s["q"], s["cache"], s["table"], plan, s["prefix"].numel(), c["kv_heads"], c["page"],
                                   s["max_q"], c["dim"] ** -0.5, window=c["window"], sinks=c["sinks"], out=s["out"])


# ---------------------------------------------------------------------------- plain forms

def _plain_normed(x, kind, weight, bias):
    if kind == "none":
        return x
    if kind == "rms":
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * weight
    x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * weight + bias


def _plain_q8(z):
    """Values as q8_1 holds them: blocks of 32, d = largest magnitude / 127, held in fp16; codes round half away from
    zero."""
    b = z.reshape(z.shape[0], -1, 32)
    d = b.abs().amax(-1, keepdim=True) / 127
    c = torch.where(d == 0, torch.zeros_like(b), b / d)
    whole = c.trunc()
    c = whole + ((c - whole).abs() >= 0.5) * c.sign()
    return (d.to(torch.float16).float() * c).reshape(z.shape)


def _plain_norm(s):
    c = s["case"]
    y = _plain_normed(s["x"].float(), c["post"], *s["post"])
    if s["gate"] is not None:
        y = y / (1 + torch.exp(-s["gate"].float()))
    h = s["h"].float() + 0.75 * y
    z = _plain_normed(h, c["pre"], *s["pre"])
    return {"h": h.to(s["h"].dtype), "z": z.to(s["x"].dtype) if c["float"] else None,
            "q8": _plain_q8(z).to(torch.bfloat16) if c["q8"] else None}


def _axis_of(sections, mixed, device):
    """The axis of each pair: sections one after another, or in turn while they have pairs left."""
    n = torch.tensor(sections, device=device)
    axis = torch.repeat_interleave(torch.arange(len(sections), device=device), n)
    if not mixed:
        return axis
    turn = torch.arange(axis.numel(), device=device) - (n.cumsum(0) - n)[axis]   # how often its axis had its turn
    return axis[torch.argsort(turn * len(sections) + axis)]


def _plain_head_norm(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w


def _plain_rotate(x, cos, sin, neox):
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    r = x[..., :2 * half]
    a, b = (r[..., :half], r[..., half:]) if neox else (r[..., 0::2], r[..., 1::2])
    y, z = a * cos - b * sin, b * cos + a * sin
    r = torch.cat([y, z], -1) if neox else torch.stack([y, z], -1).flatten(-2)
    return torch.cat([r, x[..., 2 * half:]], -1)


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
    axis = _axis_of(s["sections"], c["mixed"], s["pos"].device)
    i = torch.arange(axis.numel(), device=axis.device)
    at = s["pos"].long()[axis].T   # of each token and pair
    cos, sin = s["table"][at, i], s["table"][at, i + axis.numel()]
    q = _plain_rotate(_plain_head_norm(s["q"].float(), s["qw"]), cos, sin, c["neox"])
    k = _plain_rotate(_plain_head_norm(s["k"].float(), s["kw"]), cos, sin, c["neox"])
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


def _plain_pages(s, at):
    """Keys [n, hk, d, tokens] and values [n, hk, tokens, d] of the pages at [n, width]."""
    c = s["case"]
    d, hk, page = c["dim"], c["kv_heads"], c["page"]
    n, width = at.shape
    k, v = _plain_unpack(s["cache"][at.clamp(min=0).long().flatten()].view(-1, 18 * d), d)
    k = k.view(n, width, hk, page, d).permute(0, 2, 4, 1, 3).reshape(n, hk, d, width * page)
    return k, v.view(n, width, hk, page, d).permute(0, 2, 1, 3, 4).reshape(n, hk, width * page, d)


def _plain_scores(s, q, k, pos, j, end):
    """Scores of queries [n, hk, group x m, d] at positions pos [n, m] with keys at positions j [n, tokens] before end [n]."""
    c = s["case"]
    score = torch.matmul(q, k).mul_(c["dim"] ** -0.5)
    hide = (j[:, None] > pos[..., None]) | (j >= end[:, None])[:, None]
    if c["window"]:
        hide |= (j[:, None] <= pos[..., None] - c["window"]) & (j >= c["sinks"])[:, None]
    n, m, tokens = hide.shape
    return score.view(n, q.shape[1], -1, m, tokens).masked_fill_(hide[:, None, None], -math.inf)


def _plain_attn(s):
    c = s["case"]
    d, hk, h, page = c["dim"], c["kv_heads"], c["heads"], c["page"]
    x, dev, lq = s["q"], s["q"].device, s["max_q"]
    members, shared, tail = s["most"]
    start, first = s["start"].long(), s["group_start"].long()
    n, t = s["kv_len"].numel(), x.shape[0]
    length, kv = start[1:] - start[:-1], s["kv_len"].long()
    group = torch.searchsorted(first, torch.arange(n, device=dev), right=True) - 1
    whole = s["prefix"].long() // page
    i = torch.arange(lq, device=dev)[None]
    rows = (start[:-1, None] + i).clamp(max=t - 1)
    pos = (kv - length)[:, None] + i
    qs = x[rows].float().view(n, lq, hk, h // hk, d).permute(0, 2, 3, 1, 4)   # [n, hk, h / hk, lq, d]
    # every request's own pages
    col = whole[group][:, None] + torch.arange(tail, device=dev)
    k, v = _plain_pages(s, s["table"].gather(1, col.clamp(max=s["table"].shape[1] - 1)))
    j = whole[group][:, None] * page + torch.arange(tail * page, device=dev)
    score = _plain_scores(s, qs.reshape(n, hk, -1, d), k, pos, j, kv)
    v.masked_fill_((j >= kv[:, None])[:, None, :, None], 0)
    top = score.amax(-1, keepdim=True)
    if shared:   # the groups' pages, for the queries of all their requests at once
        m = first[:-1, None] + torch.arange(members, device=dev)
        m = m.clamp(max=n - 1)
        gk, gv = _plain_pages(s, s["table"][first[:-1], :shared])
        gj = torch.arange(shared * page, device=dev)[None].expand(m.shape[0], -1)
        gq = qs[m].permute(0, 2, 3, 1, 4, 5)   # [groups, hk, h / hk, members, lq, d]
        gscore = _plain_scores(s, gq.reshape(m.shape[0], hk, -1, d), gk, pos[m].flatten(1), gj, whole * page)
        mine = torch.arange(n, device=dev) - first[group]   # place in the group
        back = lambda a: a.view(*a.shape[:3], members, lq, -1)[group, :, :, mine]  # noqa: E731
        top = torch.maximum(top, back(gscore.amax(-1, keepdim=True)))
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = score.sub_(base).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, hk, -1, tail * page), v).view(n, hk, h // hk, lq, d)
    if shared:
        gbase = base[m].permute(0, 2, 3, 1, 4, 5).reshape(*gscore.shape[:4], 1)
        p = gscore.sub_(gbase).exp_()
        total = total + back(p.sum(-1, keepdim=True))
        go = torch.matmul(p.view(m.shape[0], hk, -1, shared * page), gv).view(m.shape[0], hk, h // hk, -1, d)
        o = o + back(go)
    o = torch.where(total == 0, torch.zeros_like(o), o / total)
    tok = torch.arange(t, device=dev)
    req = torch.searchsorted(start, tok, right=True) - 1
    return o[req, :, :, tok - start[req]].reshape(t, h, d).to(x.dtype)


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "rope": _plain_rope, "attn": _plain_attn}[state["case"]["op"]](state)


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


def _exact_norm(s, case):
    def normed(x, kind, wb):
        if kind == "none":
            return x
        weight = wb[0].double()
        if kind == "rms":
            return weight * x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + _EPS).sqrt()
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        return weight * (x - mean) / (var + _EPS).sqrt() + wb[1].double()

    y = normed(s["x"].double(), case["post"], s["post"])
    if s["gate"] is not None:
        y = y * torch.sigmoid(s["gate"].double())
    h = s["h"].double() + y * 3 / 4
    z = normed(h, case["pre"], s["pre"])
    held = None
    if case["q8"]:
        b = z.unflatten(-1, (-1, 32))
        d = b.abs().max(-1, keepdim=True).values / 127
        held = (d.half().double() * b.sign() * torch.floor(b.abs() / d + 0.5)).flatten(-2)
    return {"h": h, "z": z if case["float"] else None, "q8": held}


def _exact_rope(s, case):
    sections = s["sections"]
    half = sum(sections)
    # pair -> axis, one at a time
    axis, left = [], list(sections)
    while len(axis) < half:
        for a in range(len(left)):
            n = min(left[a], 1 if case["mixed"] else left[a])
            axis += [a] * n
            left[a] -= n
    cs = torch.stack([s["table"][s["pos"][a].long()][:, [i, half + i]] for i, a in enumerate(axis)], -1).double()
    first = torch.arange(half, device="cuda") * (1 if case["neox"] else 2)
    second = first + (half if case["neox"] else 1)

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.square().sum(-1, keepdim=True) / case["dim"] + _EPS).sqrt() * w.double()
        y = x.clone()
        cos, sin = cs[:, :1], cs[:, 1:]
        y[..., first] = x[..., first] * cos - x[..., second] * sin
        y[..., second] = x[..., first] * sin + x[..., second] * cos
        return y

    def held(x):
        x = x.unflatten(-1, (-1, 32))
        scale = (torch.take_along_dim(x, x.abs().max(-1, keepdim=True).indices, -1) / -8).half().double()
        steps = x / scale
        return (scale * (steps.sign() * torch.floor(steps.abs() + 0.5)).clamp(-8, 7)).flatten(-2)

    return {"q": turned(s["q"], s["qw"]), "k": held(turned(s["k"], s["kw"])), "v": held(s["v"].double())}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "rope":
        return _exact_rope(s, case)
    d, hk, page = case["dim"], case["kv_heads"], case["page"]
    g = case["heads"] // hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, lens, bounds = s["start"].tolist(), s["kv_len"].tolist(), s["group_start"].tolist()
    for r0, r1, prefix in zip(bounds, bounds[1:], s["prefix"].tolist()):
        whole = prefix // page * page
        for head in range(hk):
            at = lambda r, a, b: (s["table"][r].long()[torch.arange(a, b, device="cuda") // page] * page  # noqa: E731
                                  + torch.arange(a, b, device="cuda") % page)
            shared = _exact_rows(s["cache"], at(r0, 0, whole), head, d, page, hk)
            for r in range(r0, r1):
                a, e, n = starts[r], starts[r + 1], lens[r]
                mine = _exact_rows(s["cache"], at(r, whole, n), head, d, page, hk)
                k, v = (torch.cat(p) for p in zip(shared, mine))
                x = s["q"][a:e, head * g:(head + 1) * g].double().transpose(0, 1)
                p, tok = torch.arange(n - e + a, n, device="cuda")[:, None], torch.arange(n, device="cuda")
                see = tok <= p
                if case["window"]:
                    see &= (tok > p - case["window"]) | (tok < case["sinks"])
                score = torch.where(see, x @ k.T / math.sqrt(d), -math.inf)
                out[a:e, head * g:(head + 1) * g] = (torch.softmax(score, -1) @ v).transpose(0, 1)
    return out
