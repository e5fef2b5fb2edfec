"""The paged Q4_0 cache operators on the GPU against plain evaluations in 64 bits."""
import numpy as np
import pytest
import torch

import gguf_block_quantized_quantize_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# half a unit in the last place, relative: significands of 24, 11 and 8 bits
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


# ------------------------------------------------------------------ plan

def plan_ref(ctx, new, free, table, page, n_tokens):
    table = table.copy()
    width = table.shape[1]
    pos, slots, start, used, lost = [], [], [0], 0, 0
    for r, (c, n) in enumerate(zip(np.maximum(ctx, 0), np.maximum(new, 0))):
        had, has = min(-(-c // page), width), min(-(-(c + n) // page), width)
        for i in range(had, has):
            table[r, i] = free[used] if used < len(free) else -1
            used += 1
        for p in range(c, c + n):
            pos.append(p)
            pg = table[r, p // page] if p // page < width else -1
            slots.append(pg * page + p % page if pg >= 0 else -1)
        start.append(start[-1] + n)
    lost = max(0, len(pos) - n_tokens) + sum(s < 0 for s in slots[:n_tokens])
    pad = n_tokens - len(pos)
    pos, slots = (a[:n_tokens] + [-1] * pad for a in (pos, slots))
    kv = np.maximum(ctx, 0) + np.maximum(new, 0)
    return np.array(start), kv, np.array(pos), np.array(slots), min(used, len(free)), table, lost


@pytest.mark.parametrize("r, ctx_max, new_max, page, width, short, pad, seed", [
    (1, 0, 1, 16, 4, 0, 0, 0), (1, 50, 1, 16, 4, 0, 3, 1), (3, 40, 5, 16, 3, 0, 0, 2), (7, 100, 30, 48, 3, 0, 11, 3),
    (64, 500, 2, 64, 8, 0, 0, 4), (513, 900, 40, 32, 30, 0, 100, 5), (700, 60, 3, 16, 2, 0, 0, 6),
    (9, 64, 64, 16, 8, 5, 0, 7), (9, 64, 64, 16, 8, 1000, -50, 8), (5000, 300, 2, 16, 19, 0, 77, 9),
    (16384, 20, 2, 16, 2, 0, 0, 10), (0, 1, 1, 16, 2, 0, 5, 11)])
def test_plan(r, ctx_max, new_max, page, width, short, pad, seed):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, ctx_max + 1, r), rng.integers(0, new_max + 1, r)   # zero lengths among them
    if r > 5:
        new[3], ctx[4] = -4, -1
    need = sum(max(0, min(-(-(max(c, 0) + max(n, 0)) // page), width) - min(-(-max(c, 0) // page), width))
               for c, n in zip(ctx, new))
    free = rng.permutation(1 << 20)[:max(0, need + 3 - short)].astype(np.int32)
    table = rng.integers(0, 1 << 20, (r, width + 2)).astype(np.int32)[:, :width]   # rows with a wider stride
    n_tokens = max(0, int(np.maximum(new, 0).sum()) + pad)
    start, kv, pos, slots, used, ref_table, lost = plan_ref(ctx, new, free, table, page, n_tokens)
    wide = torch.full((r, width + 2), 77, dtype=torch.int32, device=DEV)
    t = wide[:, :width]
    t.copy_(torch.from_numpy(np.ascontiguousarray(table)))
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)   # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for again in range(2):   # the second call finds its own pages in the table: the same answer
        out = g.gguf_kv_plan(to(ctx), to(new), to(free), t, page, n_tokens, dev_status=status)
        got = [x.cpu().numpy() for x in out]
        assert np.array_equal(got[0], start) and np.array_equal(got[1], kv)
        assert np.array_equal(got[2], pos) and np.array_equal(got[3], slots)
        assert got[4][0] == used and np.array_equal(t.cpu().numpy(), ref_table)
        assert int(status.item()) == lost * (again + 1)
    assert bool((wide[:, width:] == 77).all())


def test_plan_large_slots():
    """Slots past 32 bits."""
    free = torch.tensor([2 ** 31 - 1, 5], dtype=torch.int32, device=DEV)
    table = torch.full((1, 2), -1, dtype=torch.int32, device=DEV)
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device=DEV)   # noqa: E731
    _, _, _, slots, _ = g.gguf_kv_plan(i32(0), i32(130), free, table, 128, 130)
    assert slots[127].item() == (2 ** 31 - 1) * 128 + 127 and slots[128].item() == 5 * 128


# ------------------------------------------------------------------ norms, rotation, store

def rope_ref(x, w, cs, rot, neox, eps):
    x = x.double().cpu()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double().cpu()
    half = rot // 2
    i = torch.arange(half) * (1 if neox else 2)
    j = i + (half if neox else 1)
    y = x.clone()
    c, s = cs[:, None, :half], cs[:, None, half:2 * half]
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


@pytest.mark.parametrize("d, h, hk, t, typ, rot, neox, norm, page, offset", [
    (64, 4, 4, 1, "bf16", 64, True, True, 16, 0), (64, 6, 2, 33, "f16", 32, False, True, 32, 0),
    (128, 24, 8, 1, "f32", 128, False, True, 16, 0), (128, 3, 1, 19, "bf16", 128, True, False, 48, 0),
    (128, 7, 1, 130, "bf16", 16, True, True, 64, 1), (256, 16, 2, 5, "f16", 64, True, True, 16, 0),
    (256, 4, 4, 50, "f32", 256, False, True, 128, 3), (256, 1, 1, 17, "bf16", 0, False, True, 16, 0),
    (64, 32, 8, 700, "bf16", 48, True, True, 16, 0), (128, 32, 8, 300, "f32", 64, True, True, 16, 0)])
def test_norm_rope_store(orc, d, h, hk, t, typ, rot, neox, norm, page, offset):
    torch.manual_seed(d + t)
    dtype, eps, npos = DTYPES[typ], 1e-6, 1000
    row = (h + 2 * hk) * d + 8
    fused = torch.randn(t * row + offset, device=DEV).mul_(2).to(dtype)[offset:].view(t, row)
    q, k, v = (fused[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, h), (h, h + hk), (h + hk, h + 2 * hk)))
    qw, kw = ((1 + 0.2 * torch.randn(d, device=DEV)) if norm else None for _ in range(2))
    ang = torch.rand(npos, max(rot // 2, 1), dtype=torch.float64) * 6.28
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, npos, (t,), dtype=torch.int32)
    pages = t // page + 3
    slots = torch.randperm(pages * page)[:t]
    if t > 10:
        pos[3], slots[5] = -1, -1          # a padding token; a token that is not stored
    cache = torch.full((pages, g.gguf_kv_page_bytes(d, hk, page)), 0xA5, dtype=torch.uint8, device=DEV)
    before = cache.clone()
    q_out, k_out = (torch.full((t, n, d), 7.0, dtype=dtype, device=DEV) for n in (h, hk))
    g.gguf_qk_norm_rope(q, k, v, qw, kw, eps, pos.to(DEV), table.to(DEV) if rot else None,
                        g.ROPE_NEOX if neox else g.ROPE_NORM, cache=cache, slots=slots.to(DEV), page_size=page,
                        q_out=q_out, k_out=k_out)
    cs = table.double()[pos.clamp(min=0).long()]
    done = pos >= 0
    for got, x, w in ((q_out, q, qw), (k_out, k, kw)):
        ref = rope_ref(x, w, cs, rot, neox, eps)
        got = got.double().cpu()
        # fp32: the norm's sum of d terms, four roundings, the rotation's three on terms up to |a| + |b|;
        # one rounding to the output type
        size = ref.abs() + ref.norm(dim=-1, keepdim=True) / np.sqrt(d) * 8
        tol = HALF_ULP[typ] * ref.abs() + 16 * 2.0 ** -24 * size
        assert bool(((got - ref).abs() <= tol)[done].all())
        assert bool((got[~done] == 7).all())
    # the stored blocks are Q4_0 of exactly these fp32 values: fp32 inputs show them as k_out
    kept = done & (slots >= 0)
    gk, gv = g.gguf_kv_get_rows(cache, slots.to(DEV), hk, d, page)
    held = lambda x: torch.from_numpy(orc.dequantize(orc.Q4_0, orc.quantize_weights(   # noqa: E731
        orc.Q4_0, x.reshape(-1, d).float().cpu().numpy()), d).astype(np.float32)).view(x.shape)
    assert torch.equal(gv.cpu()[kept], held(v)[kept])
    if typ == "f32":
        assert torch.equal(gk.cpu()[kept], held(k_out)[kept])
    else:   # a code may differ by one where the 16-bit output rounds across a code's border
        ref = rope_ref(k, kw, cs, rot, neox, eps)
        blocks = ref.unflatten(-1, (-1, 32))
        step = (blocks.abs().amax(-1, keepdim=True) / 8).expand(blocks.shape).flatten(-2)
        assert bool(((gk.double().cpu() - ref).abs() <= step * 1.01 + 1e-6)[kept].all())
    assert bool((gv[slots < 0] == 0).all()) and bool((gk[slots < 0] == 0).all())
    # nothing else of the cache was touched: rows of the other slots still decode as before
    others = torch.tensor([s for s in range(pages * page) if s not in set(slots[kept].tolist())], device=DEV)
    for a, b in zip(g.gguf_kv_get_rows(cache, others, hk, d, page), g.gguf_kv_get_rows(before, others, hk, d, page)):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_rope_in_place_and_queries_only():
    torch.manual_seed(1)
    q = torch.randn(9, 4, 128, device=DEV, dtype=torch.bfloat16)
    ang = torch.rand(40, 64, device=DEV) * 6
    table, pos = torch.cat([ang.cos(), ang.sin()], 1), torch.arange(9, dtype=torch.int32, device=DEV)
    w = torch.rand(128, device=DEV) + 0.5
    ref = g.gguf_qk_norm_rope(q, None, None, w, None, 1e-6, pos, table)
    got = q.clone()
    assert g.gguf_qk_norm_rope(got, None, None, w, None, 1e-6, pos, table, q_out=got) is got
    assert torch.equal(got, ref)
    k = torch.randn(9, 2, 128, device=DEV, dtype=torch.bfloat16)
    k_out = torch.empty_like(k)
    g.gguf_qk_norm_rope(q, k, None, w, w, 1e-6, pos, table, k_out=k_out)
    assert torch.equal(k_out, g.gguf_qk_norm_rope(k, None, None, w, None, 1e-6, pos, table))


def test_store_edge_values(orc):
    """Zero blocks, a scale that rounds to zero, ties of magnitude, the largest magnitude, and counters."""
    d, page = 64, 16
    v = torch.zeros(6, 1, d, device=DEV)
    v[1] = 1e-9
    v[2, 0, :32] = torch.tensor([3.0, -3.0] * 16)
    v[2, 0, 32:] = torch.tensor([-3.0, 3.0] * 16)
    v[3] = torch.linspace(-65000, 65000, d)
    v[4] = torch.randn(d) * 1e-6
    k = torch.randn(6, 1, d, device=DEV)
    cache = torch.zeros(1, g.gguf_kv_page_bytes(d, 1, page), dtype=torch.uint8, device=DEV)
    slots = torch.tensor([15, 3, 4, 5, 0, 16], device=DEV)      # the last is past the cache
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos = torch.tensor([0, 1, 2, 3, 9, 0], dtype=torch.int32, device=DEV)
    table = torch.cat([torch.ones(9, 32), torch.zeros(9, 32)], 1).to(DEV)
    g.gguf_qk_norm_rope(k, k, v, None, None, 0.0, pos, table, cache=cache, slots=slots, page_size=page, dev_status=status)
    assert status.item() == 2          # a position past the table, a slot past the cache
    gk, gv = g.gguf_kv_get_rows(cache, slots, 1, d, page)
    ref = torch.from_numpy(orc.dequantize(orc.Q4_0, orc.quantize_weights(orc.Q4_0, v[:, 0].cpu().numpy()), d).astype(np.float32))
    assert bool((gv[:2] == 0).all()) and torch.equal(gv[2:4, 0].cpu(), ref[2:4]) and bool((gv[4:] == 0).all())
    assert bool((gk[4:] == 0).all())


# ------------------------------------------------------------------ attention

def attn_setup(q_lens, kv_lens, h, hk, d, page, typ, seed=0, spare_cols=0, peaky=2.0):
    """Random queries and cached tokens; slots that hold no token are full of NaN scales."""
    torch.manual_seed(seed)
    n = len(kv_lens)
    counts = [-(-max(k, 0) // page) for k in kv_lens]
    pages = sum(counts) + 2
    order = torch.randperm(pages).to(torch.int32)
    table = torch.full((n, max(counts + [1]) + spare_cols), -1, dtype=torch.int32)
    at = 0
    for r, c in enumerate(counts):
        table[r, :c] = order[at:at + c]
        at += c
    cache = torch.full((pages, g.gguf_kv_page_bytes(d, hk, page)), 0xFF, dtype=torch.uint8, device=DEV)
    slots = torch.cat([table[r, :].long().repeat_interleave(page)[:k] * page + torch.arange(k) % page
                       for r, k in enumerate(kv_lens) if k > 0] + [torch.zeros(0, dtype=torch.long)])
    total = slots.numel()
    kv = torch.randn(2, total, hk, d, device=DEV) * torch.rand(2, total, hk, 1, device=DEV).mul_(1.5)
    zero = torch.zeros(total, dtype=torch.int32, device=DEV)
    if total:
        g.gguf_qk_norm_rope(kv[0][:, :0], kv[0], kv[1], None, None, 0.0, zero, None, cache=cache, slots=slots.to(DEV),
                            page_size=page)
    k, v = g.gguf_kv_get_rows(cache, slots.to(DEV), hk, d, page)
    q = (torch.randn(sum(q_lens), h, d, device=DEV) * peaky).to(DTYPES[typ])
    start = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32, device=DEV)
    return q, cache, table.to(DEV), start, torch.tensor(kv_lens, dtype=torch.int32, device=DEV), k, v


def attn_ref(q, k, v, q_lens, kv_lens, scale, window, sinks):
    """fp64 outputs, and the sums that error bounds are made of: sum p |v|, max_j scale sum |q k| and sum |v|."""
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    t, h, d = q.shape
    hk = k.shape[1]
    out, size, total = (torch.zeros(t, h, d, dtype=torch.float64) for _ in range(3))
    reach = torch.zeros(t, h, 1, dtype=torch.float64)
    a = b = 0
    for n, m in zip(q_lens, kv_lens):
        for i in range(n):
            pos = m - n + i
            j = torch.arange(max(pos + 1, 0))
            if window:
                j = j[(j > pos - window) | (j < sinks)]
            if len(j) == 0:
                continue
            for head in range(h):
                kk, vv = k[b + j, head // (h // hk)], v[b + j, head // (h // hk)]
                p = torch.softmax(kk @ q[a + i, head] * scale, 0)
                out[a + i, head], size[a + i, head] = p @ vv, p @ vv.abs()
                total[a + i, head] = vv.abs().sum(0)
                reach[a + i, head] = (kk.abs() @ q[a + i, head].abs()).max() * scale
        a, b = a + n, b + max(m, 0)
    return out, size, reach, total


def check_attn(got, refs, typ):
    """fp32: about 2^-21 from split operands, fp32 sums and the exponential of scores as large as `reach`.
    16 bits: p and v rounded to 11 bits each (2^-11 + 2^-11 of the terms), keys rounded to 11 bits move a
    score by at most 2^-12 reach, hence a probability and the sum by twice that; one rounding to the type (fp16
    below 2^-14: multiples of 2^-24). Probabilities go into the products as fp16 numbers of up to 2^10 times
    their value, which are multiples of 2^-24: 2^-35 of the row's largest at most is lost of each."""
    ref, size, reach, total = refs
    got = got.double().cpu()
    assert bool(torch.isfinite(got).all())
    if typ == "f32":
        tol = 2.0 ** -20 * size * (1 + reach)
    else:
        tol = HALF_ULP[typ] * ref.abs() * 1.01 + size * (2.0 ** -10 + 2.0 ** -11 * reach + 2.0 ** -20 * (1 + reach))
    tol = tol + 2.0 ** -34 * total
    if typ == "f16":
        tol = tol + 2.0 ** -25
    err = (got - ref).abs()
    assert bool((err <= tol + 1e-30).all()), f"worst {float((err / (tol + 1e-30)).max())}"
    # and in the mean: errors of 2^-12 relative (uniform) per operand leave a row within a few of them
    norm = float(ref.norm()) + 1e-30
    assert float(err.norm()) / norm <= {"f32": 4e-6, "f16": 2e-3, "bf16": 4e-3}[typ]


CASES = [
    # q_lens, kv_lens, h, hk, d, page, type, window, sinks
    ([1], [1], 4, 4, 64, 16, "bf16", 0, 0),
    ([1], [0], 2, 1, 128, 16, "f16", 0, 0),
    ([1, 0, 1], [333, 40, 17], 24, 8, 128, 16, "f32", 0, 0),
    ([1] * 5, [16, 15, 64, 65, 700], 8, 1, 128, 64, "bf16", 0, 0),
    ([1] * 3, [900, 1, 130], 16, 2, 256, 32, "bf16", 0, 0),
    ([1] * 3, [900, 31, 130], 32, 2, 128, 48, "f16", 0, 0),
    ([1] * 2, [600, 77], 40, 2, 64, 16, "bf16", 0, 0),
    ([1] * 4, [500, 64, 65, 3000], 8, 8, 64, 128, "f16", 64, 4),
    ([1] * 3, [513, 70, 2000], 12, 1, 128, 16, "bf16", 50, 20),
    ([1] * 3, [513, 70, 300], 6, 2, 256, 16, "f32", 33, 0),
    ([2, 3, 1], [200, 3, 513], 12, 4, 128, 16, "bf16", 0, 0),
    ([4, 1], [100, 1], 8, 2, 64, 32, "f32", 0, 0),
    ([3, 5], [2, 0], 4, 2, 64, 16, "bf16", 0, 0),           # more queries than tokens: rows that see nothing
    ([17], [17], 6, 2, 64, 16, "bf16", 0, 0),
    ([65, 1, 30], [65, 200, 140], 12, 4, 128, 16, "bf16", 0, 0),
    ([130], [300], 6, 2, 128, 64, "f16", 0, 0),
    ([150, 1], [150, 33], 8, 4, 64, 32, "bf16", 40, 4),
    ([200], [457], 4, 1, 128, 16, "bf16", 128, 16),
    ([70, 40], [70, 300], 4, 2, 256, 16, "bf16", 0, 0),
    ([90], [190], 4, 4, 256, 32, "f16", 50, 1),
    ([40, 33], [45, 33], 6, 3, 128, 16, "f32", 20, 2),
    ([257], [257], 2, 2, 128, 128, "bf16", 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_attention(case):
    q_lens, kv_lens, h, hk, d, page, typ, window, sinks = case
    q, cache, table, start, kv_len, k, v = attn_setup(q_lens, kv_lens, h, hk, d, page, typ, seed=len(CASES) + h + d)
    scale = d ** -0.5
    out = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, page, max(q_lens), scale, window=window, sinks=sinks)
    check_attn(out, attn_ref(q, k, v, q_lens, kv_lens, scale, window, sinks), typ)
    again = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, page, max(q_lens), scale, window=window, sinks=sinks)
    assert torch.equal(out, again)


def test_attention_strides_and_padding():
    """Rows with a stride, offset bases, a wider table, padding tokens after the last request."""
    q_lens, kv_lens, h, hk, d, page = [1, 2], [100, 61], 4, 2, 128, 16
    q, cache, table, start, kv_len, k, v = attn_setup(q_lens, kv_lens, h, hk, d, page, "bf16", spare_cols=3)
    wide = torch.zeros(5 * (h * d + 11) + 1, dtype=torch.bfloat16, device=DEV)[1:].view(5, h * d + 11)
    wide[:3, :h * d] = q.view(3, h * d)
    out = torch.full_like(wide, 9.0)
    g.gguf_paged_attention(wide[:, :h * d].unflatten(1, (h, d)), cache, table, start, kv_len, hk, page, 2, d ** -0.5,
                           out=out[:, :h * d].unflatten(1, (h, d)))
    check_attn(out[:3, :h * d].unflatten(1, (h, d)), attn_ref(q, k, v, q_lens, kv_lens, d ** -0.5, 0, 0), "bf16")
    assert bool((out[3:] == 9).all()) and bool((out[:, h * d:] == 9).all())


@pytest.mark.parametrize("q_len", [1, 80])
def test_attention_pages_outside_the_cache(q_len):
    """Page numbers outside the cache hide their tokens, and are counted."""
    h, hk, d, page = 4, 2, 64, 32
    q, cache, table, start, kv_len, k, v = attn_setup([q_len], [200], h, hk, d, page, "bf16")
    table[0, 1], table[0, 4] = -1, cache.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, page, q_len, 0.125, dev_status=status)
    assert status.item() > 0
    keep = torch.tensor([j for j in range(200) if j // page not in (1, 4)])
    ref = torch.zeros(q_len, h, d, dtype=torch.float64)
    qd, kd, vd = q.double().cpu(), k.double().cpu(), v.double().cpu()
    for i in range(q_len):
        j = keep[keep <= 200 - q_len + i]
        for head in range(h):
            ref[i, head] = torch.softmax(kd[j, head // 2] @ qd[i, head] * 0.125, 0) @ vd[j, head // 2]
    assert float((out.double().cpu() - ref).norm() / ref.norm()) <= 4e-3


@pytest.mark.parametrize("typ", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("q_len", [1, 60])
def test_attention_ranges(typ, q_len):
    """Scores of hundreds, tiny and huge values: no overflow, no loss."""
    h, hk, d, page = 4, 2, 128, 16
    for peaky, size in ((60.0, 1.0), (1e-3, 1.0), (2.0, 1e-4), (2.0, 2e4)):
        q, cache, table, start, kv_len, k, v = attn_setup([q_len], [300], h, hk, d, page, typ, peaky=peaky)
        slots = (table[0].long().repeat_interleave(page) * page + torch.arange(table.shape[1] * page, device=DEV) % page)[:300]
        v2 = torch.randn(300, hk, d, device=DEV).clamp(-3, 3) * size
        if typ == "f16" and size > 1e4:
            v2 = v2.clamp(-6e4, 6e4)
        zero = torch.zeros(300, dtype=torch.int32, device=DEV)
        g.gguf_qk_norm_rope(k[:, :0], k, v2, None, None, 0.0, zero, None, cache=cache, slots=slots, page_size=page)
        k2, v2 = g.gguf_kv_get_rows(cache, slots, hk, d, page)
        out = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, page, q_len, d ** -0.5)
        check_attn(out, attn_ref(q, k2, v2, [q_len], [300], d ** -0.5, 0, 0), typ)


def test_attention_streams_and_graph():
    """On a side stream, and replayed from a graph with other lengths in the same buffers."""
    h, hk, d, page = 8, 2, 128, 16
    q, cache, table, start, kv_len, k, v = attn_setup([1, 1], [600, 90], h, hk, d, page, "bf16")
    ref = attn_ref(q, k, v, [1, 1], [600, 90], d ** -0.5, 0, 0)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run = lambda: g.gguf_paged_attention(q, cache, table, start, kv_len, hk, page, 1, d ** -0.5, out=out)   # noqa: E731
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    check_attn(out, ref, "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run()
    kv_len[0] = 400
    graph.replay()
    torch.cuda.synchronize()
    kk, vv = torch.cat([k[:400], k[600:]]), torch.cat([v[:400], v[600:]])
    check_attn(out, attn_ref(q, kk, vv, [1, 1], [400, 90], d ** -0.5, 0, 0), "bf16")


def test_step_end_to_end():
    """Plan, store and attention of a prompt and then of single tokens agree with attention over all at once."""
    torch.manual_seed(3)
    h, hk, d, page, n = 4, 2, 64, 16, 2
    cap = 12
    cache = torch.zeros(cap, g.gguf_kv_page_bytes(d, hk, page), dtype=torch.uint8, device=DEV)
    table = torch.full((n, 6), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(cap, device=DEV).to(torch.int32)
    ang = torch.rand(100, 32, device=DEV) * 6
    cos_sin = torch.cat([ang.cos(), ang.sin()], 1)
    w = torch.rand(2, d, device=DEV) + 0.5
    ctx, lens, steps = [0, 0], [33, 20], []
    for step in range(4):
        new = lens if step == 0 else [1, 1]
        t = sum(new)
        q, k, v = (torch.randn(t, m, d, device=DEV).to(torch.bfloat16) for m in (h, hk, hk))
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)   # noqa: E731
        start, kv_len, pos, slots, used = g.gguf_kv_plan(i32(ctx), i32(new), free, table, page, t)
        free = free[used.item():].contiguous()
        q = g.gguf_qk_norm_rope(q, k, v, w[0], w[1], 1e-6, pos, cos_sin, cache=cache, slots=slots, page_size=page)
        out = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, page, max(new), d ** -0.5)
        ctx = [a + b for a, b in zip(ctx, new)]
        rows = [table[r].long().repeat_interleave(page)[:ctx[r]] * page + torch.arange(ctx[r], device=DEV) % page
                for r in range(n)]
        kk, vv = g.gguf_kv_get_rows(cache, torch.cat(rows), hk, d, page)
        check_attn(out, attn_ref(q, kk, vv, new, ctx, d ** -0.5, 0, 0), "bf16")


# ------------------------------------------------------------------ the binding, and all of it together

def test_binding_refuses_what_does_not_fit():
    h, hk, d, page = 4, 2, 64, 16
    q, cache, table, start, kv_len, k, v = attn_setup([1], [40], h, hk, d, page, "bf16")
    run = lambda **kw: g.gguf_paged_attention(*[kw.get(n, x) for n, x in (   # noqa: E731
        ("q", q), ("cache", cache), ("table", table), ("start", start), ("kv_len", kv_len))], kw.get("hk", hk), page, 1, 0.1,
        out=kw.get("out"), ws=kw.get("ws"))
    bad = [dict(q=q.cpu()), dict(q=q.to(torch.float64)), dict(q=q[0]), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
           dict(cache=cache[:, 1:]), dict(cache=cache.float()), dict(table=table.long()), dict(start=start.long()),
           dict(kv_len=kv_len.float()), dict(out=torch.empty_like(q, dtype=torch.float32)), dict(out=torch.empty_like(q)[:, :2]),
           dict(start=start[:1]), dict(hk=4)]
    for kw in bad:
        with pytest.raises(ValueError):
            run(**kw)
    with pytest.raises(g.GgufError) as e:
        run(ws=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5
    with pytest.raises(g.GgufError) as e:
        run(hk=3, cache=torch.zeros(2, g.gguf_kv_page_bytes(d, 3, page), dtype=torch.uint8, device=DEV))
    assert e.value.status == 3
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)   # noqa: E731
    with pytest.raises(ValueError):
        g.gguf_kv_plan(i32(2), i32(3), i32(4), torch.zeros(3, 4, dtype=torch.int32, device=DEV), 16, 1)
    with pytest.raises(ValueError):
        g.gguf_qk_norm_rope(q, k, v, None, None, 0.0, i32(1), None)                     # k of another dtype
    with pytest.raises(ValueError):
        g.gguf_qk_norm_rope(q, None, None, None, None, 0.0, i32(1), None, cache=cache)  # nothing to store
    with pytest.raises(ValueError):
        g.gguf_kv_get_rows(cache, kv_len, hk, d, page)                                  # slots must be int64
    assert torch.isfinite(run().float()).all()


def test_many_requests_and_heads():
    """More requests than a CTA has threads, of all lengths from none on; one query head per KV head."""
    n, h, hk, d, page = 700, 2, 2, 64, 16
    kv_lens = [int(x) for x in np.random.default_rng(0).integers(0, 40, n)]
    kv_lens[5] = 900
    q, cache, table, start, kv_len, k, v = attn_setup([1] * n, kv_lens, h, hk, d, page, "bf16")
    out = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, page, 1, 0.125)
    check_attn(out, attn_ref(q, k, v, [1] * n, kv_lens, 0.125, 0, 0), "bf16")


@pytest.mark.parametrize("typ, window", [("bf16", 0), ("f16", 700)])
def test_pieces_of_a_long_context(typ, window):
    """A context that many CTAs share, and one that ends inside their pieces."""
    q_lens, kv_lens, h, hk, d, page = [1, 1], [9001, 2500], 4, 1, 128, 64
    q, cache, table, start, kv_len, k, v = attn_setup(q_lens, kv_lens, h, hk, d, page, typ)
    out = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, page, 1, d ** -0.5, window=window, sinks=17 if window else 0)
    check_attn(out, attn_ref(q, k, v, q_lens, kv_lens, d ** -0.5, window, 17 if window else 0), typ)


def test_no_device_errors():
    assert g.gguf_device_errors() == 0


def test_example_attention_layer():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    out = mod.main(["--requests", "3", "--prompt", "150", "--steps", "5"])
    # the prompt, one step before the capture, and five replays
    assert out["context"] == [50 + 6, 100 + 6, 150 + 6] and out["lost"] == 0 and out["finite"]


@pytest.mark.parametrize("q_lens, kv_lens, h, hk, d, typ, window, sinks", [
    ([40], [3000], 4, 1, 128, "bf16", 0, 0),            # 40 rows x 4 heads, tokens cut into pieces
    ([70, 1, 33], [2100, 900, 1500], 4, 2, 64, "f16", 0, 0),
    ([90], [2500], 2, 1, 256, "bf16", 0, 0),
    ([150], [1900], 2, 2, 128, "bf16", 1100, 20),
    ([80, 200], [1400, 150], 2, 1, 64, "bf16", 0, 0),   # a request with fewer tokens than queries: blind rows, empty pieces
])
def test_pieces_of_a_long_chunk(q_lens, kv_lens, h, hk, d, typ, window, sinks):
    q, cache, table, start, kv_len, k, v = attn_setup(q_lens, kv_lens, h, hk, d, 16, typ)
    run = lambda: g.gguf_paged_attention(q, cache, table, start, kv_len, hk, 16, max(q_lens), d ** -0.5, window=window, sinks=sinks)   # noqa: E731
    out = run()
    check_attn(out, attn_ref(q, k, v, q_lens, kv_lens, d ** -0.5, window, sinks), typ)
    assert torch.equal(out, run())


@pytest.mark.parametrize("q, n, most, h, hk, d, typ, window, sinks", [
    (64, 20, 2100, 32, 8, 128, "bf16", 0, 0),
    (32, 40, 1300, 16, 2, 256, "f16", 0, 0),
    (61, 21, 2900, 32, 8, 64, "f16", 1500, 4),
])
def test_pieces_after_a_full_round(q, n, most, h, hk, d, typ, window, sinks):
    """A few row blocks more than SMs: the last ones are cut, the others are not."""
    q_lens = [q] * n
    kv_lens = [q - 5 if i == n - 2 else max(q, most * (i + 1) // n) for i in range(n)]   # one with fewer than its queries
    qs, cache, table, start, kv_len, k, v = attn_setup(q_lens, kv_lens, h, hk, d, 16, typ)
    run = lambda: g.gguf_paged_attention(qs, cache, table, start, kv_len, hk, 16, q, d ** -0.5, window=window, sinks=sinks)   # noqa: E731
    out = run()
    check_attn(out, attn_ref(qs, k, v, q_lens, kv_lens, d ** -0.5, window, sinks), typ)
    assert torch.equal(out, run())
