"""gguf_qk_norm_mrope (positions on several axes) against its formula in 64 bits, and against gguf_qk_norm_rope."""
import pytest
import torch

import gguf_block_quantized_quantize_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
EPS = 1e-6


def axes_of(sections, interleaved):
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            n = min(left[a], 1 if interleaved else left[a])
            out += [a] * n
            left[a] -= n
    return out


def ref(x, w, table, pos, sections, interleaved, neox):
    """64 bits, pair by pair."""
    x = x.double().cpu()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double().cpu()
    axis, half = axes_of(sections, interleaved), sum(sections)
    y, table = x.clone(), table.double().cpu()
    for i, a in enumerate(axis):
        c, s = (table[pos[a].clamp(min=0).long(), j][:, None] for j in (i, half + i))
        m, n = (i, i + half) if neox else (2 * i, 2 * i + 1)
        y[..., m] = x[..., m] * c - x[..., n] * s
        y[..., n] = x[..., n] * c + x[..., m] * s
    return y


def setup(t, h, hk, d, typ, sections, page, seed, npos=500, offset=0):
    torch.manual_seed(seed)
    row = (h + 2 * hk) * d + 8
    fused = torch.randn(t * row + offset, device=DEV).mul_(2).to(DTYPES[typ])[offset:].view(t, row)
    q, k, v = (fused[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, h), (h, h + hk), (h + hk, h + 2 * hk)))
    ang = torch.rand(npos, max(sum(sections), 1), dtype=torch.float64) * 6.28
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, npos, (len(sections), t + 3), dtype=torch.int32)[:, :t]   # rows with a wider stride
    pages = t // page + 2
    return q, k, v, table, pos, torch.randperm(pages * page)[:t], pages


CASES = [  # head size, heads, KV heads, tokens, type, sections, interleaved, neox, norm, page, first element
    (128, 24, 8, 1, "bf16", (16, 24, 24), False, True, True, 16, 0), (128, 4, 2, 37, "f32", (24, 20, 20), True, True, True, 32, 0),
    (64, 6, 2, 90, "f16", (8, 12, 12), True, False, True, 16, 0), (64, 4, 4, 21, "bf16", (1, 31), False, True, False, 16, 0),
    (256, 3, 1, 50, "f16", (16, 16), False, False, True, 48, 0), (256, 16, 2, 9, "f32", (5, 60, 63), True, True, True, 16, 0),
    (128, 7, 1, 300, "bf16", (7, 1, 30, 2), False, True, True, 64, 3), (128, 5, 5, 33, "f32", (7, 1, 30, 2), True, False, True, 16, 1),
    (128, 8, 8, 64, "bf16", (64,), False, True, True, 16, 0), (64, 2, 1, 40, "f16", (0, 32, 0, 0), True, True, True, 16, 0),
    (128, 32, 8, 900, "bf16", (24, 20, 20), True, True, True, 16, 0)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_mrope(case):
    d, h, hk, t, typ, sections, interleaved, neox, norm, page, offset = case
    q, k, v, table, pos, slots, pages = setup(t, h, hk, d, typ, sections, page, d + t, offset=offset)
    qw, kw = ((1 + 0.2 * torch.randn(d, device=DEV)) if norm else None for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    counted = 0
    if t > 10:
        pos[0, 3] = -1                      # padding
        pos[len(sections) - 1, 5] = -7      # padding by another axis
        pos[len(sections) - 1, 7] = 500     # past the table
        slots[9] = -1                       # not stored
        counted = 1
        if len(sections) > 1:
            pos[0, 8], pos[1, 8] = 777, -1  # past it on one axis, but padding by the other
    cache = torch.full((pages, g.gguf_kv_page_bytes(d, hk, page)), 0xA5, dtype=torch.uint8, device=DEV)
    before = cache.clone()
    q_out, k_out = (torch.full((t, n, d), 7.0, dtype=DTYPES[typ], device=DEV) for n in (h, hk))
    dev_pos = torch.full((len(sections), t + 5), -1, dtype=torch.int32, device=DEV)[:, :t]
    dev_pos.copy_(pos)
    g.gguf_qk_norm_mrope(q, k, v, qw, kw, EPS, dev_pos, table.to(DEV), sections, interleaved, g.ROPE_NEOX if neox else g.ROPE_NORM,
                         cache=cache, slots=slots.to(DEV), page_size=page, q_out=q_out, k_out=k_out, dev_status=status)
    assert int(status.item()) == counted
    done = ((pos >= 0) & (pos < 500)).all(0)
    for got, x, w in ((q_out, q, qw), (k_out, k, kw)):
        want = ref(x, w, table, pos.clamp(max=499), sections, interleaved, neox)
        got = got.double().cpu()
        # as for one axis: the norm's sum of d terms, four roundings, the rotation's three on terms up to |a| + |b|; one
        # rounding to the output type
        size = want.abs() + want.norm(dim=-1, keepdim=True) / d ** 0.5 * 8
        tol = HALF_STEP[typ] * want.abs() + 16 * 2.0 ** -24 * size
        assert bool(((got - want).abs() <= tol)[done].all())
        assert bool((got[~done] == 7).all())
    # the cache holds Q4_0 blocks of the turned keys and of the values: what the one-axis call stores of k_out unturned
    kept = done & (slots >= 0)
    gk, gv = g.gguf_kv_get_rows(cache, slots.to(DEV), hk, d, page)
    other = torch.zeros_like(cache)
    if typ == "f32":
        g.gguf_qk_norm_rope(q[:, :0], k_out, v, None, None, 0.0, torch.zeros(t, dtype=torch.int32, device=DEV), None, cache=other,
                            slots=slots.to(DEV), page_size=page)
        ok, ov = g.gguf_kv_get_rows(other, slots.to(DEV), hk, d, page)
        assert torch.equal(gk[kept], ok[kept]) and torch.equal(gv[kept], ov[kept])
    for got, want in ((gk, ref(k, kw, table, pos.clamp(max=499), sections, interleaved, neox)), (gv, v.double().cpu())):
        # a code is off by half a step of the block's scale, or by one at the far end of the codes (8 / -8 to 7) and on borders
        blocks = want.unflatten(-1, (-1, 32))
        step = (blocks.abs().amax(-1, keepdim=True) / 8).expand(blocks.shape).flatten(-2)
        assert bool(((got.double().cpu() - want).abs() <= step * 1.01 + 1e-6)[kept].all())
    others = torch.tensor(sorted(set(range(pages * page)) - set(slots[kept].tolist())), device=DEV)
    for a, b in zip(g.gguf_kv_get_rows(cache, others, hk, d, page), g.gguf_kv_get_rows(before, others, hk, d, page)):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("d, typ, sections, interleaved, neox", [
    (128, "bf16", (16, 24, 24), False, True), (64, "f16", (12, 10, 10), True, False), (256, "f32", (1, 2, 3, 58), True, True),
    (128, "f32", (64,), False, False)])
def test_equal_positions_are_one_axis(d, typ, sections, interleaved, neox):
    """Text among images: the same bits as the one-axis call, in the outputs and in the cache."""
    t, h, hk, page = 70, 8, 2, 16
    q, k, v, table, pos, slots, pages = setup(t, h, hk, d, typ, sections, page, 5)
    w = 1 + 0.2 * torch.randn(d, device=DEV)
    one = pos[0].contiguous().to(DEV)
    kind = g.ROPE_NEOX if neox else g.ROPE_NORM
    caches = [torch.zeros(pages, g.gguf_kv_page_bytes(d, hk, page), dtype=torch.uint8, device=DEV) for _ in range(2)]
    a = g.gguf_qk_norm_mrope(q, k, v, w, w, EPS, one.expand(len(sections), t).contiguous(), table.to(DEV), sections, interleaved, kind,
                             cache=caches[0], slots=slots.to(DEV), page_size=page)
    b = g.gguf_qk_norm_rope(q, k, v, w, w, EPS, one, table.to(DEV), kind, cache=caches[1], slots=slots.to(DEV), page_size=page)
    assert torch.equal(a, b) and torch.equal(caches[0], caches[1])
    # one row of positions for all axes
    c = g.gguf_qk_norm_mrope(q, k, v, w, w, EPS, one.expand(len(sections), t), table.to(DEV), sections, interleaved, kind,
                             cache=torch.zeros_like(caches[0]), slots=slots.to(DEV), page_size=page)
    assert torch.equal(c, b)
    # queries alone, in place
    got = q.contiguous()
    assert g.gguf_qk_norm_mrope(got, None, None, w, None, EPS, one.expand(len(sections), t).contiguous(), table.to(DEV), sections,
                                interleaved, kind, q_out=got) is got
    assert torch.equal(got, a)


def test_no_rotation():
    q = torch.randn(5, 4, 64, device=DEV)
    pos = torch.tensor([[0, 1, -1, 3, 4], [0, 1, 2, 3, 1 << 30]], dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 7)
    g.gguf_qk_norm_mrope(q, None, None, None, None, EPS, pos, None, (0, 0), q_out=out)
    keep = torch.tensor([0, 1, 3, 4], device=DEV)   # without a table no position is past it
    assert torch.equal(out[keep], q[keep]) and bool((out[2] == 7).all())


def test_binding_refuses_what_does_not_fit():
    q = torch.randn(5, 4, 64, device=DEV)
    pos = torch.zeros(2, 5, dtype=torch.int32, device=DEV)
    table = torch.zeros(9, 64, device=DEV)
    call = lambda p=pos, s=(16, 16), **kw: g.gguf_qk_norm_mrope(q, None, None, None, None, EPS, p, table, s, **kw)  # noqa: E731
    call()
    for bad in (dict(p=pos[0]), dict(p=pos[:, :4]), dict(p=pos.long()), dict(p=pos.T.contiguous().T), dict(s=(32,)), dict(s=(16, 16, 0)),
                dict(s=(-16, 48)), dict(s=(1 << 20, 16)), dict(p=pos.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(g.GgufError, match="qk_norm_mrope"):
        call(s=(16, 17))
    with pytest.raises(g.GgufError, match="axes"):
        call(p=torch.zeros(5, 5, dtype=torch.int32, device=DEV), s=(8, 8, 8, 4, 4))
