"""Forms of the paged-cache calls beyond the usual ones: one-sided norms, steps that hold more tokens than the
call, arguments without a bound, counts of what was left out, and queries whose values share a sign."""
import numpy as np
import pytest
import torch

import gguf_block_quantized_quantize_gb300 as g
from test_gpu_kv import DEV, DTYPES, HALF_ULP, attn_ref, attn_setup, check_attn, rope_ref

pytestmark = pytest.mark.gpu
I32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)   # noqa: E731


# ------------------------------------------------------------------ a norm of one side alone

@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("side", ["k", "q"])
@pytest.mark.parametrize("t, h, hk, d, neox", [
    (5, 0, 2, 128, True),        # keys alone
    (9, 4, 2, 64, False), (3, 6, 3, 256, True),
    (6000, 7, 3, 128, True),     # several rows per group of lanes, queries and keys among them
    (6000, 0, 9, 128, False)])
def test_norm_of_one_side(orc, typ, side, t, h, hk, d, neox):
    torch.manual_seed(t + h + d)
    dtype, eps, npos, page = DTYPES[typ], 1e-6, 500, 16
    q, k, v = (torch.randn(t, n, d, device=DEV).mul_(2).to(dtype) for n in (h, hk, hk))
    w = 1 + 0.2 * torch.randn(d, device=DEV)
    qw, kw = (w, None) if side == "q" else (None, w)
    ang = torch.rand(npos, d // 2, dtype=torch.float64) * 6.28
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, npos, (t,), dtype=torch.int32)
    pages = -(-t // page) + 1
    slots = torch.randperm(pages * page)[:t].to(DEV)
    cache = torch.zeros(pages, g.gguf_kv_page_bytes(d, hk, page), dtype=torch.uint8, device=DEV)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    g.gguf_qk_norm_rope(q, k, v, qw, kw, eps, pos.to(DEV), table.to(DEV), g.ROPE_NEOX if neox else g.ROPE_NORM,
                        cache=cache, slots=slots, page_size=page, q_out=q_out, k_out=k_out)
    cs = table.double()[pos.long()]
    gk, gv = g.gguf_kv_get_rows(cache, slots, hk, d, page)
    for got, x, xw in ((q_out, q, qw), (k_out, k, kw)):
        ref = rope_ref(x, xw, cs, d, neox, eps)
        # fp32: the norm's sum of d terms, four roundings, the rotation's three on terms up to |a| + |b|;
        # one rounding to the output type
        size = ref.abs() + ref.norm(dim=-1, keepdim=True) / np.sqrt(d) * 8
        assert bool(((got.double().cpu() - ref).abs() <= HALF_ULP[typ] * ref.abs() + 16 * 2.0 ** -24 * size).all())
    if typ == "f32":   # the stored blocks are Q4_0 of exactly the values that k_out shows
        held = orc.dequantize(orc.Q4_0, orc.quantize_weights(orc.Q4_0, k_out.reshape(-1, d).cpu().numpy()), d)
        assert torch.equal(gk.cpu(), torch.from_numpy(held.astype(np.float32)).view(gk.shape))
    else:              # within a code's step of the formula
        ref = rope_ref(k, kw, cs, d, neox, eps)
        step = (ref.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True) / 8).expand(t, hk, d // 32, 32).flatten(-2)
        assert bool(((gk.double().cpu() - ref).abs() <= step * 1.01 + 1e-6).all())


# ------------------------------------------------------------------ more tokens planned than the call holds

@pytest.mark.parametrize("q_lens, kv_lens, held, h, hk, d, typ, window", [
    ([3, 5, 4], [40, 9, 77], 10, 8, 2, 128, "bf16", 0),       # the last request is cut
    ([3, 5, 4], [40, 9, 77], 6, 8, 2, 64, "f16", 20),         # the second is, the third is left out
    ([3, 5, 4], [40, 9, 77], 10, 4, 2, 128, "f32", 0),
    ([70, 130], [100, 400], 150, 4, 2, 64, "bf16", 0),        # on the prompt kernel
    ([70, 130], [100, 400], 73, 8, 1, 128, "f16", 0),         # cut down to few rows
    ([130], [150], 129, 4, 2, 256, "bf16", 50),
    ([40], [3000], 33, 4, 1, 128, "bf16", 0),                 # tokens in pieces
    ([1] * 9, [30] * 9, 4, 4, 2, 128, "bf16", 0)])
def test_step_with_more_tokens_than_the_call(q_lens, kv_lens, held, h, hk, d, typ, window):
    """q_start reaches past the rows of q: the rows that are there are computed as in the whole step."""
    q, cache, table, start, kv_len, k, v = attn_setup(q_lens, kv_lens, h, hk, d, 16, typ)
    wide = torch.full((held + 3, h, d), 9.0, dtype=q.dtype, device=DEV)
    g.gguf_paged_attention(q[:held], cache, table, start, kv_len, hk, 16, max(q_lens), d ** -0.5, window=window, out=wide[:held])
    refs = attn_ref(q, k, v, q_lens, kv_lens, d ** -0.5, window, 0)
    check_attn(wide[:held], [x[:held] for x in refs], typ)
    assert bool((wide[held:] == 9).all())


@pytest.mark.parametrize("q_lens, kv_lens, most, h, typ", [
    ([3, 5, 1], [40, 9, 77], 2, 4, "bf16"), ([3, 5, 1], [40, 9, 77], 2, 4, "f32"), ([70, 130], [100, 400], 60, 8, "bf16"),
    ([70, 130], [100, 2400], 100, 2, "f16")])
def test_requests_longer_than_max_q_len(q_lens, kv_lens, most, h, typ):
    """Of a longer request the first max_q_len queries are computed, the others are not written."""
    hk, d = 2, 64
    q, cache, table, start, kv_len, k, v = attn_setup(q_lens, kv_lens, h, hk, d, 16, typ)
    out = torch.full_like(q, 9.0)
    g.gguf_paged_attention(q, cache, table, start, kv_len, hk, 16, most, d ** -0.5, out=out)
    refs = attn_ref(q, k, v, q_lens, kv_lens, d ** -0.5, 0, 0)
    done = torch.cat([torch.arange(n) < most for n in q_lens])
    check_attn(out[done], [x[done] for x in refs], typ)
    assert bool((out[~done] == 9).all())


def test_attention_after_an_overfull_plan():
    """A plan of more tokens than its arrays hold, the store and the attention over what is there."""
    torch.manual_seed(5)
    h, hk, d, page, lens, held = 4, 2, 64, 16, [30, 45], 50
    cache = torch.full((8, g.gguf_kv_page_bytes(d, hk, page)), 0xFF, dtype=torch.uint8, device=DEV)
    table = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    start, kv_len, pos, slots, _ = g.gguf_kv_plan(I32([0, 0]), I32(lens), I32(list(range(8))), table, page, held, dev_status=status)
    assert status.item() == sum(lens) - held
    q, k, v = (torch.randn(held, n, d, device=DEV).to(torch.bfloat16) for n in (h, hk, hk))
    q = g.gguf_qk_norm_rope(q, k, v, None, None, 0.0, pos, None, cache=cache, slots=slots, page_size=page)
    out = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, page, max(lens), d ** -0.5, out=torch.full_like(q, 9.0))
    kk, vv = g.gguf_kv_get_rows(cache, slots, hk, d, page)
    check_attn(out, attn_ref(q, kk, vv, [30, 20], [30, 20], d ** -0.5, 0, 0), "bf16")


# ------------------------------------------------------------------ arguments without a bound

FAR = 2 ** 63 - 1


@pytest.mark.parametrize("q_lens, kv_lens, h, hk, d, typ", [
    ([1, 1], [700, 33], 8, 2, 128, "bf16"), ([2, 3, 1], [4, 3000, 0], 4, 2, 64, "f32"), ([5], [2], 12, 1, 128, "f16"),
    ([70, 1], [150, 90], 4, 2, 64, "bf16"), ([40], [3000], 4, 1, 128, "f16"), ([90], [40], 2, 1, 256, "bf16")])
@pytest.mark.parametrize("window, sinks, most", [
    (FAR, 0, 0), (FAR, FAR, 0), (2 ** 31, 3, 0), (2 ** 31 - 1, 3, 0), (20, FAR, 0), (20, FAR - 14, FAR), (20, 2 ** 31, 0),
    (0, 0, FAR), (0, 5, 2 ** 31), (20, 4, FAR)])
def test_arguments_without_a_bound(q_lens, kv_lens, h, hk, d, typ, window, sinks, most):
    """A window or first tokens beyond any length hide nothing; max_q_len may be larger than any request."""
    q, cache, table, start, kv_len, k, v = attn_setup(q_lens, kv_lens, h, hk, d, 16, typ, spare_cols=1)
    out = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, 16, most or max(q_lens), d ** -0.5, window=window, sinks=sinks)
    limit = 10 ** 6   # past every length here
    check_attn(out, attn_ref(q, k, v, q_lens, kv_lens, d ** -0.5, min(window, limit), min(sinks, limit)), typ)


# ------------------------------------------------------------------ counts

@pytest.mark.parametrize("q_lens, kv_lens, h, hk, d, page, typ, window, sinks", [
    ([1], [200], 4, 2, 64, 32, "bf16", 0, 0),
    ([1, 1], [200, 333], 24, 2, 128, 48, "f16", 0, 0),              # two groups of rows per KV head
    ([3, 2], [100, 77], 12, 4, 128, 16, "f32", 0, 0),
    ([1, 2], [900, 1500], 8, 2, 64, 64, "bf16", 300, 40),           # a page between the first tokens and the window
    ([1], [9000], 4, 1, 128, 16, "bf16", 0, 0),                     # one unit over many CTAs
    ([80], [200], 4, 2, 64, 32, "bf16", 0, 0),
    ([300, 1, 150], [450, 100, 150], 8, 2, 128, 16, "bf16", 0, 0),  # several row blocks, and a single token beside them
    ([300], [700], 6, 1, 128, 64, "f16", 100, 20),
    ([200], [900], 2, 2, 256, 32, "bf16", 210, 0),
    ([40], [3000], 4, 1, 128, 16, "bf16", 0, 0)])                   # tokens in pieces
def test_pages_outside_the_cache_are_counted_once(q_lens, kv_lens, h, hk, d, page, typ, window, sinks):
    """Each page of a request that is outside the cache and would hold a token that some query of it sees counts one."""
    q, cache, table, start, kv_len, k, v = attn_setup(q_lens, kv_lens, h, hk, d, page, typ, spare_cols=2)
    rng = np.random.default_rng(len(q_lens) + kv_lens[0])
    rows = table.cpu().numpy()
    want = 0
    for r, (n, m) in enumerate(zip(q_lens, kv_lens)):
        for at in range(rows.shape[1]):
            if rng.random() < 0.3 or at * page >= m:
                rows[r, at] = rng.choice((-1, -7, cache.shape[0], 2 ** 31 - 1))
        j = np.arange(m)
        if window:
            j = j[(j > m - n - window) | (j < sinks)]
        want += sum(not 0 <= rows[r, at] < cache.shape[0] for at in np.unique(j // page))
    assert want > 0
    status = torch.full((1,), 5, dtype=torch.int32, device=DEV)
    out = g.gguf_paged_attention(q, cache, torch.from_numpy(rows).to(DEV), start, kv_len, hk, page, max(q_lens), d ** -0.5,
                                 window=window, sinks=sinks, dev_status=status)
    assert status.item() == 5 + want and bool(torch.isfinite(out.float()).all())


@pytest.mark.parametrize("q_len", [1, 80])
def test_pages_past_the_table_are_counted_once(q_len):
    h, hk, d, page = 8, 2, 64, 32
    q, cache, table, start, kv_len, k, v = attn_setup([q_len], [200], h, hk, d, page, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    g.gguf_paged_attention(q, cache, table[:, :4], start, kv_len, hk, page, q_len, 0.125, dev_status=status)
    assert status.item() == -(-200 // page) - 4


# ------------------------------------------------------------------ queries whose values share a sign

@pytest.mark.parametrize("times", [1.0, 8.0])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("typ, h, q_len", [("f16", 32, 1), ("bf16", 32, 1), ("f16", 64, 2), ("f16", 16, 40)])
def test_queries_of_one_sign(typ, h, q_len, d, times):
    """What the code offsets add to the scores of such queries leaves no larger error than others have."""
    hk, n = 4, 700
    q, cache, table, start, kv_len, k, v = attn_setup([q_len], [n], h, hk, d, 16, typ, seed=d)
    q = ((2 + 0.3 * torch.randn(q_len, h, d, device=DEV)) * times).to(DTYPES[typ])
    refs = attn_ref(q, k, v, [q_len], [n], d ** -0.5, 0, 0)
    out = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, 16, q_len, d ** -0.5)
    check_attn(out, refs, typ)
    err = float((out.double().cpu() - refs[0]).norm() / refs[0].norm())
    print(f"{typ} h{h} q{q_len} d{d} x{times}: {err:.2e}")
    # the output's rounding (2.1e-4 of the norm in fp16, 1.7e-3 in bf16) and 2e-4 of operands rounded to fp16
    assert err <= {"f16": 2.1e-4, "bf16": 1.7e-3}[typ] + 2e-4


# ------------------------------------------------------------------ other forms

@pytest.mark.parametrize("q_lens, kv_lens, h, hk, d, window", [
    ([1, 1], [300, 41], 12, 1, 128, 0), ([2], [900], 40, 2, 64, 100), ([1], [2500], 32, 1, 256, 0), ([30], [30], 10, 1, 64, 0)])
def test_fp32_with_many_heads_per_kv_head(q_lens, kv_lens, h, hk, d, window):
    q, cache, table, start, kv_len, k, v = attn_setup(q_lens, kv_lens, h, hk, d, 16, "f32")
    out = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, 16, max(q_lens), d ** -0.5, window=window)
    check_attn(out, attn_ref(q, k, v, q_lens, kv_lens, d ** -0.5, window, 0), "f32")


@pytest.mark.parametrize("q_lens, kv_lens, typ", [([1, 3], [333, 60], "f32"), ([1], [333], "bf16"), ([40, 1], [90, 333], "bf16"),
                                                  ([300], [300], "f16")])
def test_table_wider_than_any_request(q_lens, kv_lens, typ):
    """A table kept for long contexts, which chooses other kernels than a tight one."""
    h, hk, d = 8, 2, 128
    q, cache, table, start, kv_len, k, v = attn_setup(q_lens, kv_lens, h, hk, d, 16, typ, spare_cols=2000)
    out = g.gguf_paged_attention(q, cache, table, start, kv_len, hk, 16, max(q_lens), d ** -0.5)
    check_attn(out, attn_ref(q, k, v, q_lens, kv_lens, d ** -0.5, 0, 0), typ)
