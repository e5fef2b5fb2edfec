"""Argument checks of the paged-cache operators, without a GPU: every bad call
is refused with a status before anything is launched."""
import ctypes

import pytest

import gguf_block_quantized_quantize_gb300 as g

INVALID, TYPE, SHAPE, ALIGN, WS = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    return g.load_library()


def test_page_bytes(lib):
    for d in (64, 128, 256):
        for hk in (1, 2, 8):
            for page in (16, 48, 128):
                # 18 bytes per 32 values, keys and values
                assert g.gguf_kv_page_bytes(d, hk, page) == 2 * page * hk * d // 32 * 18
    for bad in ((96, 8, 16), (0, 8, 16), (128, 0, 16), (128, 8, 0), (128, 8, 24), (128, 8, -16), (128, 8, 1 << 21)):
        assert g.gguf_kv_page_bytes(*bad) == -1


def plan(lib, **kw):
    a = dict(ctx=256, new=256, r=4, free=256, nf=8, table=256, ld=4, width=4, page=16, n=8, start=256, kv=256, pos=256,
             slots=256, used=256, status=0, stream=None)
    a.update(kw)
    return lib.gguf_kv_plan(*a.values())


@pytest.mark.parametrize("kw, want", [
    (dict(r=-1), INVALID), (dict(nf=-1), INVALID), (dict(n=-1), INVALID), (dict(width=-1), INVALID),
    (dict(ld=3), INVALID), (dict(r=16385), SHAPE), (dict(n=1 << 31), SHAPE), (dict(page=0), SHAPE),
    (dict(page=24), SHAPE), (dict(page=-16), SHAPE), (dict(ctx=None), INVALID), (dict(new=None), INVALID),
    (dict(free=None), INVALID), (dict(table=None), INVALID), (dict(start=None), INVALID), (dict(kv=None), INVALID),
    (dict(pos=None), INVALID), (dict(slots=None), INVALID), (dict(used=None), INVALID), (dict(slots=260), ALIGN),
    (dict(ctx=257), ALIGN), (dict(status=258), ALIGN)])
def test_plan_refusals(lib, kw, want):
    assert plan(lib, **kw) == want
    assert b"kv_plan" in lib.gguf_last_error()


def rope(lib, **kw):
    a = dict(q=256, k=256, v=256, xt=g.BF16, n_tokens=4, ldq=1024, ldk=256, ldv=256, n_heads=8, n_kv_heads=2,
             head_dim=128, q_norm=256, k_norm=256, eps=1e-6, positions=256, cos_sin=256, n_positions=64, rot=128,
             rope_type=g.ROPE_NEOX, q_out=256, ldqo=1024, k_out=0, ldko=0, cache=256, n_pages=4, page_size=16, slots=256,
             dev_status=0)
    a.update(kw)
    return lib.gguf_qk_norm_rope(ctypes.byref(g.QkRopeArgs(*a.values())), None)


@pytest.mark.parametrize("kw, want", [
    (dict(xt=g.Q8_1), TYPE), (dict(n_tokens=-1), INVALID), (dict(n_heads=-1), INVALID), (dict(head_dim=96), SHAPE),
    (dict(n_kv_heads=0), SHAPE), (dict(page_size=17), SHAPE), (dict(n_pages=-1), INVALID), (dict(rot=8), SHAPE),
    (dict(rot=256), SHAPE), (dict(rot=-16), INVALID), (dict(rope_type=1), INVALID), (dict(ldq=1023), INVALID),
    (dict(ldqo=1023), INVALID), (dict(ldk=255), INVALID), (dict(ldv=255), INVALID), (dict(k_out=256), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q_out=None), INVALID),
    (dict(slots=None), INVALID), (dict(positions=None), INVALID), (dict(cos_sin=None), INVALID), (dict(q=257), ALIGN),
    (dict(q_norm=260), ALIGN), (dict(k_norm=264), ALIGN), (dict(cos_sin=260), ALIGN), (dict(cache=264), ALIGN),
    (dict(slots=260), ALIGN), (dict(positions=258), ALIGN), (dict(n_heads=65536, ldq=1 << 30, ldqo=1 << 30), SHAPE)])
def test_rope_refusals(lib, kw, want):
    assert rope(lib, **kw) == want
    assert b"qk_norm_rope" in lib.gguf_last_error()


def test_rope_nothing_to_do(lib):
    assert rope(lib, n_tokens=0, q=None, positions=None) == 0
    assert lib.gguf_qk_norm_rope(None, None) == INVALID


@pytest.mark.parametrize("kw, want", [
    (dict(ot=g.Q8_1), TYPE), (dict(d=32), SHAPE), (dict(hk=0), SHAPE), (dict(page=8), SHAPE), (dict(pages=-1), INVALID),
    (dict(n=-1), INVALID), (dict(n=1 << 32), SHAPE), (dict(slots=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(cache=None), INVALID), (dict(cache=264), ALIGN), (dict(slots=260), ALIGN),
    (dict(k=257), ALIGN)])
def test_get_rows_refusals(lib, kw, want):
    a = dict(cache=256, pages=4, page=16, hk=2, d=128, slots=256, n=4, k=256, v=256, ot=g.F32, stream=None)
    a.update(kw)
    assert lib.gguf_kv_get_rows(*a.values()) == want


def attn(lib, ws=256, ws_bytes=1 << 40, **kw):
    a = dict(q=256, qt=g.BF16, n_tokens=4, ldq=1024, cache=256, n_pages=4, page_size=16, block_table=256, ld_table=4,
             width=4, q_start=256, kv_len=256, n_requests=4, max_q_len=1, n_heads=8, n_kv_heads=2, head_dim=128,
             scale=0.1, window=0, sinks=0, out=256, ldo=1024, dev_status=0)
    a.update(kw)
    return lib.gguf_paged_attention(ctypes.byref(g.AttnArgs(*a.values())), ws, ws_bytes, None)


@pytest.mark.parametrize("kw, want", [
    (dict(qt=g.Q4_0), TYPE), (dict(n_tokens=-1), INVALID), (dict(n_requests=-1), INVALID), (dict(width=-1), INVALID),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(head_dim=80), SHAPE), (dict(page_size=20), SHAPE),
    (dict(n_kv_heads=3), SHAPE), (dict(n_heads=0), SHAPE), (dict(n_requests=16385), SHAPE), (dict(max_q_len=0), INVALID),
    (dict(ldq=1000), INVALID), (dict(ldo=1000), INVALID), (dict(ld_table=3), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(cache=None), INVALID), (dict(block_table=None), INVALID),
    (dict(q_start=None), INVALID), (dict(kv_len=None), INVALID), (dict(q=257), ALIGN), (dict(out=257), ALIGN),
    (dict(cache=264), ALIGN), (dict(kv_len=257), ALIGN), (dict(q_start=258), ALIGN), (dict(block_table=258), ALIGN),
    (dict(qt=g.F32, n_tokens=200000, max_q_len=200000, width=25000, ld_table=25000), SHAPE)])
def test_attention_refusals(lib, kw, want):
    assert attn(lib, **kw) == want
    assert b"paged_attention" in lib.gguf_last_error()


def test_attention_nothing_to_do(lib):
    assert attn(lib, n_tokens=0, q=None, out=None) == 0
    assert attn(lib, n_requests=0, q=None, out=None) == 0
    assert lib.gguf_paged_attention(None, None, 0, None) == INVALID
    assert lib.gguf_paged_attention_ws_size(None) == 0
