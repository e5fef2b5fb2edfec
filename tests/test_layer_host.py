"""Argument checks of the operators around the products of a layer (block norms, positions on several axes), without
a GPU: every bad call is refused with a status before anything is launched."""
import ctypes

import pytest

import gguf_block_quantized_quantize_gb300 as g

INVALID, TYPE, SHAPE, ALIGN, WS = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    return g.load_library()


def norm(lib, **kw):
    a = dict(x=256, xt=g.BF16, ldx=128, h=256, ht=g.BF16, ldh=128, gate=256, gt=g.BF16, ldg=128, gate_act=g.GATE_SILU,
             n_tokens=4, k=128, post_kind=g.NORM_RMS, post_w=256, post_b=0, post_eps=1e-6, pre_kind=g.NORM_LAYER, pre_w=256,
             pre_b=256, pre_eps=1e-6, branch_scale=1.0, residual_scale=1.0, h_out=256, ldho=128, z=256, zt=g.BF16, ldz=128,
             z_q8_1=256)
    a.update(kw)
    return lib.gguf_block_norm(ctypes.byref(g.BlockNormArgs(*a.values())), None)


@pytest.mark.parametrize("kw, want", [
    (dict(xt=g.Q8_1), TYPE), (dict(ht=g.F16), TYPE), (dict(ht=g.Q4_0), TYPE), (dict(xt=g.F32), TYPE), (dict(zt=g.Q8_1), TYPE),
    (dict(gt=g.F16), TYPE), (dict(n_tokens=-1), INVALID), (dict(k=-1), INVALID), (dict(k=0), SHAPE),
    (dict(k=32769, ldx=1 << 16, ldh=1 << 16, ldg=1 << 16, ldho=1 << 16, ldz=1 << 16), SHAPE), (dict(n_tokens=1 << 31), SHAPE),
    (dict(k=100), SHAPE), (dict(post_kind=3), INVALID), (dict(pre_kind=-1), INVALID), (dict(gate_act=4), INVALID),
    (dict(gate_act=-1), INVALID), (dict(x=None), INVALID), (dict(x=None, gate=None), INVALID),
    (dict(post_eps=-1.0), INVALID), (dict(pre_eps=float("nan")), INVALID), (dict(ldx=127), INVALID), (dict(ldh=127), INVALID),
    (dict(ldg=127), INVALID), (dict(ldg=-128), INVALID), (dict(ldho=127), INVALID), (dict(ldz=127), INVALID),
    (dict(h_out=None, z=None, z_q8_1=None), INVALID),
    (dict(x=None, h=None, gate=None, post_kind=g.NORM_NONE), INVALID), (dict(x=257), ALIGN), (dict(h=257), ALIGN),
    (dict(gate=257), ALIGN), (dict(h_out=257), ALIGN), (dict(z=257), ALIGN), (dict(z_q8_1=258), ALIGN), (dict(post_w=258), ALIGN),
    (dict(pre_b=258), ALIGN)])
def test_block_norm_refusals(lib, kw, want):
    assert norm(lib, **kw) == want
    assert b"block_norm" in lib.gguf_last_error()


def test_block_norm_nothing_to_do(lib):
    assert norm(lib, n_tokens=0, x=None, gate=None, post_kind=g.NORM_NONE, h=None) == 0
    assert lib.gguf_block_norm(None, None) == INVALID


def mrope(lib, sections=(16, 24, 24), n_axes=3, ld=4, interleaved=0, axes=True, **kw):
    a = dict(q=256, k=256, v=256, xt=g.BF16, n_tokens=4, ldq=1024, ldk=256, ldv=256, n_heads=8, n_kv_heads=2,
             head_dim=128, q_norm=256, k_norm=256, eps=1e-6, positions=256, cos_sin=256, n_positions=64, rot=128,
             rope_type=g.ROPE_NEOX, q_out=256, ldqo=1024, k_out=0, ldko=0, cache=256, n_pages=4, page_size=16, slots=256,
             dev_status=0)
    a.update(kw)
    x = g.RopeAxes(n_axes, ld, (ctypes.c_int32 * 4)(*sections), interleaved)
    return lib.gguf_qk_norm_mrope(ctypes.byref(g.QkRopeArgs(*a.values())), ctypes.byref(x) if axes else None, None)


@pytest.mark.parametrize("kw, want", [
    (dict(axes=False), INVALID), (dict(n_axes=0), SHAPE), (dict(n_axes=5), SHAPE), (dict(n_axes=-1), SHAPE), (dict(n_axes=2), SHAPE),
    (dict(sections=(16, 24, 25)), SHAPE), (dict(sections=(-16, 40, 40)), INVALID), (dict(rot=64), SHAPE), (dict(ld=3), INVALID), (dict(ld=-4), INVALID),
    (dict(sections=(0, 0, 0), rot=0, ld=-1), INVALID), (dict(xt=g.Q8_1), TYPE), (dict(head_dim=96), SHAPE), (dict(rot=24), SHAPE),
    (dict(positions=None), INVALID), (dict(cos_sin=None), INVALID), (dict(positions=258), ALIGN), (dict(cos_sin=260), ALIGN),
    (dict(rope_type=1), INVALID), (dict(ldq=1023), INVALID)])
def test_mrope_refusals(lib, kw, want):
    assert mrope(lib, **kw) == want
    assert b"qk_norm_mrope" in lib.gguf_last_error()


def test_mrope_nothing_to_do(lib):
    assert mrope(lib, n_tokens=0, q=None, positions=None) == 0
    assert lib.gguf_qk_norm_mrope(None, ctypes.byref(g.RopeAxes()), None) == INVALID


def test_prefix_plan_bytes(lib):
    # a header, an entry per request and group, two words per token, the lengths
    assert g.gguf_prefix_plan_bytes(0, 0, 0) == 32 + 4
    assert g.gguf_prefix_plan_bytes(5, 2, 11) == 32 + 7 * 32 + 11 * 8 + 11 * 4
    for bad in ((-1, 0, 0), (0, -1, 0), (0, 0, -1), (16385, 0, 0), (0, 16385, 0), (0, 0, 1 << 31)):
        assert g.gguf_prefix_plan_bytes(*bad) == -1


def plan(lib, **kw):
    a = dict(start=256, kv=256, r=4, group=256, prefix=256, ng=2, page=16, n=8, plan=256, bytes=1 << 20, stream=None)
    a.update(kw)
    return lib.gguf_prefix_plan(*a.values())


@pytest.mark.parametrize("kw, want", [
    (dict(r=-1), INVALID), (dict(ng=-1), INVALID), (dict(n=-1), INVALID), (dict(r=16385), SHAPE), (dict(ng=16385), SHAPE),
    (dict(n=1 << 31), SHAPE), (dict(page=0), SHAPE), (dict(page=24), SHAPE), (dict(page=1 << 21), SHAPE), (dict(start=None), INVALID),
    (dict(kv=None), INVALID), (dict(group=None), INVALID), (dict(prefix=None), INVALID), (dict(plan=None), INVALID),
    (dict(start=258), ALIGN), (dict(kv=257), ALIGN), (dict(group=258), ALIGN), (dict(prefix=258), ALIGN), (dict(plan=264), ALIGN),
    (dict(bytes=32 + 6 * 32 + 8 * 8 + 9 * 4 - 1), WS)])
def test_prefix_plan_refusals(lib, kw, want):
    assert plan(lib, **kw) == want
    assert b"prefix_plan" in lib.gguf_last_error()


def prefix(lib, plan=256, plan_bytes=1 << 20, ng=2, ws=256, ws_bytes=1 << 40, **kw):
    a = dict(q=256, qt=g.BF16, n_tokens=4, ldq=1024, cache=256, n_pages=4, page_size=16, block_table=256, ld_table=4,
             width=4, q_start=0, kv_len=0, n_requests=4, max_q_len=1, n_heads=8, n_kv_heads=2, head_dim=128,
             scale=0.1, window=0, sinks=0, out=256, ldo=1024, dev_status=0)
    a.update(kw)
    return lib.gguf_prefix_attention(ctypes.byref(g.AttnArgs(*a.values())), plan, plan_bytes, ng, ws, ws_bytes, None)


@pytest.mark.parametrize("kw, want", [
    (dict(qt=g.Q4_0), TYPE), (dict(n_tokens=-1), INVALID), (dict(n_requests=-1), INVALID), (dict(ng=-1), INVALID),
    (dict(ng=16385), SHAPE), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(head_dim=80), SHAPE),
    (dict(page_size=20), SHAPE), (dict(n_kv_heads=3), SHAPE), (dict(n_requests=16385), SHAPE), (dict(max_q_len=0), INVALID),
    (dict(n_tokens=(1 << 27) + 1), SHAPE), (dict(n_tokens=1 << 20, width=1 << 26, ld_table=1 << 26), SHAPE), (dict(ldq=1000), INVALID), (dict(ldo=1000), INVALID), (dict(ld_table=3), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(plan=None), INVALID), (dict(plan_bytes=32 + 6 * 32 + 4 * 8 + 9 * 4 - 1), WS), (dict(cache=None), INVALID), (dict(block_table=None), INVALID), (dict(plan=264), ALIGN),
    (dict(q=257), ALIGN), (dict(out=257), ALIGN), (dict(cache=264), ALIGN), (dict(block_table=258), ALIGN), (dict(dev_status=258), ALIGN)])
def test_prefix_attention_refusals(lib, kw, want):
    assert prefix(lib, **kw) == want
    assert b"prefix_attention" in lib.gguf_last_error()


def test_prefix_attention_nothing_to_do(lib):
    assert prefix(lib, n_tokens=0, q=None, out=None, plan=None) == 0
    assert prefix(lib, n_requests=0, q=None, out=None, plan=None) == 0
    assert lib.gguf_prefix_attention(None, 256, 1 << 20, 2, None, 0, None) == INVALID
    assert lib.gguf_prefix_attention_ws_size(None, 2) == 0
