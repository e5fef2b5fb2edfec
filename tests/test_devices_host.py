"""Tensors of several devices in the native module's calls, without a GPU: tensors that say where they are and hold nothing."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import gguf_block_quantized_quantize_gb300 as g

R, T, H, HK, D, PAGE = 4, 4, 2, 1, 64, 16


def made(away):
    """The tensors of the calls; those whose names are in `away` live on the second device."""
    sizes = dict(q=(T, H, D), k=(T, HK, D), v=(T, HK, D), q_out=(T, H, D), x=(T, 128), h=(T, 128), kf=(T, HK, D), vf=(T, HK, D))
    ints = dict(ctx=R, new=R, free=8, q_start=R + 1, kv_len=R, pos=T, used=1, group=2, prefix=1)
    dev = lambda name: f"cuda:{1 if name in away else 0}"   # noqa: E731
    x = {n: torch.empty(s, device=dev(n)) for n, s in sizes.items()}
    x.update({n: torch.empty(s, dtype=torch.int32, device=dev(n)) for n, s in ints.items()})
    x["table"] = torch.empty(R, 3, dtype=torch.int32, device=dev("table"))
    x["axes"] = torch.empty(3, T, dtype=torch.int32, device=dev("axes"))
    x["slots"] = torch.empty(T, dtype=torch.int64, device=dev("slots"))
    x["cache"] = torch.empty(8, g.gguf_kv_page_bytes(D, HK, PAGE), dtype=torch.uint8, device=dev("cache"))
    x["plan"] = torch.empty(4096, dtype=torch.uint8, device=dev("plan"))
    return x


CALLS = {
    "kv_plan": (lambda b, x: b.kv_plan(x["ctx"], x["new"], x["free"], x["table"], PAGE, T, x["q_start"], x["kv_len"], x["pos"], x["slots"],
                                       x["used"], None, 0), "table"),
    "qk_norm_rope": (lambda b, x: b.qk_norm_rope(x["q"], x["k"], x["v"], None, None, 0.0, x["pos"], None, g.ROPE_NEOX, x["cache"], x["slots"],
                                                 PAGE, x["q_out"], None, None, 0), "q_out"),
    "kv_get_rows": (lambda b, x: b.kv_get_rows(x["cache"], x["slots"], HK, D, PAGE, x["kf"], x["vf"], 0), "slots"),
    "paged_attention": (lambda b, x: b.paged_attention(x["q"], x["cache"], x["table"], x["q_start"], x["kv_len"], HK, PAGE, 1, 1.0, 0, 0,
                                                       x["q_out"], None, None, 0), "q_out"),
    "qk_norm_mrope": (lambda b, x: b.qk_norm_mrope(x["q"], x["k"], x["v"], None, None, 0.0, x["axes"], None, g.ROPE_NEOX, x["cache"], x["slots"],
                                                   PAGE, x["q_out"], None, None, 0, (0, 0, 0), 0), "q_out"),
    "block_norm": (lambda b, x: b.block_norm(x["x"], x["h"], None, 0, 1.0, 1.0, 0, None, None, 0.0, 1, None, None, 0.0, x["h"], None, None, 0),
                   "h"),
    "prefix_plan": (lambda b, x: b.prefix_plan(x["q_start"], x["kv_len"], x["group"], x["prefix"], PAGE, T, x["plan"], 0), "prefix"),
    "prefix_attention": (lambda b, x: b.prefix_attention(x["q"], x["cache"], x["table"], x["plan"], 1, HK, PAGE, 1, 1.0, 0, 0, x["q_out"], None,
                                                         None, 0), "q_out"),
}


@pytest.mark.parametrize("name", ["qk_norm_mrope", "block_norm", "prefix_plan", "prefix_attention"])
def test_one_device(name):
    call, other = CALLS[name]
    with FakeTensorMode(), pytest.raises(ValueError, match="on the device of the call's other tensors"):
        call(g._bound(), made({other}))


@pytest.mark.parametrize("name", ["kv_plan", "qk_norm_rope", "kv_get_rows", "paged_attention"])
def test_any_device(name):
    """The cache's own calls leave it to their caller which tensors the current device can read: past the module's checks the
    library finds that these tensors have no memory."""
    call, other = CALLS[name]
    for away in (set(), {other}):
        with FakeTensorMode():
            assert call(g._bound(), made(away)) == 1
        assert b"null pointer" in g.load_library().gguf_last_error()
