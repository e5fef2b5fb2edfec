"""gguf_prefix_attention in calls whose answer could depend on what the host arguments choose: windows of requests that
share nothing, groups whose first request is short, requests of more than max_q_len queries, plans of other sizes."""
import ctypes

import numpy as np
import pytest
import torch

import gguf_block_quantized_quantize_gb300 as g
from test_gpu_kv import check_attn
from test_gpu_prefix import DEV, ONE, batch, poisoned, reference, run

pytestmark = pytest.mark.gpu


def reads_together(b, max_q, window=0, sinks=0):
    """Whether the call goes through the kernels that read shared tokens together (one by one, the workspace is
    gguf_paged_attention's)."""
    q, t = b["q"], b["table"]
    a = g.AttnArgs(q.data_ptr(), g._TYPE_OF[q.dtype], q.shape[0], q.stride(0), b["cache"].data_ptr(), b["cache"].shape[0], b["page"],
                   t.data_ptr(), t.stride(0), t.shape[1], 0, 0, t.shape[0], max_q, q.shape[1], b["hk"], q.shape[2], b["scale"],
                   window, sinks, q.data_ptr(), q.stride(0), 0)
    lib = g.load_library()
    return lib.gguf_prefix_attention_ws_size(ctypes.byref(a), b["prefix"].numel()) != lib.gguf_paged_attention_ws_size(ctypes.byref(a))


def paged(b, max_q, window=0, sinks=0, **kw):
    return g.gguf_paged_attention(b["q"], b["cache"], b["table"], b["start"], b["kv_len"], b["hk"], b["page"], max_q, b["scale"],
                                  window=window, sinks=sinks, **kw)


# ---------------------------------------------------------------- windows

def seen_pages(b, window, sinks, max_q=1 << 30):
    """Of each request, which pages of its row some query sees: of it, or of its group where they are shared."""
    page, see = b["page"], []
    for n, kv in zip(b["q_lens"], b["kv_lens"]):
        pos, j = np.arange(kv - n, kv)[:max_q, None], np.arange(max(kv, 0))[None]
        some = ((j <= pos) & ((j > pos - window) | (j < sinks) if window else True)).any(0)
        mine = np.zeros(b["table"].shape[1], dtype=bool)
        mine[np.flatnonzero(some) // page] = True
        see.append(mine)
    bounds = b["gs"].tolist()
    for s, e, prefix in zip(bounds, bounds[1:], b["prefix"].tolist()):
        if e - s >= 2:
            whole = max(prefix, 0) // page
            any_of = np.any([m[:whole] for m in see[s:e]], axis=0)
            for m in see[s:e]:
                m[:whole] = any_of
    return np.array(see)


def hide_pages(b, see, how):
    """Pages that no query sees are not there any more (-1), or hold what their next owner left (NaN scales)."""
    gone = torch.from_numpy(~see).to(DEV)
    if how == "stale":
        old = b["table"][gone]
        b["cache"][old[old >= 0].long()] = 0xFF
    else:
        b["table"] = b["table"].masked_fill(gone, -1)
    return int((~see).sum())


WINDOWS = [
    # groups, h, hk, d, page, type, window, sinks: single tokens and chunks outside every group, groups of one, groups whose
    # prefix is shorter than the sinks or than a page
    ([(None, ONE(*range(300, 900, 7)) + [(9, 700), (30, 1000)]), (320, ONE(*range(330, 400, 10))), (200, ONE(500))], 16, 4, 128, 16, "bf16", 100, 20),
    ([(None, ONE(*range(200, 600, 6)) + [(12, 500)]), (100, ONE(*range(500, 520, 4)))], 8, 1, 256, 32, "f16", 64, 40),
    ([(15, ONE(*range(200, 600, 6))), (None, [(20, 400), (3, 500)])], 6, 2, 64, 16, "f32", 77, 33),
    ([(64, ONE(*range(300, 700, 4)) + [(40, 500)])], 8, 1, 128, 16, "bf16", 64, 200),
    ([(400, ONE(*range(700, 900, 4)) + [(18, 800)]), (None, ONE(*range(90, 700, 10)) + [(50, 600)])], 16, 2, 64, 48, "f16", 50, 1),
]


@pytest.mark.parametrize("how", ["freed", "stale"])
@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: "-".join(str(x).replace(" ", "")[:60] for x in c))
def test_windows_of_own_tokens(case, how):
    """Between the sinks and the window of a request nothing is read, counted, or let into the outputs."""
    groups, h, hk, d, page, typ, window, sinks = case
    b = batch(groups, h, hk, d, page, typ, seed=h + d)
    refs = reference(b, window, sinks)
    table = b["table"]
    assert hide_pages(b, seen_pages(b, window, sinks), how) > int((table < 0).sum())
    n = b["q"].shape[0]
    assert reads_together(b, n, window, sinks)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    check_attn(run(b, window, sinks, max_q=n, dev_status=status, ws=poisoned(b, n, window, sinks)), refs, typ)
    assert int(status.item()) == 0
    check_attn(paged(b, n, window, sinks, dev_status=status), refs, typ)
    assert int(status.item()) == 0


# ---------------------------------------------------------------- rows of the table

SHORT = [
    # groups, h, hk, d, page, type: a group's first request ends in the prefix, or has no token at all
    ([(320, [(1, 50), *ONE(*range(330, 360))])], 8, 2, 64, 16, "bf16"),
    ([(320, [(1, 50), (2, 400), (1, 330)])], 8, 2, 128, 16, "f16"),                        # few rows: one kernel
    ([(320, [(0, 0), (1, 10), (3, 200), (1, 500), (1, 500), (2, 320)])], 6, 2, 64, 32, "f32"),
    ([(640, [(2, 33), *ONE(*[700] * 20)]), (160, ONE(170, 100, 180)), (96, [(1, 95), (1, 96), (30, 130)])], 16, 2, 256, 32, "bf16"),
    ([(4000, [(1, 2000), (1, 3999), *ONE(*range(4001, 4150, 2)), (5, 60)])], 32, 8, 128, 64, "bf16"),   # two row blocks
    ([(320, ONE(40, 120, 90))], 16, 2, 64, 16, "f16"),                                     # all of them end in it
]


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("fill", [-1, 0])
@pytest.mark.parametrize("case", SHORT, ids=lambda c: "-".join(str(x).replace(" ", "")[:60] for x in c))
def test_a_short_request_comes_first(case, fill, wide):
    """Every row lists the pages of its own tokens, and no more."""
    groups, h, hk, d, page, typ = case
    b = batch(groups, h, hk, d, page, typ, seed=h + d, wide=wide)
    refs = reference(b)
    kv = torch.tensor(b["kv_lens"], device=DEV)
    past = torch.arange(b["table"].shape[1], device=DEV)[None] * page >= kv[:, None]
    b["table"] = b["table"].masked_fill(past, fill)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    check_attn(run(b, dev_status=status), refs, typ)
    assert int(status.item()) == 0


# ---------------------------------------------------------------- max_q_len

LONG = [
    # groups, h, hk, d, page, type
    ([(320, [(1, 400), (5, 350), (9, 330), (1, 321)]), (None, [(7, 100), (2, 50), (60, 300)])], 8, 2, 64, 16, "bf16"),
    ([(320, [(1, 400), (5, 350), (70, 500), (2, 321)])], 24, 8, 128, 32, "f16"),
    ([(320, [(1, 400), (5, 350), (33, 390), (2, 321)]), (None, [(7, 100), (2, 1)])], 6, 2, 64, 16, "f32"),
    ([(160, [(40, 300)] * 12)], 8, 1, 256, 16, "bf16"),
]


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("most", [1, 3, 6])
@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(str(x).replace(" ", "")[:60] for x in c))
def test_more_queries_than_max_q_len(case, most, wide):
    """Of a request with more queries than max_q_len the first max_q_len are computed, however the call goes, and the
    other rows of out stay as they are."""
    groups, h, hk, d, page, typ = case
    b = batch(groups, h, hk, d, page, typ, seed=h + d, wide=wide)
    refs = reference(b)
    mine = torch.cat([torch.arange(n) < most for n in b["q_lens"]])
    b["table"] = b["table"].masked_fill(torch.from_numpy(~seen_pages(b, 0, 0, most)).to(DEV), -1)   # (for the other queries alone)
    for call in (run, paged):
        out = torch.full_like(b["q"], 7.0)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        call(b, max_q=most, out=out, dev_status=status)
        check_attn(out[mine.to(DEV)], [x[mine] for x in refs], typ)
        assert bool((out[~mine.to(DEV)] == 7).all())
        assert int(status.item()) == 0
    if wide:
        assert reads_together(b, most)


# ---------------------------------------------------------------- plans of other sizes

@pytest.mark.parametrize("groups, h, d, typ", [
    ([(64, ONE(70, 80, 90, 100, 77, 88))], 8, 64, "bf16"),           # few rows, a CTA per unit
    ([(64, ONE(70, 80, 90, 3000, 77, 88))], 8, 64, "f32"),           # units over several CTAs
    ([(64, [(30, 120), (1, 80), (40, 90)])], 8, 128, "f16"),         # both kernels, row blocks in pieces
    ([(64, [(2, 500)] + [(2, 70 + r) for r in range(47)])], 64, 256, "bf16"),   # the prompt kernel alone, in pieces
])
def test_another_plan_one_by_one(groups, h, d, typ):
    """A plan of other sizes, where the requests go one by one: nothing is written, and it is counted once."""
    b = batch(groups, h, 2, d, 16, typ, wide=False)
    refs = reference(b)
    t, most = b["q"].shape[0], max(b["q_lens"])
    assert not reads_together(b, most)
    make = lambda page=16, n=t, ng=1: g.gguf_prefix_plan(b["start"], b["kv_len"], b["gs"][:ng + 1], b["prefix"][:ng], page, n)   # noqa: E731
    out = torch.full_like(b["q"], 7.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = lambda plan: g.gguf_prefix_attention(b["q"], b["cache"], b["table"], plan, 1, 2, 16, most, b["scale"], out=out,   # noqa: E731
                                                dev_status=status)
    fewer = torch.zeros_like(make())
    fewer[:make(ng=0).numel()] = make(ng=0)   # of no group, in room for one
    for i, plan in enumerate((make(page=32), make(n=t + 1), fewer, torch.zeros_like(make()))):
        call(plan)
        assert bool((out == 7).all()) and int(status.item()) == i + 1
    call(make())
    check_attn(out, refs, typ)
    assert int(status.item()) == 4


# ---------------------------------------------------------------- what is not shared

@pytest.mark.parametrize("groups, window, sinks", [
    ([(None, ONE(100, 200, 33, 700))], 0, 0),                 # no group
    ([(320, [(3, 400)])], 0, 0),                              # one request
    ([(3000, ONE(*range(3010, 3050, 10)))], 64, 4),           # a window that hides nearly all of a wide table
])
@pytest.mark.parametrize("typ", ["bf16", "f32"])
def test_calls_with_nothing_to_share(groups, window, sinks, typ):
    """They go one by one, whatever the table's width: gguf_paged_attention's workspace, and its bits."""
    b = batch(groups, 8, 2, 128, 16, typ)
    if groups[0][0] is None:
        b["gs"], b["prefix"] = b["gs"][:1], b["prefix"][:0]
    most = max(b["q_lens"])
    assert not reads_together(b, most, window, sinks)
    out = run(b, window, sinks)
    check_attn(out, reference(b, window, sinks), typ)
    assert torch.equal(out, paged(b, most, window, sinks))


# ---------------------------------------------------------------- fp32 over long prefixes

@pytest.mark.parametrize("members, h, hk, d, prefix", [(40, 24, 8, 64, 30000), (60, 12, 4, 128, 16000), (30, 8, 2, 256, 12000)])
def test_long_prefixes_in_fp32(members, h, hk, d, prefix):
    """What the matrix unit cuts off of a sum, always towards zero, does not add up along the prefix.  A tile's products are
    cut off three times, by 2^-23 of them at most; probabilities and values stand in two parts, each pair right to 2^-23:
    together (5 x 2^-23) below 2^-20 of the outputs, along them."""
    b = batch([(prefix, ONE(*range(prefix + 1, prefix + 1 + members)))], h, hk, d, 16, "f32", seed=d)
    refs = reference(b)
    assert reads_together(b, 1)
    got = run(b)
    check_attn(got, refs, "f32")
    err = got.double().cpu() - refs[0]
    along = float((err * refs[0]).sum() / refs[0].square().sum())
    assert abs(along) < 2.0 ** -20


# ---------------------------------------------------------------- one by one: lengths and counts

@pytest.mark.parametrize("n, d, typ", [(1, 64, "bf16"), (1, 128, "f32"), (40, 64, "f16"), (40, 256, "bf16")])
def test_lengths_far_past_the_table_one_by_one(n, d, typ):
    """As where tokens are read together: 2^16 tiles past the table are counted, and no more walked over."""
    b = batch([(96, ONE(*[150] * 9)), (None, [(n, 40)])], 8, 2, d, 16, typ, wide=False)
    assert not reads_together(b, n)
    lens = b["kv_len"].clone()
    lens[9] = 1 << 30            # its 40 tokens lie in 3 pages, whose last 8 slots hold none
    b["table"][9, 2] = -1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for window, sinks, past in ((0, 0, 1 << 16), (100, 20, 0)):
        status.zero_()
        got = run({**b, "kv_len": lens}, window, sinks, dev_status=status)
        assert int(status.item()) == (int((b["table"][9] < 0).sum()) + past if past else 0)
        seen = 32 if not window else 20   # the window is past the table
        short = {**b, "kv_lens": b["kv_lens"][:9] + [seen + n - 1], "slots": b["slots"][:9] + [b["slots"][9][:seen]]}
        check_attn(got, reference(short) if not window else [torch.cat([x[:9], y[9:]]) for x, y in zip(reference(b, window, sinks), reference(short))], typ)


def test_many_fp32_queries_are_not_counted_one_by_one():
    """One by one a request's units x tiles have to fit in 32 bits; the other way has no such bound."""
    lib = g.load_library()

    def sizes(n, width, qt):
        a = g.AttnArgs(256, qt, n, 4096, 256, 4, 16, 256, width, width, 256, 256, 1, n, 32, 8, 128, 0.1, 0, 0, 256, 4096, 0)
        return lib.gguf_prefix_attention_ws_size(ctypes.byref(a), 0), lib.gguf_paged_attention_ws_size(ctypes.byref(a))

    for n, width, qt, same in ((8, 64, g.F32, True), (8192, 512, g.F32, True), (60000, 512, g.F32, False), (8192, 1 << 18, g.F32, False),
                               (60000, 512, g.BF16, True), (8192, 1 << 18, g.BF16, True)):
        prefix, one = sizes(n, width, qt)
        assert (prefix == one) == same and prefix > 0
