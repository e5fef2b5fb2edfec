"""gguf_prefix_plan and gguf_prefix_attention against plain evaluations in 64 bits, and against gguf_paged_attention."""
import numpy as np
import pytest
import torch

import gguf_block_quantized_quantize_gb300 as g
from test_gpu_kv import DTYPES, check_attn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def batch(groups, h, hk, d, page, typ, seed=0, peaky=2.0, wide=True):
    """groups: (shared tokens or None for requests outside every group, [(queries, tokens of the whole request), ..]).
    Slots that hold no token are full of NaN scales.  wide: a table of so many columns that the library reads the shared
    tokens together; else one of the requests' own width, with which short requests go one by one."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = np.random.default_rng(seed)
    q_lens, kv_lens, starts, prefix, plans = [], [], [], [], []
    for shared, members in groups:
        if shared is not None:
            starts.append(len(q_lens))
            prefix.append(shared)
        for m, (n, kv) in enumerate(members):
            whole = max(shared or 0, 0) // page if len(members) > 1 else 0
            plans.append((len(starts) - 1 if shared is not None else -1, m, whole))
            q_lens.append(n)
            kv_lens.append(kv)
    starts.append(len(q_lens) if groups[-1][0] is not None else next(i for i in range(len(plans), -1, -1) if i == 0 or plans[i - 1][0] >= 0))
    counts = [max(-(-max(kv, 0) // page), whole) for kv, (_, _, whole) in zip(kv_lens, plans)]
    pages = sum(counts) + 3
    order = rnd.permutation(pages).astype(np.int32)
    table = np.full((len(q_lens), max(counts + [1]) + 1), -1, dtype=np.int32)
    at, leader = 0, 0
    for r, (group, m, whole) in enumerate(plans):
        leader = r if m == 0 else leader
        if m == 0 and group >= 0:
            table[r, :whole] = order[at:at + whole]
            at += whole
        elif group >= 0:
            table[r, :whole] = table[leader, :whole]
        n = max(0, counts[r] - (whole if group >= 0 else 0))
        first = whole if group >= 0 else 0
        table[r, first:first + n] = order[at:at + n]
        at += n
    cache = torch.full((pages, g.gguf_kv_page_bytes(d, hk, page)), 0xFF, dtype=torch.uint8, device=DEV)
    slots, stored = [], set()   # of every request's tokens
    leader = 0
    for r, (group, m, whole) in enumerate(plans):
        leader = r if m == 0 else leader
        row = table[r].astype(np.int64).copy()
        if group >= 0:
            row[:whole] = table[leader, :whole]
        tok = np.arange(max(kv_lens[r], 0))
        slots.append(row[tok // page] * page + tok % page)
        stored.update(slots[-1].tolist())
    stored = torch.tensor(sorted(stored), dtype=torch.int64, device=DEV)
    n = stored.numel()
    if n:
        kv = torch.randn(2, n, hk, d, generator=gen, device=DEV) * torch.rand(2, n, hk, 1, generator=gen, device=DEV).mul_(1.5)
        g.gguf_qk_norm_rope(kv[0][:, :0], kv[0], kv[1], None, None, 0.0, torch.zeros(n, dtype=torch.int32, device=DEV), None,
                            cache=cache, slots=stored, page_size=page)
    q = (torch.randn(sum(q_lens), h, d, generator=gen, device=DEV) * peaky).to(DTYPES[typ])
    ints = lambda a: torch.tensor(np.asarray(a, dtype=np.int32), device=DEV)   # noqa: E731
    if wide:   # 200000 tiles of heads of 64 and 8 rows, as the rule counts them, take more than it gives a call one by one
        table = np.pad(table, ((0, 0), (0, 200000 * 16 // (page * hk * len(q_lens)) + 1)), constant_values=-1)
    return dict(q=q, cache=cache, table=ints(table), start=ints(np.r_[0, np.cumsum(q_lens)]), kv_len=ints(kv_lens), gs=ints(starts),
                prefix=ints(prefix), hk=hk, page=page, slots=slots, q_lens=q_lens, kv_lens=kv_lens, scale=d ** -0.5)


def reference(b, window=0, sinks=0):
    """64-bit outputs and what error bounds are made of (see check_attn), request by request."""
    t, h, d = b["q"].shape
    out, size, total = (torch.zeros(t, h, d, dtype=torch.float64, device=DEV) for _ in range(3))
    reach = torch.zeros(t, h, 1, dtype=torch.float64, device=DEV)
    a = 0
    for n, kv, slots in zip(b["q_lens"], b["kv_lens"], b["slots"]):
        if n and len(slots):
            k, v = (x.double().transpose(0, 1).repeat_interleave(h // b["hk"], 0) for x in g.gguf_kv_get_rows(
                b["cache"], torch.from_numpy(slots).to(DEV), b["hk"], d, b["page"]))
            q = b["q"][a:a + n].double().transpose(0, 1)
            pos = torch.arange(kv - n, kv, device=DEV)[:, None]
            j = torch.arange(len(slots), device=DEV)
            see = j <= pos
            if window:
                see &= (j > pos - window) | (j < sinks)
            some = see.any(1)
            s = torch.where(see, q @ k.transpose(1, 2) * b["scale"], -float("inf"))
            p = torch.where(some[:, None], torch.softmax(s, -1), 0.0)
            out[a:a + n], size[a:a + n] = (p @ v).transpose(0, 1), (p @ v.abs()).transpose(0, 1)
            total[a:a + n] = (see.double() @ v.abs()).transpose(0, 1)
            reach[a:a + n] = (torch.where(see, q.abs() @ k.abs().transpose(1, 2), 0.0).amax(-1) * b["scale"]).T[..., None]
        a += n
    return [x.cpu() for x in (out, size, reach, total)]


def run(b, window=0, sinks=0, max_q=None, **kw):
    plan = g.gguf_prefix_plan(b["start"], b["kv_len"], b["gs"], b["prefix"], b["page"], b["q"].shape[0])
    return g.gguf_prefix_attention(b["q"], b["cache"], b["table"], plan, b["prefix"].numel(), b["hk"], b["page"],
                                   max_q or max(b["q_lens"] + [1]), b["scale"], window=window, sinks=sinks, **kw)


def poisoned(b, max_q, window=0, sinks=0):
    """A workspace of NaN: nothing is read that the call has not written."""
    import ctypes
    q, t = b["q"], b["table"]
    a = g.AttnArgs(q.data_ptr(), g._TYPE_OF[q.dtype], q.shape[0], q.stride(0), b["cache"].data_ptr(), b["cache"].shape[0], b["page"],
                   t.data_ptr(), t.stride(0), t.shape[1], 0, 0, t.shape[0], max_q, q.shape[1], b["hk"], q.shape[2], b["scale"],
                   window, sinks, q.data_ptr(), q.stride(0), 0)
    n = int(g.load_library().gguf_prefix_attention_ws_size(ctypes.byref(a), b["prefix"].numel()))
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)


ONE = lambda *kv: [(1, n) for n in kv]   # noqa: E731
CASES = [
    # groups, h, hk, d, page, type, window, sinks
    ([(40, ONE(50, 61))], 8, 2, 64, 16, "bf16", 0, 0),                                    # few rows: one kernel
    ([(700, ONE(760, 745))], 24, 8, 128, 16, "f32", 0, 0),
    ([(700, ONE(*range(705, 725)))], 24, 8, 128, 16, "bf16", 0, 0),                       # 60 rows: both
    ([(1000, ONE(*range(1001, 1131, 2)))], 32, 8, 128, 64, "bf16", 0, 0),                 # 260 rows: two row blocks
    ([(333, ONE(400, 340, 334, 500, 1000, 350)), (64, ONE(70, 80, 90)), (5, ONE(9, 8))], 16, 2, 256, 32, "bf16", 0, 0),
    ([(333, ONE(*range(340, 373)))], 16, 1, 256, 16, "f16", 0, 0),                        # 528 rows of 256
    ([(2000, [(4, 2100), (3, 2005), (4, 2004), (2, 2300), (1, 2001)])], 8, 2, 64, 48, "f16", 0, 0),
    ([(None, ONE(100, 33)), (160, ONE(200, 161, 177, 190, 300)), (96, ONE(130))], 12, 4, 128, 32, "bf16", 0, 0),   # outside; a group of one
    ([(0, ONE(20, 30)), (-5, ONE(40, 17)), (15, ONE(16, 31)), (16, ONE(17, 40))], 8, 8, 128, 16, "f16", 0, 0),
    ([(320, [(1, 400), (0, 350), (2, 100), (1, 1), (1, 0), (3, 2), (1, 321), (1, 320)])], 16, 2, 64, 16, "bf16", 0, 0),  # shorter than the prefix
    ([(320, [(1, 40), (1, 50), (1, 33)])], 32, 4, 128, 64, "bf16", 0, 0),                 # all of them
    ([(512, ONE(*range(520, 540)))], 8, 2, 128, 16, "bf16", 100, 4),                      # the window begins in the prefix
    ([(512, ONE(*range(520, 900, 20)))], 32, 8, 64, 32, "f16", 200, 20),                  # in it, or after it
    ([(128, ONE(*range(300, 340)))], 8, 1, 128, 16, "bf16", 64, 1000),                    # sinks past the prefix
    ([(640, ONE(700, 2000))], 6, 2, 256, 16, "f32", 77, 33),
    ([(96, ONE(700, 110, 98, 99))], 6, 2, 64, 16, "f32", 0, 0),
    ([(256, [(40, 300), (1, 257), (33, 600), (17, 289)])], 8, 2, 128, 32, "bf16", 0, 0),  # chunks beside single tokens
    ([(256, [(70, 340), (20, 300)])], 4, 4, 256, 16, "f16", 90, 5),
    ([(48, [(100, 60), (3, 50)])], 6, 3, 64, 16, "bf16", 0, 0),                           # a chunk that begins before the prefix ends
    ([(800, ONE(*[820] * 3)), (720, ONE(*[722] * 30)), (16, ONE(*[90] * 7)), (2000, ONE(2001, 2002))], 40, 2, 128, 16, "bf16", 0, 0),
    ([(100, [(5, 120)] * 9)], 7, 1, 128, 16, "f32", 0, 0),
]


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "")[:60] for x in c))
def test_prefix_attention(case, wide):
    groups, h, hk, d, page, typ, window, sinks = case
    b = batch(groups, h, hk, d, page, typ, seed=h + d, wide=wide)
    refs = reference(b, window, sinks)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    most = max(b["q_lens"])
    out = run(b, window, sinks, dev_status=status, ws=poisoned(b, most, window, sinks))
    check_attn(out, refs, typ)
    assert int(status.item()) == 0
    assert torch.equal(out, run(b, window, sinks))           # the same bits again
    check_attn(run(b, window, sinks, max_q=1000), refs, typ)   # max_q_len chooses kernels
    paged = g.gguf_paged_attention(b["q"], b["cache"], b["table"], b["start"], b["kv_len"], hk, page, most, b["scale"],
                                   window=window, sinks=sinks)
    check_attn(paged, refs, typ)
    assert wide or torch.equal(out, paged)   # one by one they are the same kernels


def plan_ref(start, kv, gs, prefix, page, n_tokens):
    """Entries and tokens of a plan, one by one."""
    R, NG = len(kv), len(prefix)
    entries, tokens = [], []
    group = {r: j for j in range(NG) for r in range(max(gs[j], 0), min(gs[j + 1], R))}
    shared = [max(p, 0) // page * page // 16 if min(gs[j + 1], R) - max(gs[j], 0) >= 2 else 0 for j, p in enumerate(prefix)]
    for r in range(R):
        n = max(0, min(start[r + 1], n_tokens) - start[r])
        lo = kv[r] - (start[r + 1] - start[r])
        hi = lo + n - 1
        j = group.get(r, -1)
        t0 = shared[j] if j >= 0 else 0
        entries.append([start[r], n, t0, max(t0, hi // 16 + 1 if n and hi >= 0 else 0), lo, hi, r, R + j if t0 else -1])
    for j in range(NG):
        members = [e for e in entries[max(gs[j], 0):min(gs[j + 1], R)] if e[1]]
        if not shared[j]:
            entries.append([0] * 7 + [-1])
            continue
        s, e = max(gs[j], 0), min(gs[j + 1], R)
        n = max(0, min(start[e], n_tokens) - start[s])
        lo, hi = min([m[4] for m in members], default=2 ** 31 - 1), max([m[5] for m in members], default=-2 ** 31)
        entries.append([start[s], n, 0, min(shared[j], hi // 16 + 1) if n and hi >= 0 else 0, lo, hi, s, -1])
    for t in range(n_tokens):
        r = next((r for r in range(R) if start[r] <= t < start[r + 1]), -1)
        j = group.get(r, -1) if r >= 0 else -1   # request in the low half, group + 1 above it
        tokens.append([kv[r] - (start[r + 1] - t), r | ((j if j >= 0 and shared[j] else -1) + 1) << 16] if r >= 0 else [-1, -1])
    return np.array(entries, dtype=np.int64).reshape(-1, 8), np.array(tokens, dtype=np.int64).reshape(-1, 2)


@pytest.mark.parametrize("r, ng, seed", [(1, 0, 0), (1, 1, 1), (7, 3, 2), (40, 11, 3), (300, 5, 4), (0, 0, 5), (6, 1, 6), (90, 90, 7)])
def test_plan(r, ng, seed):
    rng = np.random.default_rng(seed)
    page = int(rng.choice([16, 32, 48]))
    q = rng.integers(0, 4, r)
    start = np.r_[0, np.cumsum(q)] + (2 if seed % 2 else 0)   # tokens before the first request
    kv = rng.integers(0, 400, r)
    gs = np.sort(rng.integers(0, r + 1, ng + 1))
    if seed == 6:
        gs[:] = [-4, 999]                                     # cut to the requests that there are
    prefix = rng.integers(-3, 300, ng)
    for n_tokens in (int(start[-1]) + 3, max(0, int(start[-1]) - 2)):
        to = lambda a: torch.tensor(np.asarray(a, dtype=np.int32), device=DEV)   # noqa: E731
        out = torch.full((g.gguf_prefix_plan_bytes(r, ng, n_tokens) + 64,), 0x7F, dtype=torch.uint8, device=DEV)
        g.gguf_prefix_plan(to(start), to(kv), to(gs), to(prefix), page, n_tokens, out=out)
        assert bool((out[-64:] == 0x7F).all())
        got = out[:-64].view(torch.int32).cpu().numpy().astype(np.int64)
        entries, tokens = plan_ref(start.tolist(), kv.tolist(), gs.tolist(), prefix.tolist(), page, n_tokens)
        assert got[1:5].tolist() == [r, ng, n_tokens, page]
        mine = got[8:8 + 8 * (r + ng)].reshape(-1, 8)
        for a, b in zip(mine, entries):
            if b[1]:
                assert a.tolist() == b.tolist()
            else:   # no queries: nothing else of it counts but the range of a request's tiles
                assert a[1] == 0 and (a[2] == b[2] and a[7] == b[7])
        at = 8 + 8 * (r + ng) + 2 * n_tokens
        assert np.array_equal(got[8 + 8 * (r + ng):at].reshape(-1, 2), tokens)
        assert np.array_equal(got[at:], np.r_[start, kv])


def test_groups_out_of_range():
    """Bounds of groups past the requests are cut; the answer is that of the requests that there are."""
    b = batch([(200, ONE(220, 230, 250, 240, 260, 233))], 16, 4, 64, 16, "bf16")
    refs = reference(b)
    b["gs"] = torch.tensor([-7, 100], dtype=torch.int32, device=DEV)
    check_attn(run(b), refs, "bf16")
    b["gs"] = torch.tensor([5, 1], dtype=torch.int32, device=DEV)      # decreasing: no group, every row lists all its pages
    check_attn(run(b), refs, "bf16")


def test_rows_outside_and_strides():
    """Queries in a wider array, tokens before the first request and after the last; outputs there stay as they are."""
    b = batch([(300, ONE(310, 333, 320, 350, 400)), (64, [(2, 100), (3, 90)])], 12, 4, 128, 16, "bf16")
    refs = reference(b)
    t, h, d = b["q"].shape
    for odd in (8, 3):
        wide = torch.full((t + 5, h * d + odd), float("nan"), dtype=torch.bfloat16, device=DEV)
        q = wide.as_strided((t + 5, h, d), (h * d + odd, d, 1))
        q[2:t + 2] = b["q"]
        out = torch.full((t + 5, h * d + odd), 7.0, dtype=torch.bfloat16, device=DEV)
        view = out.as_strided((t + 5, h, d), (h * d + odd, d, 1))
        moved = {**b, "q": q, "start": b["start"] + 2}
        run(moved, out=view, max_q=3)
        check_attn(view[2:t + 2], refs, "bf16")
        assert bool((out[:2] == 7).all()) and bool((out[t + 2:] == 7).all()) and bool((out[:, h * d:] == 7).all())


@pytest.mark.parametrize("typ", ["bf16", "f32"])
def test_more_queries_than_rows(typ):
    """A plan whose requests reach past the rows of q: the queries that q holds, at their positions."""
    b = batch([(130, [(2, 150), (2, 140), (3, 200), (2, 133)])], 8, 2, 64, 16, typ)
    refs = reference(b)
    for held in (8, 5, 1):
        got = run({**b, "q": b["q"][:held].contiguous()}, max_q=3)
        check_attn(got, [x[:held] for x in refs], typ)


def test_another_plan():
    """A plan of other sizes: where shared tokens are read together nothing is written, and it is counted."""
    b = batch([(64, ONE(70, 80, 90, 100, 77, 88))], 8, 2, 64, 16, "bf16")
    t = b["q"].shape[0]
    make = lambda page=16, n=t: g.gguf_prefix_plan(b["start"], b["kv_len"], b["gs"], b["prefix"], page, n)   # noqa: E731
    out = torch.full_like(b["q"], 7.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = lambda plan, **kw: g.gguf_prefix_attention(b["q"], b["cache"], b["table"], plan, 1, 2, 16, 1, 0.125, out=out,   # noqa: E731
                                                      dev_status=status, **kw)
    for i, plan in enumerate((make(page=32), make(n=t + 1), torch.zeros_like(make()))):
        call(plan)
        assert bool((out == 7).all()) and int(status.item()) == i + 1
    call(make())
    check_attn(out, reference({**b, "scale": 0.125}), "bf16")
    with pytest.raises(g.GgufError, match="plan of"):
        call(make()[:-8])


@pytest.mark.parametrize("members, h, typ", [(3, 4, "bf16"), (40, 4, "bf16"), (3, 4, "f32"), (6, 16, "f16")])
def test_pages_outside_the_cache_are_counted_once(members, h, typ):
    """A page outside the cache hides its tokens: counted once for a group's shared page, once for a request's own."""
    b = batch([(96, [(1, 150)] * members), (None, ONE(40))], h, 1 if h == 4 else 2, 64, 32, typ)
    table = b["table"]
    table[:members, 1] = 1 << 29                # of the group, read together
    table[1, 3] = -1                            # of request 1's own tokens 96 ..
    table[members, 0] = b["cache"].shape[0]     # of the request outside
    see = [torch.ones(len(s), dtype=torch.bool) for s in b["slots"]]
    for r in range(members):
        see[r][32:64] = False
    see[1][96:128] = False
    see[members][:32] = False
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = run(b, dev_status=status).double().cpu()
    assert int(status.item()) == 3
    hk, d = b["hk"], 64
    for r, slots in enumerate(b["slots"]):
        k, v = (x.double().cpu().transpose(0, 1).repeat_interleave(h // hk, 0)
                for x in g.gguf_kv_get_rows(b["cache"], torch.from_numpy(slots[see[r].numpy()]).to(DEV), hk, d, 32))
        p = torch.softmax((b["q"][r].double().cpu()[:, None] @ k.transpose(1, 2)) * b["scale"], -1)
        want = (p @ v)[:, 0]
        assert float((got[r] - want).norm() / want.norm()) <= {"f32": 4e-6, "f16": 2e-3, "bf16": 4e-3}[typ]


def test_pages_past_the_table():
    b = batch([(96, [(1, 150)] * 9)], 8, 2, 64, 16, "bf16")
    cut = {**b, "table": b["table"][:, :5].contiguous()}    # tokens 80 .. are not in it: one by one, five pages each
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = run(cut, dev_status=status)
    assert int(status.item()) == 9 * 5
    short = {**b, "kv_lens": [80] * 9, "slots": [s[:80] for s in b["slots"]]}
    check_attn(got, reference(short), "bf16")


@pytest.mark.parametrize("members, typ", [(40, "bf16"), (9, "bf16"), (9, "f32")])
def test_lengths_far_past_the_table(members, typ):
    """A length that no table holds sees what the table has; 2^16 tiles past it are counted, and no more walked over."""
    b = batch([(96, [(1, 150)] * members), (None, ONE(40))], 8, 2, 64, 16, typ)
    lens = b["kv_len"].clone()
    lens[members] = 1 << 30      # its 40 tokens lie in 3 pages, whose last 8 slots hold none
    b["table"][members, 2] = -1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = run({**b, "kv_len": lens}, dev_status=status)
    assert int(status.item()) == int((b["table"][members] < 0).sum()) + (1 << 16)
    short = {**b, "kv_lens": b["kv_lens"][:members] + [32], "slots": b["slots"][:members] + [b["slots"][members][:32]]}
    check_attn(got, reference(short), typ)


def test_no_room_for_the_output():
    """Memory that is not there is torch's own error, as where torch makes the output."""
    b = batch([(96, [(1, 150)] * 4)], 8, 2, 64, 16, "bf16")
    plan = g.gguf_prefix_plan(b["start"], b["kv_len"], b["gs"], b["prefix"], 16, 4)
    with pytest.raises(torch.OutOfMemoryError):
        g.gguf_prefix_attention(b["q"][:1].expand(1 << 31, 8, 64), b["cache"], b["table"], plan, 1, 2, 16, 1, 0.1)
    with pytest.raises(ValueError, match="q"):
        g._bound().prefix_attention("q", b["cache"], b["table"], plan, 1, 2, 16, 1, 0.1, 0, 0, None, None, None, 0)
    check_attn(run(b), reference(b), "bf16")


def test_values_of_one_size_and_peaks():
    """A prefix that holds nearly all the weight, or nearly none of it: the join of two very different maxima."""
    for typ, gain in (("bf16", 12.0), ("f16", 12.0), ("f32", 30.0)):
        b = batch([(400, ONE(*range(420, 450)))], 8, 2, 128, 16, typ, seed=3, peaky=gain)
        check_attn(run(b), reference(b), typ)
        b["q"] = (b["q"].float() * 1e-3).to(b["q"].dtype)
        check_attn(run(b), reference(b), typ)


def test_graph_and_streams():
    """Captured with its plan, replayed with other lengths and groups on another stream; two streams at once."""
    b = batch([(512, ONE(*range(600, 632)))], 16, 4, 128, 16, "bf16", seed=1)
    refs = reference(b)
    other = {**b, "kv_lens": [570 + r for r in range(32)], "slots": [s[:570 + r] for r, s in enumerate(b["slots"])]}
    other["kv_len"] = torch.tensor(other["kv_lens"], dtype=torch.int32, device=DEV)
    other_refs = reference(other)
    sizes = {k: b[k].clone() for k in ("kv_len", "gs", "prefix")}
    out = torch.empty_like(b["q"])
    live = {**b, **sizes}
    run(live, out=out)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        run(live, out=out)
        run(live, out=out)
    for kv, prefix, want in ((b["kv_lens"], 512, refs), (other["kv_lens"], 400, other_refs), (b["kv_lens"], 0, refs), (b["kv_lens"], 300, refs)):
        sizes["kv_len"].copy_(torch.tensor(kv, dtype=torch.int32))
        sizes["prefix"].fill_(prefix)
        out.fill_(7)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()
        check_attn(out, want, "bf16")
    eager = run(b)
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        with torch.cuda.stream(side[i % 2]):
            outs.append(run(b if i % 2 else other))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, eager) if i % 2 else True
        check_attn(o, refs if i % 2 else other_refs, "bf16")


def test_long_prefix_of_a_large_batch():
    """Pieces over all CTAs, several row blocks and rounds; offsets of a large cache."""
    b = batch([(6000, ONE(*range(6001, 6131)))], 32, 8, 128, 64, "bf16", seed=2)
    check_attn(run(b), reference(b), "bf16")
    b = batch([(3000 + 500 * i, ONE(*range(3500 + 500 * i, 3512 + 500 * i))) for i in range(6)], 16, 2, 256, 32, "f16", seed=2)
    check_attn(run(b), reference(b), "f16")


def test_no_groups():
    b = batch([(None, ONE(100, 200, 33, 700))], 8, 2, 64, 16, "bf16")
    b["gs"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    check_attn(run(b), reference(b), "bf16")
    empty = {**b, "q": b["q"][:0], "start": torch.zeros_like(b["start"])}
    assert run(empty).shape[0] == 0


def test_no_groups_and_no_arrays():
    """The C call without groups needs no arrays of them."""
    b = batch([(None, ONE(100, 200, 33, 700))], 8, 2, 64, 16, "bf16")
    t = b["q"].shape[0]
    plan = torch.empty(g.gguf_prefix_plan_bytes(4, 0, t), dtype=torch.uint8, device=DEV)
    st = g.load_library().gguf_prefix_plan(b["start"].data_ptr(), b["kv_len"].data_ptr(), 4, None, None, 0, 16, t, plan.data_ptr(),
                                           plan.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    out = g.gguf_prefix_attention(b["q"], b["cache"], b["table"], plan, 0, 2, 16, 1, b["scale"])
    check_attn(out, reference(b), "bf16")


def test_another_device_is_refused(monkeypatch):
    b = batch([(64, ONE(70, 80, 90))], 8, 2, 64, 16, "bf16")
    monkeypatch.setattr(g, "_DEVICE", lambda: 7)
    x = torch.randn(4, 64, device=DEV)
    for call in (lambda: run(b), lambda: g.gguf_block_norm(x, x),
                 lambda: g.gguf_qk_norm_mrope(x.view(4, 1, 64), None, None, None, None, 1e-6, torch.zeros(2, 4, dtype=torch.int32, device=DEV),
                                              None, (0, 0))):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_no_device_errors():
    assert g.gguf_device_errors() == 0
