"""gguf_block_norm against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import gguf_block_quantized_quantize_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
KINDS = {"none": g.NORM_NONE, "rms": g.NORM_RMS, "layer": g.NORM_LAYER}
ACTS = {"none": g.GATE_NONE, "sigmoid": g.GATE_SIGMOID, "tanh": g.GATE_TANH, "silu": g.GATE_SILU}


def normed(v, kind, w, b, eps):
    """N(v), and how large the terms are that it is made of: |v| and |mean| over the root, times the weight, and the bias."""
    if kind == "none":
        return v, v.abs()
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    root = ((v - mean).square().mean(-1, keepdim=True) + eps).sqrt()
    w = 1.0 if w is None else w.double()
    b = 0.0 if b is None else b.double()
    size = (v.abs() + v.abs().mean(-1, keepdim=True) * (kind == "layer")) / root * abs(w if isinstance(w, float) else w.abs())
    return (v - mean) / root * w + b, size + (b if isinstance(b, float) else b.abs())


def ref(x, h, gate=None, act="none", bs=1.0, rs=1.0, post="none", post_wb=(None, None), pre="rms", pre_wb=(None, None), eps=1e-6):
    """h' and z in 64 bits, and bounds of what fp32 arithmetic may be off of them."""
    # One step of fp32 is off by u = 2^-24 of its result at most.  N: the sum of a row is a chain of up to 64 values in a
    # thread, 5 steps over a warp and up to 16 over the warps, times 1 / k (two roundings), the root, and two products and
    # a sum: at most (64 + 5 + 16) / 2 + 8 steps on the size of its terms, twice that for LAYER, whose mean is such a sum
    # too (and whose differences take one more).  The gate: e^x to 2 steps, a sum, a quotient, the product; tanh to 2 steps:
    # 8 with the scales.  A following N has the error of its input in all its terms: as much again, and once more in the
    # root.
    u = 2.0 ** -24
    steps = lambda kind: {"none": 0, "rms": 51, "layer": 2 * 51}[kind]   # noqa: E731
    err = 0.0
    out = torch.zeros_like(h, dtype=torch.float64) if x is None else None
    if x is not None:
        y, size = normed(x.double(), post, *post_wb, eps)
        if gate is not None:
            a = gate.double()
            a = {"none": a, "sigmoid": torch.sigmoid(a), "tanh": torch.tanh(a), "silu": a * torch.sigmoid(a)}[act]
            y, size = y * a, size * a.abs()
        out, err = bs * y, (steps(post) + 8) * u * size * abs(bs)
    if h is not None:
        out = out + rs * h.double()
        err = err + 2 * u * (abs(rs) * h.double().abs() + out.abs())
    z, size = normed(out, pre, *pre_wb, eps)
    if pre == "none":
        return out, err, z, err
    mean = out.mean(-1, keepdim=True) if pre == "layer" else 0.0
    root = ((out - mean).square().mean(-1, keepdim=True) + eps).sqrt()
    w = 1.0 if pre_wb[0] is None else pre_wb[0].double().abs()
    err = torch.as_tensor(err, device=out.device).expand(out.shape)
    big = err.square().mean(-1, keepdim=True).sqrt()   # in the root, and in the mean, by Cauchy-Schwarz
    return out, err, z, steps(pre) * u * size + (err + big) * w / root + size * big / root


def check(got, want, err, what):
    bound = err + HALF_STEP[got.dtype] * (want.abs() + err) + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)   # fp16 subnormals
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"{what}: {float((off / bound.clamp(min=1e-300)).max())} times what is allowed"


def check_q8(blocks, z, err):
    """|held - z|: half a step d, d's rounding to fp16 (2^-11 of it, or half an fp16 subnormal step) times the code, and z's error,
    which reaches d too."""
    n, k = z.shape
    raw = blocks.view(n, k // 32, 36)
    d = raw[..., :2].contiguous().view(torch.float16).double()
    s = raw[..., 2:4].contiguous().view(torch.float16).double()
    q = raw[..., 4:].contiguous().view(torch.int8).double()
    zb, eb = z.view(n, -1, 32), err.view(n, -1, 32)
    top = zb.abs().amax(-1, keepdim=True)
    e = eb.amax(-1, keepdim=True)
    step = (top + e) / 127
    half = step * 2.0 ** -11 + 2.0 ** -25
    assert bool(((d - top / 127).abs() <= e / 127 + half + 2.0 ** -23 * step).all())
    assert bool(((q * d - zb).abs() <= 0.5 * step * (1 + 2.0 ** -20) + 127 * half + 2 * e).all())
    assert bool((q.abs() <= 127).all())
    total = q.sum(-1, keepdim=True)
    assert bool(((s - d * total).abs() <= total.abs() * 2 * half + s.abs() * 2.0 ** -11 + 2.0 ** -25).all())


def make(t, k, typ, resid, gate, seed, pad=0, lead=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    def rows(dtype, n=t):   # rows of a wider array that starts `lead` values late
        buf = torch.randn(n * (k + pad) + lead, generator=gen, device=DEV).to(dtype)
        return buf[lead:].view(n, k + pad)[:, :k]
    x, h = rows(DTYPES[typ]), rows(DTYPES[resid])
    x.mul_(0.7).add_(0.1)
    h.mul_(torch.rand(t, 1, generator=gen, device=DEV).mul_(3).add_(0.3).to(h.dtype))
    gt = {"none": None, "rows": rows(DTYPES[typ]), "row": rows(DTYPES[typ], 1)[0], "row32": rows(torch.float32, 1)[0],
          "rows32": rows(torch.float32)}[gate]
    wb = [(1 + 0.2 * torch.randn(k, generator=gen, device=DEV), 0.2 * torch.randn(k, generator=gen, device=DEV)) for _ in range(2)]
    return x, h, gt, wb


CASES = [  # tokens, k, x, residual, post, pre, gate, activation, padding of the rows, first element
    (1, 4096, "bf16", "bf16", "none", "rms", "none", "none", 0, 0), (1, 1, "f32", "f32", "rms", "rms", "none", "none", 0, 0),
    (3, 7, "bf16", "f32", "layer", "layer", "rows", "tanh", 0, 0), (5, 32, "f16", "f16", "rms", "rms", "row", "silu", 0, 0),
    (130, 96, "bf16", "bf16", "rms", "layer", "rows", "sigmoid", 8, 8), (9, 256, "f16", "f32", "layer", "rms", "row32", "none", 0, 0),
    (17, 1000, "bf16", "bf16", "layer", "layer", "rows", "silu", 0, 0), (4, 1111, "f32", "f32", "layer", "rms", "row", "sigmoid", 0, 0),
    (33, 2048, "f16", "f32", "rms", "rms", "rows", "sigmoid", 0, 0), (7, 2080, "bf16", "f32", "rms", "none", "rows32", "tanh", 0, 0),
    (6, 4096, "bf16", "bf16", "rms", "rms", "none", "none", 1, 3), (300, 4128, "f32", "f32", "rms", "layer", "none", "none", 32, 0),
    (2, 8192, "f16", "f16", "layer", "layer", "rows", "sigmoid", 0, 0), (5, 16384, "bf16", "bf16", "rms", "rms", "row", "tanh", 0, 0),
    (3, 20000, "f32", "f32", "layer", "rms", "rows", "sigmoid", 0, 0), (2, 32768, "bf16", "f32", "rms", "layer", "rows", "silu", 0, 0),
    (2, 32768, "f16", "f16", "layer", "layer", "none", "none", 5, 1), (3, 16416, "f32", "f32", "none", "rms", "none", "none", 3, 0)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_block_norm(case):
    t, k, typ, resid, post, pre, gate, act, pad, lead = case
    x, h, gt, (pw, nw) = make(t, k, typ, resid, gate, k + t, pad, lead)
    kw = dict(gate=gt, gate_act=ACTS[act], branch_scale=0.75, residual_scale=1.25, post_kind=KINDS[post], post_weight=pw[0],
              post_bias=pw[1] if post == "layer" else None, pre_kind=KINDS[pre], pre_weight=nw[0],
              pre_bias=nw[1] if pre == "layer" else None)
    want = ref(x, h, gt, act, 0.75, 1.25, post, (pw[0], kw["post_bias"]), pre, (nw[0], kw["pre_bias"]))
    out = torch.empty(t, k + pad, dtype=x.dtype, device=DEV).fill_(7)[:, :k]
    h2, z, q8 = g.gguf_block_norm(x, h, out=out, q8_1=k % 32 == 0, **kw)
    assert z is out and h2.dtype == h.dtype
    check(h2, *want[:2], "h'")
    check(z, *want[2:], "z")
    if k % 32 == 0:
        check_q8(q8, *want[2:])
        # the blocks are those of the fp32 values of z
        z32 = torch.empty(t, k, dtype=torch.float32, device=DEV)
        g.gguf_block_norm(x, h, out=z32, **kw)
        assert torch.equal(g.gguf_quantize_q8_1(z32), q8)
        alone = g.gguf_block_norm(x, h, q8_1=True, **kw)   # without z as floats
        assert alone[1] is None and torch.equal(alone[2], q8) and torch.equal(alone[0], h2)
    again = g.gguf_block_norm(x, h, **kw)   # the same bits, from other tensors
    assert torch.equal(again[0], h2) and torch.equal(again[1], z) and again[2] is None
    if pad:
        assert bool((out._base.view(t, k + pad)[:, k:] == 7).all())


def test_parts_left_out():
    x, h, gt, (pw, nw) = make(5, 512, "bf16", "bf16", "rows", 1)
    # the norm before the first block: nothing but z
    h2, z, _ = g.gguf_block_norm(None, h, pre_weight=nw[0])
    assert h2 is None
    check(z, *ref(None, h, pre_wb=(nw[0], None))[2:], "z")
    # no residual
    h2, z, _ = g.gguf_block_norm(x, None, gate=gt, gate_act=g.GATE_TANH, pre_weight=nw[0])
    want = ref(x, None, gt, "tanh", pre_wb=(nw[0], None))
    check(h2, *want[:2], "h'")
    check(z, *want[2:], "z")
    # no norm at all: the sum alone, which is z too, rounded
    h2, z, _ = g.gguf_block_norm(x, h, pre_kind=g.NORM_NONE, out=torch.empty(5, 512, device=DEV))
    assert torch.equal(z, x.float() + h.float()) and torch.equal(h2, z.bfloat16())
    # no weights
    _, z, _ = g.gguf_block_norm(x, h, post_kind=g.NORM_LAYER, pre_kind=g.NORM_LAYER)
    check(z, *ref(x, h, post="layer", pre="layer")[2:], "z")
    # no tokens
    assert g.gguf_block_norm(x[:0], h[:0])[1].shape == (0, 512)


@pytest.mark.parametrize("typ, k", [("bf16", 2048), ("f32", 777)])
def test_in_place(typ, k):
    x, h, _, (pw, nw) = make(40, k, typ, typ, "none", 2)
    kw = dict(post_kind=g.NORM_RMS, post_weight=pw[0], pre_weight=nw[0])
    h2, z, _ = g.gguf_block_norm(x, h, **kw)
    a, b, _ = g.gguf_block_norm(x, h, residual_out=h, out=x, **kw)
    assert a is h and b is x and torch.equal(h, h2) and torch.equal(x, z)


@pytest.mark.parametrize("k", [64, 96, 1024, 1030])
def test_rows_stay_apart(k):
    """NaN, infinities and zeros of a row stay in it; a row of zeros gives zeros."""
    x, h, _, (pw, nw) = make(12, k, "bf16", "bf16", "none", 3)
    kw = dict(post_kind=g.NORM_LAYER, post_weight=pw[0], pre_kind=g.NORM_RMS, pre_weight=nw[0], q8_1=k % 32 == 0,
              out=torch.empty_like(x))
    clean = g.gguf_block_norm(x, h, **{**kw, "out": torch.empty_like(x)})
    x[2, 5], x[4, 0], h[7, k - 1] = float("nan"), float("inf"), -float("inf")
    x[9], h[9] = 0, 0
    got = g.gguf_block_norm(x, h, **kw)
    keep = torch.tensor([i for i in range(12) if i not in (2, 4, 7, 9)], device=DEV)
    for a, b in zip(got, clean):
        assert a is None or torch.equal(a[keep], b[keep])
    assert bool(torch.isnan(got[1][2]).all()) and bool((got[1][9] == 0).all()) and bool((got[0][9] == 0).all())
    if k % 32 == 0:
        assert bool((got[2][9] == 0).all())


def test_ranges():
    """Large, small and far-off-centre rows: nothing overflows on the way, and the centred norm keeps its digits."""
    k = 1024
    gen = torch.Generator(device=DEV).manual_seed(4)
    base = torch.randn(6, k, generator=gen, device=DEV)
    h = base * torch.tensor([1e15, 1e-12, 1.0, 1e-30, 3.0, 1.0], device=DEV)[:, None]
    h[2] += 1000.0
    for pre in ("rms", "layer"):
        _, z, q8 = g.gguf_block_norm(None, h, pre_kind=KINDS[pre], eps=1e-20, out=torch.empty_like(h), q8_1=True)
        want = ref(None, h, pre=pre, eps=1e-20)
        check(z, *want[2:], pre)
        check_q8(q8, *want[2:])


def test_offsets_past_32_bits():
    k, step = 256, (1 << 30) + 8   # rows 2 GiB apart
    big = torch.empty(4 * step, dtype=torch.bfloat16, device=DEV)
    rows = torch.as_strided(big, (4, k), (step, 1))
    x, h, _, (_, nw) = make(4, k, "bf16", "bf16", "none", 5)
    rows.copy_(h)
    want = g.gguf_block_norm(x, h, pre_weight=nw[0])
    got = g.gguf_block_norm(x, rows, pre_weight=nw[0], residual_out=rows)
    assert torch.equal(rows, want[0]) and torch.equal(got[1], want[1])


def test_streams_graph_and_products():
    """Norm, product and norm, as a block runs, captured and replayed on another stream with other values."""
    k, n = 1024, 512
    x, h, _, (pw, nw) = make(4, k, "bf16", "bf16", "none", 6)
    torch.manual_seed(7)
    w = torch.randint(0, 256, (n, g.gguf_row_size(g.Q8_0, k)), dtype=torch.uint8, device=DEV)
    w.view(n, -1, 34)[..., :2] = torch.tensor([0x00, 0x2c], dtype=torch.uint8, device=DEV)   # scales of 2^-4
    y = torch.empty(4, n, dtype=torch.bfloat16, device=DEV)

    def step(a, b):
        h2, _, q8 = g.gguf_block_norm(a, b, post_kind=g.NORM_RMS, post_weight=pw[0], pre_weight=nw[0], q8_1=True)
        g.gguf_mul_mat(w, g.Q8_0, n, k, q8, xt=g.Q8_1, m=4, out=y)
        return h2, g.gguf_block_norm(y, h2[:, :n].contiguous(), pre_weight=nw[0][:n])[1]

    stream = torch.cuda.Stream()
    sx, sh = x.clone(), h.clone()
    torch.cuda.synchronize()   # the load of the kernels, and the buffers, before the capture
    step(sx, sh)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step(sx, sh)
    for seed in (8, 9):
        a, b, _, _ = make(4, k, "bf16", "bf16", "none", seed)
        sx.copy_(a)
        sh.copy_(b)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()
        want = step(a, b)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # q8_1 rows from the norm give the product that the norm's fp32 rows give
        z32 = torch.empty(4, k, device=DEV)
        g.gguf_block_norm(a, b, post_kind=g.NORM_RMS, post_weight=pw[0], pre_weight=nw[0], out=z32)
        want = step(a, b)
        assert torch.equal(y, g.gguf_mul_mat(w, g.Q8_0, n, k, z32, out_dtype=torch.bfloat16))


def test_binding_refuses_what_does_not_fit():
    x, h, _, (pw, _) = make(4, 64, "bf16", "bf16", "none", 10)
    f = g.gguf_block_norm
    for bad in (dict(residual=h[:3]), dict(residual=h.T), dict(x=x.cpu()), dict(x=x[0]), dict(pre_weight=pw[0][:63]),
                dict(pre_weight=pw[0].bfloat16()), dict(gate=x[:2]), dict(gate=x[0, :63]), dict(out=x[:, :63]),
                dict(residual_out=torch.empty(4, 64, device=DEV)), dict(out_q8_1=torch.empty(4, 71, dtype=torch.uint8, device=DEV)),
                dict(x=x.long()), dict(gate=h[:, ::2])):
        args = {"x": x, "residual": h, **bad}
        with pytest.raises(ValueError):
            f(args.pop("x"), args.pop("residual"), **args)
    with pytest.raises(ValueError):
        f(None, None)
    with pytest.raises(g.GgufError, match="block_norm"):
        f(x, h.half())
    with pytest.raises(g.GgufError, match="block_norm"):
        f(x, h, pre_kind=9)
    assert np.isfinite(f(x, h)[1].float().cpu().numpy()).all()


@pytest.mark.parametrize("t, k, typ, resid, post, pre, gate, pad, lead", [
    (1300, 288, "bf16", "bf16", "rms", "rms", "none", 0, 0), (1501, 512, "f16", "f32", "layer", "rms", "rows", 8, 0),
    (1219, 2048, "bf16", "f32", "rms", "layer", "row", 0, 0), (2500, 1000, "f32", "f32", "rms", "rms", "rows32", 24, 4),
    (1300, 4096, "f16", "f16", "layer", "layer", "rows", 0, 0), (1250, 8224, "bf16", "bf16", "none", "rms", "rows", 0, 0),
    (1220, 16384, "bf16", "f32", "rms", "rms", "none", 0, 0), (1220, 4100, "f32", "f32", "none", "layer", "none", 0, 0),
    (1300, 17000, "bf16", "bf16", "rms", "rms", "none", 0, 0), (1300, 700, "bf16", "bf16", "rms", "rms", "none", 1, 1)])
def test_many_rows(t, k, typ, resid, post, pre, gate, pad, lead):
    """More rows than the GPU holds at once: copies of rows ahead, strides, in place."""
    x, h, gt, (pw, nw) = make(t, k, typ, resid, gate, 21, pad, lead)
    kw = dict(gate=gt, gate_act=g.GATE_SIGMOID, branch_scale=0.75, post_kind=KINDS[post], post_weight=pw[0],
              post_bias=pw[1] if post == "layer" else None, pre_kind=KINDS[pre], pre_weight=nw[0],
              pre_bias=nw[1] if pre == "layer" else None)
    want = ref(x, h, gt, "sigmoid", 0.75, 1.0, post, (pw[0], kw["post_bias"]), pre, (nw[0], kw["pre_bias"]))
    out = torch.empty_like(x)
    h2, z, q8 = g.gguf_block_norm(x, h, out=out, q8_1=k % 32 == 0, **kw)
    check(h2, *want[:2], "h'")
    check(z, *want[2:], "z")
    if k % 32 == 0:
        check_q8(q8, *want[2:])
    for _ in range(3):   # the same bits, whatever the order of the rows
        again = g.gguf_block_norm(x, h, **kw)
        assert torch.equal(again[0], h2) and torch.equal(again[1], z)
    a, b, _ = g.gguf_block_norm(x, h, residual_out=h, out=x, **kw)
    assert torch.equal(a, h2) and torch.equal(b, z)
    alone = g.gguf_block_norm(None, h, pre_weight=nw[0])[1]
    check(alone, *ref(None, h, pre_wb=(nw[0], None))[2:], "z alone")
    assert g.gguf_device_errors() == 0
