"""The operators of a layer on one long prompt, run together: norm to q8_1 rows, products, rotation on three axes and
store, attention over the shared prompt, output product, norm with the residual sum."""
import importlib.util
import os

import pytest
import torch

import gguf_block_quantized_quantize_gb300 as g
from test_gpu_block_norm import check, ref as norm_ref
from test_gpu_kv import check_attn
from test_gpu_mrope import ref as rope_ref
from test_gpu_prefix import reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
HIDDEN, H, HK, D, PAGE, REQUESTS, PROMPT = 512, 16, 4, 64, 16, 12, 320
SECTIONS = (12, 10, 10)


def q8_0(n, k, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randint(0, 256, (n, g.gguf_row_size(g.Q8_0, k)), dtype=torch.uint8, generator=gen, device=DEV)
    w.view(n, -1, 34)[..., :2] = torch.tensor([0x00, 0x10], dtype=torch.uint8, device=DEV)   # scales of 2^-11
    return w


class Step:
    def __init__(self):
        gen = torch.Generator(device=DEV).manual_seed(1)
        rows = (H + 2 * HK) * D
        self.wqkv, self.wo = q8_0(rows, HIDDEN, 2), q8_0(HIDDEN, H * D, 3)
        self.w = [1 + 0.2 * torch.randn(n, generator=gen, device=DEV) for n in (HIDDEN, D, D, HIDDEN, HIDDEN)]
        ang = torch.rand(600, D // 2, generator=gen, device=DEV, dtype=torch.float64) * 6.28
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
        width = PROMPT // PAGE + 4
        pages = PROMPT // PAGE + REQUESTS * 4
        self.cache = torch.zeros(pages, g.gguf_kv_page_bytes(D, HK, PAGE), dtype=torch.uint8, device=DEV)
        # a table wide enough that the shared tokens are read together
        self.table = torch.full((REQUESTS, width + 5000), -1, dtype=torch.int32, device=DEV)
        order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        self.table[:, :PROMPT // PAGE] = order[:PROMPT // PAGE]
        self.free = order[PROMPT // PAGE:].contiguous()
        self.groups = torch.tensor([0, REQUESTS], dtype=torch.int32, device=DEV)
        self.prefix = torch.tensor([PROMPT], dtype=torch.int32, device=DEV)
        kv = torch.randn(2, PROMPT, HK, D, generator=gen, device=DEV)
        slots = (order[:PROMPT // PAGE].long()[:, None] * PAGE + torch.arange(PAGE, device=DEV)).flatten()
        g.gguf_qk_norm_rope(kv[0][:, :0], kv[0], kv[1], None, None, 0.0, torch.zeros(PROMPT, dtype=torch.int32, device=DEV), None,
                            cache=self.cache, slots=slots, page_size=PAGE)

    def __call__(self, h, ctx, new, t, most):
        s = {}
        s["start"], s["kv_len"], pos, s["slots"], _ = g.gguf_kv_plan(ctx, new, self.free, self.table, PAGE, t)
        s["pos"] = torch.stack([pos, pos // 2, pos // 3]).contiguous()
        s["z"] = torch.empty(t, HIDDEN, device=DEV)
        _, _, s["xq"] = g.gguf_block_norm(None, h, pre_weight=self.w[0], out=s["z"], q8_1=True)
        rows = (H + 2 * HK) * D
        s["qkv"] = g.gguf_mul_mat(self.wqkv, g.Q8_0, rows, HIDDEN, s["xq"], xt=g.Q8_1, m=t,
                                  out=torch.empty(t, rows, dtype=torch.bfloat16, device=DEV))
        q, k, v = (s["qkv"][:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, H), (H, H + HK), (H + HK, H + 2 * HK)))
        s["q"] = g.gguf_qk_norm_mrope(q, k, v, self.w[1], self.w[2], 1e-6, s["pos"], self.cos_sin, SECTIONS, True, cache=self.cache,
                                      slots=s["slots"], page_size=PAGE)
        plan = g.gguf_prefix_plan(s["start"], s["kv_len"], self.groups, self.prefix, PAGE, t)
        s["o"] = g.gguf_prefix_attention(s["q"], self.cache, self.table, plan, 1, HK, PAGE, most, D ** -0.5)
        s["y"] = g.gguf_mul_mat(self.wo, g.Q8_0, HIDDEN, H * D, s["o"].flatten(1))
        s["h"], s["next"], _ = g.gguf_block_norm(s["y"], h, post_kind=g.NORM_RMS, post_weight=self.w[3], pre_kind=g.NORM_LAYER,
                                                 pre_weight=self.w[4], branch_scale=0.5)
        return s


@pytest.fixture
def fixed_order():
    """Products whose sums do not depend on the run (split K adds its parts as they come)."""
    g.gguf_set_option("mmq_split_k", 0)
    yield
    g.gguf_set_option("mmq_split_k", 1)


def test_a_layers_step(fixed_order):
    """Every stage against its formula on what the stage before gave, eager and replayed from a graph, step after step."""
    step = Step()
    gen = torch.Generator(device=DEV).manual_seed(5)
    lens = [1 + r % 3 for r in range(REQUESTS)]
    t = sum(lens)
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)   # noqa: E731
    ctx, new = ints([PROMPT] * REQUESTS), ints(lens)
    h = torch.randn(t, HIDDEN, generator=gen, device=DEV).to(torch.bfloat16)
    step(h, ctx, new, t, 3)   # the load of the kernels before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = step(h, ctx, new, t, 3)
    kept = step.table.clone()
    for i in range(3):
        h.copy_(torch.randn(t, HIDDEN, generator=gen, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        check(s["z"], *norm_ref(None, h, pre_wb=(step.w[0], None))[2:], "first norm")
        assert torch.equal(s["xq"], g.gguf_quantize_q8_1(s["z"]))
        x = s["qkv"][:, :H * D].unflatten(1, (H, D))
        want = rope_ref(x, step.w[1], step.cos_sin, s["pos"].cpu(), SECTIONS, True, True)
        size = want.abs() + want.norm(dim=-1, keepdim=True) / D ** 0.5 * 8
        assert bool(((s["q"].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size).all())
        kv_lens = [PROMPT + n * (i + 1) for n in lens]
        assert s["kv_len"].tolist() == kv_lens
        slots = []
        for r, n in enumerate(kv_lens):
            tok = torch.arange(n, device=DEV)
            slots.append((step.table[r, tok // PAGE].long() * PAGE + tok % PAGE).cpu().numpy())
        b = dict(q=s["q"], cache=step.cache, hk=HK, page=PAGE, slots=slots, q_lens=lens, kv_lens=kv_lens, scale=D ** -0.5)
        check_attn(s["o"], reference(b), "bf16")
        want = norm_ref(s["y"], h, bs=0.5, post="rms", post_wb=(step.w[3], None), pre="layer", pre_wb=(step.w[4], None))
        check(s["h"], *want[:2], "h'")
        check(s["next"], *want[2:], "next")
        # the same from single calls: the graph's bits
        again = {k: v.clone() for k, v in s.items()}
        eager = step(h, ctx, new, t, 3)
        torch.cuda.synchronize()
        for k in ("xq", "qkv", "q", "o", "y", "h", "next"):
            assert torch.equal(eager[k], again[k]), k
        ctx.copy_(again["kv_len"])
        # the pages that the step took leave the list
        step.free.copy_(torch.roll(step.free, -int((step.table != kept).sum())))
        kept = step.table.clone()
    assert g.gguf_device_errors() == 0


def test_example_shared_prompt():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_prompt.py")
    spec = importlib.util.spec_from_file_location("shared_prompt", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    out = mod.main(["--requests", "6", "--prompt", "192", "--steps", "3"])
    # two times a step before the capture and three replays
    assert out["context"] == [192 + 8] * 6 and out["lost"] == 0 and out["finite"]
