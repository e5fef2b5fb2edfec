"""Many questions about one long prompt of text and images, as a serving loop runs a layer of it: the norm before the
layer with the q8_1 rows of its products, q / k / v products, per-head norms and rotation by (time, height, width) with
the store into a paged Q4_0 cache, attention that reads the shared prompt once for all requests, the output product,
and the norm after it with the residual sum.  The prompt is stored once; its pages stand in every request's block table.

    python examples/shared_prompt.py [--requests 32] [--prompt 4096] [--steps 16]

The weights are random Q4_K blocks of N(0, 0.02)-sized values; the point is the calls and their order, and the printed
times per step, with the prompt read once for all requests and with each request reading it for itself.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gguf_block_quantized_quantize_gb300 as g  # noqa: E402
from gguf_block_quantized_quantize_gb300 import synth  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 4096, 32, 8, 128, 64
SECTIONS = (24, 20, 20)   # rotated pairs of time, height and width, in turn


class Layer:
    """Weights, cache pages and block tables of one layer; request 0 stores the prompt for all."""

    def __init__(self, requests: int, prompt: int, steps: int, device, seed: int = 0):
        if prompt % PAGE:
            raise ValueError(f"prompt must be a multiple of {PAGE}: whole pages are shared")
        dev = torch.device(device)
        q, kv = HEADS * DIM, KV_HEADS * DIM
        block = lambda n, k, s: synth.safe_blocks_device(g.Q4_K, n, k, seed=seed + s, device=dev)   # noqa: E731
        self.w = {"q": block(q, HIDDEN, 1), "k": block(kv, HIDDEN, 2), "v": block(kv, HIDDEN, 3), "o": block(HIDDEN, q, 4)}
        self.head_norm, self.norm = torch.ones(DIM, device=dev), torch.ones(HIDDEN, device=dev)
        angle = torch.arange(prompt + steps + 8, device=dev)[:, None] * 10000.0 ** (-torch.arange(0, DIM, 2, device=dev) / DIM)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        own = -(-(steps + 8) // PAGE)
        pages = prompt // PAGE + requests * own
        self.cache = torch.zeros(pages, g.gguf_kv_page_bytes(DIM, KV_HEADS, PAGE), dtype=torch.uint8, device=dev)
        self.table = torch.full((requests, prompt // PAGE + own), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(pages, dtype=torch.int32, device=dev)
        self.ctx = torch.zeros(requests, dtype=torch.int32, device=dev)
        self.groups = torch.tensor([0, requests], dtype=torch.int32, device=dev)
        self.prefix = torch.full((1,), prompt, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def step(self, h, new_len, max_q_len: int, positions=None, share: bool = True):
        """Residual rows h [tokens, HIDDEN], the requests' tokens one after another -> the layer's residual rows.
        positions [3, tokens]; None: the plan's, on all axes, as for text."""
        t = h.shape[0]
        start, kv_len, pos, slots, used = g.gguf_kv_plan(self.ctx, new_len, self.free, self.table, PAGE, t, dev_status=self.status)
        if positions is None:
            positions = pos.expand(3, t)
        _, _, xq = g.gguf_block_norm(None, h, pre_weight=self.norm, q8_1=True)
        qkv = torch.empty(t, (HEADS + 2 * KV_HEADS) * DIM, dtype=h.dtype, device=h.device)
        nq, nk = HEADS * DIM, KV_HEADS * DIM
        q, k, v = qkv[:, :nq], qkv[:, nq:nq + nk], qkv[:, nq + nk:]
        g.gguf_mul_mat_segments(g.Q4_K, HIDDEN, xq, [(self.w["q"], nq, q), (self.w["k"], nk, k), (self.w["v"], nk, v)], xt=g.Q8_1)
        q = g.gguf_qk_norm_mrope(q.unflatten(1, (HEADS, DIM)), k.unflatten(1, (KV_HEADS, DIM)), v.unflatten(1, (KV_HEADS, DIM)),
                                 self.head_norm, self.head_norm, 1e-6, positions, self.cos_sin, SECTIONS, True, cache=self.cache,
                                 slots=slots, page_size=PAGE, dev_status=self.status)
        if share:
            plan = g.gguf_prefix_plan(start, kv_len, self.groups, self.prefix, PAGE, t)   # once for all layers of a step
            o = g.gguf_prefix_attention(q, self.cache, self.table, plan, 1, KV_HEADS, PAGE, max_q_len, DIM ** -0.5,
                                        dev_status=self.status)
        else:
            o = g.gguf_paged_attention(q, self.cache, self.table, start, kv_len, KV_HEADS, PAGE, max_q_len, DIM ** -0.5,
                                       dev_status=self.status)
        y = g.gguf_mul_mat(self.w["o"], g.Q4_K, HIDDEN, nq, o.flatten(1))
        # the next block would take the third result; here the residual stream is what goes on
        h, _, _ = g.gguf_block_norm(y, h, post_kind=g.NORM_RMS, post_weight=self.norm, pre_weight=self.norm, q8_1=True)
        # the pages that were taken leave the free list (the list is rolled, so that its address stays)
        at = (torch.arange(self.free.numel(), device=h.device) + used) % self.free.numel()
        self.free.copy_(self.free[at])
        self.ctx.copy_(kv_len)
        return h


def image_positions(tokens: int, wide: int, device) -> torch.Tensor:
    """Some text, whose three positions are equal, then one image of `wide` patches a row: (time, height, width)."""
    i = torch.arange(tokens, device=device)
    text = tokens // 4
    patch = i - text
    return torch.where(patch < 0, i, text + torch.stack([0 * patch, patch // wide, patch % wide])).to(torch.int32).contiguous()


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=32)
    ap.add_argument("--prompt", type=int, default=4096, help=f"tokens of the shared prompt, a multiple of {PAGE}")
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args(argv)
    dev = torch.device("cuda")
    layer = Layer(a.requests, a.prompt, 3 * a.steps + 3, dev)
    gen = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(a.prompt, HIDDEN, generator=gen, device=dev).to(torch.bfloat16)
    # the prompt, by request 0 alone; then its pages stand in every row
    new = torch.zeros(a.requests, dtype=torch.int32, device=dev)
    new[0] = a.prompt
    y = layer.step(x, new, a.prompt, image_positions(a.prompt, 53, dev))
    layer.table[1:] = layer.table[0].clone()
    layer.ctx.fill_(a.prompt)
    one = torch.ones(a.requests, dtype=torch.int32, device=dev)
    hs = (y[-1] + torch.randn(a.requests, HIDDEN, generator=gen, device=dev)).to(torch.bfloat16)
    times = {}
    for share in (True, False):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):   # one step outside the graph (lazy allocations)
            hs.copy_(layer.step(hs, one, 1, share=share).tanh())
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            hs.copy_(layer.step(hs, one, 1, share=share).tanh())
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(a.steps):
            graph.replay()
        torch.cuda.synchronize()
        times[share] = (time.perf_counter() - t0) * 1e6 / a.steps
    out = {"shared_us": times[True], "alone_us": times[False], "context": layer.ctx.tolist(), "lost": int(layer.status.item()),
           "finite": bool(torch.isfinite(hs).all())}
    print(f"{a.requests} requests on a prompt of {a.prompt} tokens: step {times[True]:.1f} us with the prompt read once, "
          f"{times[False]:.1f} us request by request; {out['lost']} tokens or pages left out")
    return out


if __name__ == "__main__":
    main()
