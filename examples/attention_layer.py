"""A GGUF attention layer as a serving loop runs it: quantized q / k / v products,
per-head norms and rotation with the store into a paged Q4_0 cache, attention over
it, and the quantized output product; a prompt first, then single tokens from one
captured CUDA graph.

    python examples/attention_layer.py [--requests 4] [--prompt 200] [--steps 16]

The weights are random Q4_K blocks of N(0, 0.02)-sized values; the point is the
calls and their order, and the printed times per step.
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


class AttentionLayer:
    """Weights, cache pages and block tables of one layer for a fixed set of requests."""

    def __init__(self, requests: int, max_tokens: int, device, seed: int = 0):
        dev = torch.device(device)
        q, kv = HEADS * DIM, KV_HEADS * DIM
        block = lambda n, k, s: synth.safe_blocks_device(g.Q4_K, n, k, seed=seed + s, device=dev)   # noqa: E731
        self.w = {"q": block(q, HIDDEN, 1), "k": block(kv, HIDDEN, 2), "v": block(kv, HIDDEN, 3), "o": block(HIDDEN, q, 4)}
        self.q_norm, self.k_norm = torch.ones(DIM, device=dev), torch.ones(DIM, device=dev)
        angle = torch.arange(max_tokens, device=dev)[:, None] * 10000.0 ** (-torch.arange(0, DIM, 2, device=dev) / DIM)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        width = -(-max_tokens // PAGE)
        self.cache = torch.zeros(requests * width, g.gguf_kv_page_bytes(DIM, KV_HEADS, PAGE), dtype=torch.uint8, device=dev)
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device=dev)
        self.free = torch.randperm(requests * width, device=dev).to(torch.int32)
        self.ctx = torch.zeros(requests, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def step(self, x: torch.Tensor, new_len: torch.Tensor, max_q_len: int) -> torch.Tensor:
        """x [tokens, HIDDEN], the requests' tokens one after another -> the layer's output rows."""
        t = x.shape[0]
        start, kv_len, pos, slots, used = g.gguf_kv_plan(self.ctx, new_len, self.free, self.table, PAGE, t,
                                                         dev_status=self.status)
        qkv = torch.empty(t, (HEADS + 2 * KV_HEADS) * DIM, dtype=x.dtype, device=x.device)
        nq, nk = HEADS * DIM, KV_HEADS * DIM
        q, k, v = qkv[:, :nq], qkv[:, nq:nq + nk], qkv[:, nq + nk:]
        g.gguf_mul_mat_segments(g.Q4_K, HIDDEN, x, [(self.w["q"], nq, q), (self.w["k"], nk, k), (self.w["v"], nk, v)])
        q = g.gguf_qk_norm_rope(q.unflatten(1, (HEADS, DIM)), k.unflatten(1, (KV_HEADS, DIM)), v.unflatten(1, (KV_HEADS, DIM)),
                                self.q_norm, self.k_norm, 1e-6, pos, self.cos_sin, g.ROPE_NEOX, cache=self.cache,
                                slots=slots, page_size=PAGE, dev_status=self.status)
        o = g.gguf_paged_attention(q, self.cache, self.table, start, kv_len, KV_HEADS, PAGE, max_q_len, DIM ** -0.5,
                                   dev_status=self.status)
        # the pages that were taken leave the free list (the list is rolled, so that its address stays)
        at = (torch.arange(self.free.numel(), device=x.device) + used) % self.free.numel()
        self.free.copy_(self.free[at])
        self.ctx.copy_(kv_len)
        return g.gguf_mul_mat(self.w["o"], g.Q4_K, HIDDEN, nq, o.flatten(1))


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=200, help="tokens of the longest prompt; the others are shorter")
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args(argv)
    dev = torch.device("cuda")
    layer = AttentionLayer(a.requests, a.prompt + a.steps + 8, dev)
    lens = [max(1, a.prompt * (i + 1) // a.requests) for i in range(a.requests)]
    gen = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(sum(lens), HIDDEN, generator=gen, device=dev).to(torch.bfloat16)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    y = layer.step(x, torch.tensor(lens, dtype=torch.int32, device=dev), max(lens))
    torch.cuda.synchronize()
    prompt_ms = (time.perf_counter() - t0) * 1e3

    one = torch.ones(a.requests, dtype=torch.int32, device=dev)
    ends = torch.tensor(lens, device=dev).cumsum(0) - 1
    xs = y[ends].clone()   # each request's newest row feeds the next step
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # one step outside the graph (lazy allocations)
        xs.copy_(layer.step(xs, one, 1).tanh())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xs.copy_(layer.step(xs, one, 1).tanh())
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    step_us = (time.perf_counter() - t0) * 1e6 / a.steps
    out = {"tokens": sum(lens), "prompt_ms": prompt_ms, "step_us": step_us, "context": layer.ctx.tolist(),
           "lost": int(layer.status.item()), "finite": bool(torch.isfinite(xs).all())}
    print(f"{a.requests} requests, {sum(lens)} prompt tokens: {prompt_ms:.2f} ms the first time; "
          f"decode step {step_us:.1f} us; contexts {out['context']}; {out['lost']} tokens without a page")
    return out


if __name__ == "__main__":
    main()
