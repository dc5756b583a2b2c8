#!/usr/bin/env python3
"""Serves a stack of attention layers: prompts of ragged lengths, then tokens
one at a time, over a paged 8-bit cache.

    python examples/serve_attention.py [--layers 4] [--requests 8] [--tokens 32]

The layers have the TinyLlama shape (hidden 2048, 32 heads x 64, 4 KV heads);
their linears are planned and packed (HyperLinear, random weights) and each
output is added to its input, as a residual.  The page plan is made once per
step for all layers; finished requests give their pages back and new prompts
take their places.  Prints rows per second of both phases."""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_planner_amd import nn as htnn  # noqa: E402
from block_planner_amd import workloads as wl  # noqa: E402


def main() -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=32)
    args = ap.parse_args()
    dev, hidden, heads, kv_heads, dim = torch.device("cuda:0"), 2048, 32, 4, 64
    shape_qkv = wl.LinearShape("qkv", (heads + 2 * kv_heads) * dim, hidden)
    shape_out = wl.LinearShape("o", hidden, heads * dim)

    def linear(layer, shape):
        lin = torch.nn.Linear(shape.k, shape.n, bias=False, device=dev)
        with torch.no_grad():
            lin.weight.copy_(wl.tinyllama_weight_gpu(layer, shape, dev))
        return htnn.HyperLinear.from_linear(lin)

    layers = [htnn.HyperAttention(linear(i, shape_qkv), linear(i, shape_out), heads, kv_heads, dim, qk_norm=True)
              for i in range(args.layers)]
    R = args.requests
    pool = htnn.KVPool(args.layers, n_pages=R * 40, n_kv_heads=kv_heads, head_dim=dim, max_requests=R, max_pages=40,
                       device=dev)
    g = torch.Generator(device=dev)
    g.manual_seed(0)

    def step(q_len):
        plan = pool.plan(q_len)
        x = torch.randn(sum(q_len), hidden, generator=g, device=dev)
        for i, layer in enumerate(layers):
            x = x + layer(x, pool, i, plan)
        return x

    def timed(what, steps):
        torch.cuda.synchronize()
        t, rows = time.perf_counter(), 0
        for q_len in steps:
            x = step(q_len)
            rows += sum(q_len)
        torch.cuda.synchronize()
        t = time.perf_counter() - t
        assert bool(torch.isfinite(x).all())
        print(f"{what}: {rows} rows in {t * 1e3:.2f} ms, {rows / t:.0f} rows/s, {int(pool.n_free)} pages free")

    prompts = [100 + 37 * r for r in range(R)]
    step([1] * R)                                       # first use of every kernel
    pool.release([True] * R)
    timed("prompts", [prompts])
    timed("tokens", [[1] * R] * args.tokens)
    half = [r % 2 == 0 for r in range(R)]
    pool.release(half)
    timed("mixed", [[200 if h else 1 for h in half]] + [[1] * R] * args.tokens)
    return 0


if __name__ == "__main__":
    sys.exit(main())
