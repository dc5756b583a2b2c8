#!/usr/bin/env python3
"""Heals a quantised output layer from its full-precision teacher.

    python examples/distill_head.py [--steps 20] [--rows 1024] [--top 32]

Hidden states run through AddRMSNorm and a trainable HyperLinear (the student's
output layer, TinyLlama's width of 2048 and 32000 tokens, its weight planned
and packed again every few steps); a plain linear over the same norm is the
teacher.  Once per batch the teacher's top log probabilities are kept
(api.token_logprobs); the student learns from them (nn.distill_loss), its
gradient runs back through the packed weight and the norm.  Prints the loss,
both models' agreement on the likeliest token and rows per second."""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_planner_amd import api  # noqa: E402
from block_planner_amd import nn as htnn  # noqa: E402


def main() -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rows", type=int, default=1024)
    ap.add_argument("--top", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=32000)
    args = ap.parse_args()
    dev = torch.device("cuda:0")
    torch.manual_seed(0)
    teacher = torch.nn.Linear(args.hidden, args.vocab, bias=False, device=dev)
    with torch.no_grad():
        teacher.weight.mul_(4)
    # a coarse plan, so that there is something to heal
    student = htnn.HyperLinear.from_linear(teacher, inference_only=False, eps_int4=0.5)
    student.refresh_every = 4
    norm = htnn.AddRMSNorm(args.hidden, device=dev)
    opt = torch.optim.Adam([*student.parameters(), *norm.parameters()], lr=1e-4)
    weight = torch.full((args.rows,), 1.0 / args.rows, device=dev)
    torch.cuda.synchronize()
    began = time.perf_counter()
    for step in range(args.steps):
        x, stream = torch.randn(2, args.rows, args.hidden, device=dev)
        with torch.no_grad():
            h = x + stream
            logits = teacher(h * torch.rsqrt(h.square().mean(-1, keepdim=True) + norm.eps))
            kept = api.token_logprobs(logits, top=args.top)
        y, _ = norm(x, stream)
        out = student(y)
        loss = htnn.distill_loss(out, kept.top_tokens, kept.top_logprobs, weight)
        opt.zero_grad()
        loss.backward()
        opt.step()
        if step % 5 == 0 or step == args.steps - 1:
            mine = api.token_logprobs(out.detach(), kept.top_tokens[:, 0].contiguous(), top=1)
            agree = (mine.top_tokens[:, 0] == kept.top_tokens[:, 0]).float().mean().item()
            print(f"step {step}: loss {loss.item():.4f}, same token {agree:.3f}, "
                  f"its log probability {mine.logprobs.mean().item():.3f}, entropy {mine.entropy.mean().item():.3f}", flush=True)
    torch.cuda.synchronize()
    t = time.perf_counter() - began
    assert torch.isfinite(loss).item()
    print(f"{args.steps} steps of {args.rows} rows: {args.steps * args.rows / t:.0f} rows/s")
    return 0


if __name__ == "__main__":
    sys.exit(main())
