"""Serving from compressed records: prompts, then decode steps, then the end of
one request, on random weights.

Each step makes one plan from the requests' lengths and, per layer, rotates
the queries and keys, appends the new keys and values to the layer's INT4
records and attends over them; no page of 16-bit keys or values exists.

    python examples/serve_step.py [--layers N] [--steps N] [--fmt int4|fp8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from quantization_rope_reuse_amd import hkv  # noqa: E402

D = hkv.HEAD_DIM


class Server:
    """Fixed request rows over one pool of blocks per layer."""

    def __init__(self, layers=2, rows=4, q_heads=32, kv_heads=8, blocks=64, block_tokens=16, max_blocks=16,
                 max_tokens=256, fmt="int4", device="cuda", seed=0):
        self.fmt, self.tb, self.hq, self.hk = fmt, block_tokens, q_heads, kv_heads
        self.max_tokens = max_tokens
        i32 = dict(dtype=torch.int32, device=device)
        self.kv_len = torch.zeros(rows, **i32)
        self.table = torch.full((rows, max_blocks), -1, **i32)
        self.free = torch.arange(blocks, **i32)
        self.free_count = torch.tensor([blocks], **i32)
        self.records = [hkv.alloc_records(1, blocks, fmt, block_tokens, kv_heads, device=device)[0]
                        for _ in range(layers)]
        g = torch.Generator(device).manual_seed(seed)
        width = q_heads * D
        self.proj = [torch.randn(width, (q_heads + 2 * kv_heads) * D, device=device, generator=g)
                     .mul_(width ** -0.5).bfloat16() for _ in range(layers)]

    def step(self, x, new_tokens, max_queries):
        """x [n_tokens, q_heads * 128]: the packed hidden states of the new
        tokens (rows past the step's own are padding); new_tokens int32 per
        row, -1 where a request ends.  Returns (hidden states, plan)."""
        plan = hkv.plan_step(self.kv_len, new_tokens, self.table, self.free, self.free_count, self.tb, x.shape[0])
        self.kv_len, self.free_count = plan.kv_len, plan.free_count
        for w, records in zip(self.proj, self.records):
            qkv = (x @ w).view(x.shape[0], -1, D)
            q, k, v = qkv.split([self.hq, self.hk, self.hk], 1)
            hkv.rope_heads(q, k, plan.positions, 500000.0, "half_split", q_out=q, k_out=k)
            hkv.append_tokens(k, v, plan.slots, records, self.fmt, self.tb)
            out = torch.zeros_like(q, memory_format=torch.contiguous_format)
            hkv.attend_records(q, records, self.fmt, self.tb, self.hk, self.table, plan.kv_len, plan.q_start,
                               max_queries=max_queries, out=out)
            x = x + out.flatten(1)
            x = x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)
        return x, plan


def run(layers=2, steps=20, fmt="int4", device="cuda"):
    """Three prompts of different lengths, `steps` decode steps, the first
    request ends and another takes its row.  Returns every step's hidden
    states and plan."""
    s = Server(layers=layers, fmt=fmt, device=device)
    g = torch.Generator(device).manual_seed(1)
    i32 = dict(dtype=torch.int32, device=device)
    history = []

    def hidden(n):
        return torch.randn(n, s.hq * D, device=device, generator=g).bfloat16()

    prompts = [37, 5, 100]
    history.append(s.step(hidden(sum(prompts)), torch.tensor(prompts + [0], **i32), max(prompts)))
    for _ in range(steps):
        history.append(s.step(hidden(3), torch.tensor([1, 1, 1, 0], **i32), 1))
    history.append(s.step(hidden(22), torch.tensor([-1, 1, 1, 20], **i32), 20))
    history.append(s.step(hidden(12), torch.tensor([9, 1, 1, 1], **i32), 9))
    return s, history


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--fmt", default="int4", choices=["int4", "fp8"])
    a = ap.parse_args()
    server, history = run(a.layers, a.steps, a.fmt)
    x, plan = history[-1]
    print(f"{len(history)} steps, lengths {plan.kv_len.tolist()}, free blocks {int(plan.free_count)}, "
          f"|hidden| {float(x.float().norm()):.4f}")
