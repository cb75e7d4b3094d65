#!/usr/bin/env python3
"""A speculative verifier's attention layer with a block-quantized paged cache.

Two sequences of different lengths share one cache.  A prompt's keys and values
go in with kv_write; then, step by step, the width-6 verifier projects its new
tokens (qgemv_q4_0 on one q|k|v weight), writes their keys and values,
attends to everything so far with attn_paged, and projects the result
(qgemv_q4_0).  The step is captured once as a CUDA graph: lengths, slots and
page tables are device tensors that the host changes between replays.  At the
end kv_read takes one sequence's cache back, and its last step's attention is
compared with a dense one over those values.

    python examples/verifier_attention.py [--format q8_0|q4_0|f16] [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

HIDDEN, HEADS, KV_HEADS, DIM, ROWS, PAGE = 5120, 40, 8, 128, 6, 64


def run(fmt: str = "q8_0", steps: int = 4, prompts: tuple[int, ...] = (197, 70), device: str = "cuda:0") -> float:
    """The steps; the largest difference from the dense attention."""
    from block_quantized_gemv_quantize_gb300 import ops, synth

    batch, n = len(prompts), len(prompts) * ROWS
    wide = (HEADS + 2 * KV_HEADS) * DIM
    w_qkv = ops.qpack_q4_0(torch.from_numpy(synth.q4_0_weights(wide, HIDDEN, seed=1)).to(device), wide, HIDDEN)
    w_out = ops.qpack_q4_0(torch.from_numpy(synth.q4_0_weights(HIDDEN, HEADS * DIM, seed=2)).to(device), HIDDEN,
                           HEADS * DIM)
    g = torch.Generator(device=device)
    g.manual_seed(3)

    # pages: each sequence takes them from one pool as it grows
    longest = max(prompts) + steps * ROWS
    per = -(-longest // PAGE)
    pages = batch * per
    table = torch.randperm(pages, generator=g, device=device).int().view(batch, per).contiguous()
    cache = torch.zeros((pages, ops.kv_page_bytes(fmt, PAGE, KV_HEADS, DIM)), dtype=torch.uint8, device=device)

    def slots_of(b: int, lo: int, hi: int) -> torch.Tensor:
        p = torch.arange(lo, hi, device=device)
        return table[b].long()[p // PAGE] * PAGE + p % PAGE

    for b, length in enumerate(prompts):
        k, v = (torch.randn((length, KV_HEADS, DIM), generator=g, device=device) for _ in range(2))
        ops.kv_write(cache, k, v, slots_of(b, 0, length), fmt, PAGE)

    x = torch.empty((n, HIDDEN), device=device)
    slots = torch.empty(n, dtype=torch.int64, device=device)
    lens = torch.empty(batch, dtype=torch.int32, device=device)

    def step():
        qkv = ops.qgemv_q4_0(w_qkv, ops.quantize_q8_1(x), n, HIDDEN, wide).view(n, HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
        ops.kv_write(cache, k, v, slots, fmt, PAGE)
        a = ops.attn_paged(q, cache, table, lens, fmt, PAGE, KV_HEADS, rows=ROWS)
        return q, a, ops.qgemv_q4_0(w_out, ops.quantize_q8_1(a.view(n, HEADS * DIM)), n, HEADS * DIM, HIDDEN)

    def inputs(i: int) -> list[int]:
        x.copy_(torch.randn((n, HIDDEN), generator=g, device=device))
        now = [p + (i + 1) * ROWS for p in prompts]
        slots.copy_(torch.cat([slots_of(b, m - ROWS, m) for b, m in enumerate(now)]))
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        return now

    inputs(0)
    step()  # the first call of a kernel is not one to capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, a, y = step()
    for i in range(steps):
        now = inputs(i)
        graph.replay()

    # one sequence's last step, densely over what the cache holds
    b, length = batch - 1, now[-1]
    k, v = ops.kv_read(cache, slots_of(b, 0, length), fmt, PAGE, KV_HEADS, DIM)
    rows = slice(b * ROWS, (b + 1) * ROWS)
    k, v = (t.double().repeat_interleave(HEADS // KV_HEADS, 1) for t in (k, v))
    score = torch.einsum("rhd,phd->hrp", q[rows].double(), k) / DIM ** 0.5
    end = length - ROWS + 1 + torch.arange(ROWS, device=device)
    score = score.masked_fill(torch.arange(length, device=device) >= end[:, None], float("-inf"))
    want = torch.einsum("hrp,phd->rhd", torch.softmax(score, -1), v)
    assert bool(torch.isfinite(y).all())
    return float((a[rows].double() - want).abs().max())


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--format", default="q8_0", choices=["q8_0", "q4_0", "f16"])
    p.add_argument("--steps", type=int, default=4)
    a = p.parse_args()
    print(f"{a.format}: largest difference from dense attention over the cache's values {run(a.format, a.steps):.2e}")


if __name__ == "__main__":
    main()
