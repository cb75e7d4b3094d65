#!/usr/bin/env python3
"""A speculative verifier's sparse layer in MXFP4.

Experts' weights go into MXFP4 with quantize_mxfp4 and into the products' tiles
with qpack_mxfp4.  Then, step by step, the width-6 verifier routes its new
tokens (moe_route), takes them through their experts' gate and up projections
(moe_gate_up_mxfp4) and back (moe_down_mxfp4).  The step is captured once as a
CUDA graph: which expert has how many tokens is read on the device.  Unused
places of the batch have logits of minus infinity and come out as zeros.  At the end the
last step is compared with a dense layer of the weights' MXFP4 values.

    python examples/sparse_layer.py [--dtype float32|float16|bfloat16] [--steps N] [--tokens N]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

HIDDEN, INNER, EXPERTS, TOP_K = 1024, 352, 16, 4


def run(dtype: torch.dtype = torch.float32, steps: int = 4, tokens: int = 6, device: str = "cuda:0") -> float:
    """The steps; the largest difference from the dense layer, over the largest output."""
    from block_quantized_gemv_quantize_gb300 import ops

    g = torch.Generator(device=device)
    g.manual_seed(3)
    values, packs = [], []
    for n, k in ((INNER, HIDDEN), (INNER, HIDDEN), (HIDDEN, INNER)):
        blocks = ops.quantize_mxfp4(torch.randn((EXPERTS * n, k), generator=g, device=device) / math.sqrt(k))
        values.append(ops.dequantize_mxfp4(blocks).view(EXPERTS, n, k))
        packs.append(ops.qpack_mxfp4(blocks, EXPERTS, n, k))

    x = torch.zeros((tokens, HIDDEN), dtype=dtype, device=device)
    logits = torch.zeros((tokens, EXPERTS), device=device)

    def step():
        ids, weights, offsets, order = ops.moe_route(logits, TOP_K)
        h = ops.moe_gate_up_mxfp4(packs[0], packs[1], x, offsets, INNER, order, TOP_K)
        return ids, weights, h, ops.moe_down_mxfp4(packs[2], h, offsets, HIDDEN, order, weights)

    step()  # (loads the kernels, which a capture cannot)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, weights, h, out = step()
    for _ in range(steps):
        x.copy_(torch.randn((tokens, HIDDEN), generator=g, device=device))
        logits.copy_(torch.randn((tokens, EXPERTS), generator=g, device=device))
        logits[tokens - 1:] = -math.inf  # an unused place
        graph.replay()
    torch.cuda.synchronize()
    assert bool((out[tokens - 1:] == 0).all()) and bool((ids[tokens - 1:] == -1).all())

    want = torch.zeros((tokens, HIDDEN), dtype=torch.float64, device=device)
    for t in range(tokens - 1):
        for j in range(TOP_K):
            e = int(ids[t, j])
            gate, up = (v[e].double() @ x[t].double() for v in values[:2])
            want[t] += float(weights[t, j]) * (values[2][e].double() @ (gate * torch.sigmoid(gate) * up))
    return float((out.double() - want).abs().max() / want.abs().max())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--dtype", default="float32", choices=("float32", "float16", "bfloat16"))
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=6)
    a = ap.parse_args()
    print(f"largest difference from the dense layer: {run(getattr(torch, a.dtype), a.steps, a.tokens):.3g} of the largest output")


if __name__ == "__main__":
    main()
