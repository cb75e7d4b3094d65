"""Plain 64-bit implementation of the MXFP4 format and of the sparse layer's
calls, from their definitions (include/qgemv.h), and the bounds that the
library's fp32 arithmetic has against it.  Test code only."""
import math

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def quantize(x):
    """x [N, K] (CPU) -> uint8 [N, K/32, 17], one block at a time in Python numbers."""
    x = x.double()
    N, K = x.shape
    out = torch.zeros((N, K // 32, 17), dtype=torch.uint8)
    for n in range(N):
        for b in range(K // 32):
            v = x[n, 32 * b:32 * b + 32].tolist()
            if not all(math.isfinite(f) for f in v):
                out[n, b, 0] = 255
                continue
            top = max(abs(f) for f in v)
            e = 0 if top == 0 else min(254, max(0, 127 + math.frexp(top)[1] - 1 - 2))
            codes = []
            for f in v:
                y = abs(f) * 2.0 ** (127 - e)
                code = min(range(8), key=lambda c: (abs(y - float(GRID[c])), c % 2))
                codes.append(code | (8 if math.copysign(1.0, f) < 0 else 0))
            out[n, b, 0] = e
            for i in range(16):
                out[n, b, 1 + i] = codes[i] | codes[i + 16] << 4
    return out


def values(blocks):
    """uint8 [..., K/32, 17] -> fp64 [..., K]."""
    code = torch.cat([blocks[..., 1:] & 15, blocks[..., 1:] >> 4], -1).long()
    v = GRID.to(blocks.device)[code & 7] * (1 - 2 * (code >> 3)).double()
    scale = ((blocks[..., 0].long() - 127 + 1023) << 52).view(torch.float64)
    scale = torch.where(blocks[..., 0] == 255, torch.full_like(scale, math.nan), scale)
    return (v * scale[..., None]).reshape(*blocks.shape[:-2], -1)


def random_blocks(g, *shape, lo=118, hi=124):
    """Blocks [*shape[:-1], shape[-1]/32, 17] of random codes and scales."""
    blocks = torch.randint(0, 256, (*shape[:-1], shape[-1] // 32, 17), generator=g, dtype=torch.uint8)
    blocks[..., 0] = torch.randint(lo, hi, blocks.shape[:-1], generator=g, dtype=torch.uint8)
    return blocks


def route(logits, top_k, score, renormalize, scale):
    """(ids, weights fp64) of logits [T, E] (CPU)."""
    ids, weights = [], []
    for row in logits.double().tolist():
        alive = [(-l, e) for e, l in enumerate(row) if l > -math.inf]
        chosen = sorted(alive)[:top_k]
        top = -min(alive)[0] if alive else 0.0
        if score == "softmax":
            total = sum(math.exp(-l - top) for l, _ in alive)
            w = [math.exp(-l - top) / total for l, _ in chosen]
            logs = [-l for l, _ in chosen]
        else:
            logs = [(-math.log1p(math.exp(l)) if l < 0 else -l - math.log1p(math.exp(-l))) for l, _ in chosen]
            w = [math.exp(l) for l in logs]
        if renormalize and chosen:
            w = [math.exp(l - max(logs)) for l in logs]
            w = [v / sum(w) for v in w]
        ids.append([e for _, e in chosen] + [-1] * (top_k - len(chosen)))
        weights.append([v * scale for v in w] + [0.0] * (top_k - len(chosen)))
    return torch.tensor(ids, dtype=torch.int32).view(-1, top_k), torch.tensor(weights, dtype=torch.float64).view(-1, top_k)


def group(ids, experts):
    """(offsets, order) int32 of ids [T, k]."""
    flat = ids.flatten().tolist()
    lists = [[] for _ in range(experts + 1)]
    for slot, e in enumerate(flat):
        lists[e if 0 <= e < experts else experts].append(slot)
    ends = [0]
    for part in lists[:-1]:
        ends.append(ends[-1] + len(part))
    return torch.tensor(ends, dtype=torch.int32), torch.tensor([s for part in lists for s in part], dtype=torch.int32)


def product(w, x, ids, rows_of):
    """(y, bound) [slots, N] fp64: each slot's row through its expert's weight,
    and how far fp32 sums of it may be off: a rounding of every operand of x
    (2^-23 of it and 2^-38 of its row's largest), the sums of 32 products (32
    roundings of a tensor core, which may cut: 2^-23 each), a fused
    multiply-add a block and the sum over the warps that share K."""
    K = x.shape[1]
    y = torch.zeros((ids.numel(), w.shape[1]), dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(y)
    x64 = x.double()
    for e in range(w.shape[0]):
        s = torch.nonzero(ids.flatten() == e)[:, 0]
        if s.numel():
            xe = x64[rows_of(s)]
            y[s] = xe @ w[e].T
            mag = xe.abs() @ w[e].abs().T
            top = xe.abs().amax(-1, keepdim=True) * w[e].abs().sum(-1)
            bound[s] = mag * (2.0 ** -23 + 32 * 2.0 ** -23 + (K / 32 + 16) * 2.0 ** -24) + top * 2.0 ** -38
    return y, bound


def rounded(value, bound, dtype):
    """A bound for the value's rounding to dtype (smallest steps included), on top of its own."""
    tiny = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[dtype]
    return bound + HALF_STEP[dtype] * (value.abs() + bound) + tiny


def gate_up(gate, gate_bound, up, up_bound):
    """silu(gate) * up with the bounds of its factors carried on (|silu'| <= 1.1;
    exp, sum, quotient and product: 8 roundings)."""
    s = gate * torch.sigmoid(gate)
    h = s * up
    return h, 1.1 * gate_bound * (up.abs() + up_bound) + s.abs() * up_bound + h.abs() * 8 * 2.0 ** -24


def down(y, bound, weights):
    """The weighted sum of a token's slots, a fused multiply-add each."""
    T, k = weights.shape
    w = weights.double()[..., None]
    terms = y.view(T, k, -1) * w
    return terms.sum(1), (bound.view(T, k, -1) * w.abs()).sum(1) + terms.abs().sum(1) * k * 2.0 ** -24


def close(got, want, bound):
    """got within bound of want everywhere, NaN and infinities in the same places."""
    got = got.double()
    same = (got == want) | (got.isnan() & want.isnan())
    off = (got - want).abs()
    ok = same | (off <= bound)
    assert bool(ok.all()), f"{int((~ok).sum())} of {ok.numel()} off, worst by {float((off / bound)[~ok].max()):.3g} bounds"
