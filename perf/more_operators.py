"""A sparse layer in microscaled 4-bit floating point: what is measured, and each
operator in its plain form.

MXFP4 (blocks of 32 values of one row, 17 bytes): a byte e, the block's scale
2^(e - 127), then 16 bytes of codes, value i < 16 in the low nibble of byte i
and value i + 16 in its high nibble.  A code is sign, two bits of exponent and
one of mantissa: 0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives.
    quantize    e = 127 + floor(log2 max|x|) - 2, limited to 0 .. 254; the code
                nearest to x / 2^(e - 127), of two equally near the even one, at
                most 6; a block of zeros has e = 0, one that holds a NaN or an
                infinity e = 255, which makes all its values NaN

The router gives each token the top_k experts of largest logit (of equal ones
the lowest), never one whose logit is minus infinity or NaN: a place that no
expert is left for has id -1 and weight 0.
    softmax     weight = softmax over all experts at the chosen one
    sigmoid     weight = 1 / (1 + e^-logit)
    then, where asked, divided by the token's sum of weights; times `scale`
Place j of token t is slot t top_k + j.  `order` has the slots of expert 0, then
those of expert 1 and so on, each expert's ascending, at its end the slots
without one; expert e's are order[offsets[e]] .. order[offsets[e + 1] - 1].

The products, e(s) being the expert of slot s (a slot without one gives zeros):
    gemm        y[s] = W_e(s) x[s / top_k]
    gate_up     h[s] = silu(G_e(s) x[s / top_k]) U_e(s) x[s / top_k]
    down        out[t] = sum_j weight[t, j] W_e(s) h[s],  s = t top_k + j
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 32
BLOCK_BYTES = 17
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # odd rows of a projection, cut out of a wider tensor
        dict(name="quantize_rows", op="quantize", dtype="f16", n=199, k=1056, wide=True),
        # the down projections of a layer's experts, from a training checkpoint
        dict(name="quantize_experts", op="quantize", dtype="bf16", n=32 * 5120, k=1408, wide=False),
        # one token's router: latency only
        dict(name="route_token", op="route", dtype="f32", tokens=1, experts=64, top_k=6, score="softmax",
             renormalize=True, scale=1.0, pad=0, masked=0),
        # a long prompt's router with sigmoid scores, padded, some experts switched off
        dict(name="route_prompt", op="route", dtype="bf16", tokens=17391, experts=128, top_k=8, score="sigmoid",
             renormalize=True, scale=2.5, pad=37, masked=3),
        # a dense layer in four bits under the widest verifier: one expert
        dict(name="gemm_dense17", op="gemm", dtype="bf16", tokens=17, experts=1, top_k=1, k=5120, n=17408, pad=0),
        # few large experts, ragged, sizes that fill no tile
        dict(name="gemm_ragged", op="gemm", dtype="f16", tokens=2999, experts=8, top_k=2, k=1056, n=4104, pad=11),
        # one token of a sparse layer: the experts' weights and nothing else
        dict(name="gate_up_token", op="gate_up", dtype="bf16", tokens=1, experts=64, top_k=6, k=5120, n=1408, pad=0),
        # the width-6 verifier
        dict(name="gate_up_verify6", op="gate_up", dtype="f32", tokens=6, experts=64, top_k=6, k=5120, n=1408, pad=0),
        # a prompt
        dict(name="gate_up_prompt", op="gate_up", dtype="bf16", tokens=4096, experts=64, top_k=6, k=5120, n=1408,
             pad=0),
        dict(name="down_verify6", op="down", dtype="f32", tokens=6, experts=64, top_k=6, k=1408, n=5120, pad=0),
        # a batch of single tokens over many small experts, some of its places unused
        dict(name="down_batch", op="down", dtype="bf16", tokens=96, experts=128, top_k=8, k=768, n=2048, pad=5),
        dict(name="down_prompt", op="down", dtype="bf16", tokens=4096, experts=64, top_k=6, k=1408, n=5120, pad=0),
    ]


def _spread(rng, lo, hi):
    """A whole number, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _drawn(rng)
    limit = {n: max(work(c)[n] for c in listed() if c["op"] == case["op"]) for n in ("bytes", "flops")}
    while any(work(case)[n] > limit[n] for n in limit):  # no dearer than the dearest listed one
        size = "tokens" if case.get("tokens", 1) > 1 else "experts" if case.get("experts", 1) > 8 else "n"
        case[size] = max(1, case[size] * 3 // 4)
        if "pad" in case:
            case["pad"] = 0
        if "top_k" in case:
            case["top_k"] = min(case["top_k"], case["experts"])
    return case


def _drawn(rng):
    op = rng.choice(["quantize", "route", "gemm", "gate_up", "gate_up", "down", "down"])
    dtype = rng.choice(["bf16", "bf16", "f32", "f16"])
    if op == "quantize":
        k = BLOCK * _spread(rng, 1, 176)
        return dict(op=op, dtype=dtype, n=_spread(rng, 1, 2 ** 27 // k), k=k, wide=rng.random() < 0.5)
    experts = rng.choice([1, 4, 8, 16, 60, 64, 96, 128, 256])
    top_k = min(experts, rng.choice([1, 2, 4, 6, 8]))
    tokens = _spread(rng, 1, 20000 if op == "route" else 6000)
    pad = rng.choice([0, 0, min(7, tokens - 1)])
    if op == "route":
        return dict(op=op, dtype=dtype, tokens=tokens, experts=experts, top_k=top_k,
                    score=rng.choice(["softmax", "softmax", "sigmoid"]), renormalize=rng.random() < 0.6,
                    scale=rng.choice([1.0, 1.0, 2.5]), pad=pad, masked=rng.choice([0, 0, experts // 3]))
    k = BLOCK * _spread(rng, 2, 160)
    return dict(op=op, dtype=dtype, tokens=tokens, experts=experts, top_k=top_k, k=k,
                n=rng.choice([1, 4, 8, 32]) * _spread(rng, 8, 160), pad=pad)


def _ids(case):
    """The slots' experts [tokens][top_k], some of them far more popular than
    others and -1 for the padding: part of the case, not of the seed."""
    tokens, experts, top_k = case["tokens"], case["experts"], case["top_k"]
    g = torch.Generator()
    g.manual_seed(tokens * 1000003 + experts * 1009 + top_k)
    liked = 0.7 * torch.randn(experts, generator=g)
    noise = -torch.log(-torch.log(torch.rand((tokens, experts), generator=g).clamp(1e-7, 1 - 1e-7)))
    ids = torch.argsort(liked + noise, dim=-1, descending=True)[:, :top_k]
    ids[tokens - case["pad"]:] = -1
    return ids


# ------------------------------------------------------------------ the plain form


def _power(n):
    """2^n in fp64, from its bits, for whole n."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _quantize(x):
    """x [rows, K] -> uint8 [rows, K / 32, 17]."""
    x = x.float().unflatten(-1, (-1, BLOCK))
    mag = x.abs()
    top = mag.amax(-1, keepdim=True)
    fine = torch.isfinite(mag).all(-1, keepdim=True)
    e = (torch.frexp(torch.where(fine, top, torch.ones_like(top)))[1] - 3 + 127).clamp(0, 254)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    # (in 64 bits: the quotient of a block whose scale is 2^127 or 2^-127)
    y = torch.where(fine, mag, torch.zeros_like(mag)).double() * _power(127 - e)
    code = torch.zeros(y.shape, dtype=torch.uint8, device=x.device)
    for c in range(7):  # above the middle of two neighbours, or on it with the upper one even
        middle = (GRID[c] + GRID[c + 1]) / 2
        code += (y >= middle) if c % 2 else (y > middle)
    code |= (torch.signbit(x) & fine).to(torch.uint8) << 3
    e = torch.where(fine, e, torch.full_like(e, 255)).to(torch.uint8)
    return torch.cat([e, code[..., :16] | code[..., 16:] << 4], -1)


def _dequantize(blocks):
    """uint8 [rows, K / 32, 17] -> fp32 [rows, K]."""
    e = blocks[..., :1].int()
    code = torch.cat([blocks[..., 1:] & 15, blocks[..., 1:] >> 4], -1)
    value = torch.tensor(GRID + [-v for v in GRID], device=blocks.device)[code.int()]
    scale = torch.where(e == 255, torch.full_like(value[..., :1], math.nan), _power(e - 127).float())
    return (value * scale).flatten(-2)


def _plain_route(s):
    case = s["case"]
    logits = s["logits"].float()
    logits = torch.where(torch.isnan(logits), torch.full_like(logits, -math.inf), logits)
    ranked, at = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, ids = ranked[:, :case["top_k"]], at[:, :case["top_k"]]
    live = top > -math.inf
    if case["score"] == "softmax":
        best = ranked[:, :1]
        best = torch.where(torch.isinf(best), torch.zeros_like(best), best)
        weights, total = torch.exp(top - best), torch.exp(ranked - best).sum(-1, keepdim=True)
        if case["renormalize"]:
            total = weights.sum(-1, keepdim=True)
    else:
        weights = 1.0 / (1.0 + torch.exp(-top))
        total = weights.sum(-1, keepdim=True) if case["renormalize"] else torch.ones_like(weights[:, :1])
    weights = weights / torch.where(live.any(-1, keepdim=True), total, torch.ones_like(total)) * case["scale"]
    weights = torch.where(live, weights, torch.zeros_like(weights))
    ids = torch.where(live, ids, torch.full_like(ids, -1)).int()
    key = torch.where(ids < 0, case["experts"], ids).flatten()
    order = torch.sort(key, stable=True).indices.int()
    counts = (key[:, None] == torch.arange(case["experts"], device=key.device)).sum(0)
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)]).int()
    return ids, weights, offsets, order


def _plain_products(s):
    case = s["case"]
    slots, n = case["tokens"] * case["top_k"], case["n"]
    down = case["op"] == "down"
    y = torch.zeros((slots, n), device="cuda")
    done = 0
    for e, count in enumerate(s["counts"]):
        if count:
            at = s["order"][done:done + count].long()
            x = s["x"][at if down else at // case["top_k"]].float()
            rows = [x @ _dequantize(w[e]).t() for w in s["blocks"]]
            y[at] = rows[0] if len(rows) == 1 else rows[0] / (1.0 + torch.exp(-rows[0])) * rows[1]
            done += count
    if down:
        y = (y.view(case["tokens"], case["top_k"], n) * s["weights"][..., None]).sum(1)
    return y.to(s["dtype"])


# ------------------------------------------------------------------ inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _rows(shape, g):
    """Activations: a few strong channels."""
    x = torch.randn(shape, generator=g, device="cuda")
    return torch.where(torch.rand(shape[-1:], generator=g, device="cuda") < 0.01, 12.0 * x, x)


def prepare(case, seed):
    g = _generator(seed)
    op, dtype = case["op"], TYPES[case["dtype"]]
    state = dict(case=case, dtype=dtype)
    if op == "quantize":
        k = case["k"]
        x = torch.empty((case["n"], k + 40 if case["wide"] else k), dtype=dtype, device="cuda")
        for lo in range(0, case["n"], 8192):  # a bounded piece at a time; rows of different size
            part = torch.randn((min(8192, case["n"] - lo), x.shape[1]), generator=g, device="cuda")
            x[lo:lo + 8192] = part * torch.exp(torch.randn((part.shape[0], 1), generator=g, device="cuda") - 4.0)
        state["x"] = x[:, 8:k + 8] if case["wide"] else x
        return state
    tokens, experts, top_k = case["tokens"], case["experts"], case["top_k"]
    if op == "route":
        logits = 2.0 * torch.randn((tokens, experts), generator=g, device="cuda")
        logits += torch.randn(experts, generator=g, device="cuda")
        off = torch.randperm(experts, generator=g, device="cuda")[:case["masked"]]
        logits[:, off] = -math.inf
        logits[tokens - case["pad"]:] = -math.inf
        state["logits"] = logits.to(dtype)
        return state
    n, k = case["n"], case["k"]
    ids = _ids(case).flatten()
    key = torch.where(ids < 0, experts, ids)
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    state["counts"] = counts.tolist()
    state["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).int().cuda()
    state["order"] = torch.sort(key, stable=True).indices.int().cuda()
    state["blocks"] = []
    for _ in range(2 if op == "gate_up" else 1):
        blocks = torch.empty((experts, n, k // BLOCK, BLOCK_BYTES), dtype=torch.uint8, device="cuda")
        for e in range(experts):
            blocks[e] = _quantize(torch.randn((n, k), generator=g, device="cuda") * (0.7 / math.sqrt(k)))
        state["blocks"].append(blocks)
    if op == "down":
        h = _rows((tokens * top_k, k), g)
        state["x"] = (h * torch.rand(h.shape, generator=g, device="cuda")).to(dtype)
        weights = torch.rand((tokens, top_k), generator=g, device="cuda") + 0.05
        state["weights"] = weights / weights.sum(-1, keepdim=True)
        state["weights"][ids.view(tokens, top_k).cuda() < 0] = 0.0
    else:
        state["x"] = _rows((tokens, k), g).to(dtype)
    if own:
        from block_quantized_gemv_quantize_gb300 import ops

        state["packs"] = [ops.qpack_mxfp4(b, experts, n, k) for b in state["blocks"]]
    return state


# ------------------------------------------------------------------ one pass


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from block_quantized_gemv_quantize_gb300 import ops

        if op == "quantize":
            return ops.dequantize_mxfp4(ops.quantize_mxfp4(state["x"]), dtype=state["dtype"])
        if op == "route":
            return ops.moe_route(state["logits"], case["top_k"], score=case["score"],
                                 renormalize=case["renormalize"], scale=case["scale"])
        if op == "gemm":
            return ops.qgemm_mxfp4(*state["packs"], state["x"], state["offsets"], case["n"], order=state["order"],
                                   top_k=case["top_k"])
        if op == "gate_up":
            return ops.moe_gate_up_mxfp4(*state["packs"], state["x"], state["offsets"], case["n"], state["order"],
                                         case["top_k"])
        return ops.moe_down_mxfp4(*state["packs"], state["x"], state["offsets"], case["n"], state["order"],
                                  state["weights"])
    if op == "quantize":
        return torch.cat([_dequantize(_quantize(x)).to(state["dtype"]) for x in state["x"].split(32768)])
    return _plain_route(state) if op == "route" else _plain_products(state)


def work(case):
    size = BYTES[case["dtype"]]
    if case["op"] == "quantize":
        values = case["n"] * case["k"]
        return {"bytes": 2 * values * size + 2 * (values // BLOCK) * BLOCK_BYTES, "flops": 4 * values}
    tokens, slots = case["tokens"], case["tokens"] * case["top_k"]
    if case["op"] == "route":
        return {"bytes": tokens * case["experts"] * size + 12 * slots + 4 * (case["experts"] + 1),
                "flops": 4 * tokens * case["experts"]}
    ids = _ids(case)
    live, used = int((ids >= 0).sum()), int(torch.unique(ids[ids >= 0]).numel())
    weights = 2 if case["op"] == "gate_up" else 1
    n, k = case["n"], case["k"]
    held = weights * used * n * (k // BLOCK) * BLOCK_BYTES
    if case["op"] == "down":
        rows = live * k * size + tokens * n * size + 4 * slots
    else:
        rows = (tokens - case["pad"]) * k * size + slots * n * size
    return {"bytes": held + rows + 4 * slots + 4 * (case["experts"] + 1), "flops": 2 * weights * live * n * k}


# ------------------------------------------------------------------ the definition, in 64 bits


def _two_to(n):
    """2^n in fp64 (a library power need not be exact), n whole and above -1023."""
    table = torch.tensor([math.ldexp(1.0, i) for i in range(-300, 301)], dtype=torch.float64, device=n.device)
    return table[n + 300]


def _exact_values(blocks):
    """uint8 [rows, K / 32, 17] -> fp64 [rows, K], from the bits of the codes."""
    b = blocks.to(torch.int64)
    both = torch.stack([b[..., 1:] % 16, b[..., 1:] // 16], dim=-2).flatten(-2)
    exponent, mantissa = both // 2 % 4, both % 2
    size = torch.where(exponent == 0, mantissa * 0.5,
                       (1.0 + 0.5 * mantissa.double()) * (2 ** exponent // 2).double())
    size = size * (1 - 2 * (both // 8)).double()
    scale = _two_to(b[..., :1] - 127)
    return (size * torch.where(b[..., :1] == 255, torch.full_like(scale, math.nan), scale)).flatten(-2)


def _exact_rounded(x):
    """The values that a quantized x holds, in fp64."""
    x = x.double().reshape(x.shape[0], -1, BLOCK)
    top = x.abs().max(dim=-1, keepdim=True).values
    power = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))).clamp(-200, 200).long()
    power = torch.where(_two_to(power) > top, power - 1, power)  # (where the logarithm rounds to the next whole one)
    power = torch.where(_two_to(power + 1) <= top, power + 1, power)
    unit = _two_to((power - 2).clamp(-127, 127))
    y = x.abs() / unit
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    return (torch.sign(x) * torch.clamp(torch.round(y / step) * step, max=6.0) * unit).flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return torch.cat([_exact_rounded(x) for x in s["x"].split(16384)])
    if case["op"] == "route":
        logits = s["logits"].double()
        tokens, top_k = case["tokens"], case["top_k"]
        ids = torch.full((tokens, top_k), -1, dtype=torch.int32, device="cuda")
        weights = torch.zeros((tokens, top_k), dtype=torch.float64, device="cuda")
        left = torch.nan_to_num(logits, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
        score = torch.softmax(left, dim=-1) if case["score"] == "softmax" else torch.sigmoid(left)
        column = torch.arange(case["experts"], device="cuda")
        for j in range(top_k):
            top = left.max(dim=-1, keepdim=True).values
            first = torch.where(left == top, column, case["experts"]).min(dim=-1).values
            live = top[:, 0] > -math.inf
            ids[live, j] = first[live].to(torch.int32)
            weights[live, j] = score[live, first[live]]
            left = torch.where(column == first[:, None], -math.inf, left)
        if case["renormalize"]:
            weights = weights / torch.where(weights > 0, weights, 0.0).sum(-1, keepdim=True).clamp(min=1e-300)
        lists = [[] for _ in range(case["experts"] + 1)]
        for slot, e in enumerate(ids.flatten().tolist()):
            lists[e].append(slot)  # (-1: the last)
        ends = [0]
        for found in lists[:-1]:
            ends.append(ends[-1] + len(found))
        whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return ids, weights * case["scale"], whole(ends), whole([slot for found in lists for slot in found])
    ids, n, top_k = _ids(case).cuda(), case["n"], case["top_k"]
    out = torch.zeros((case["tokens"] * (1 if case["op"] == "down" else top_k), n), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        token, place = torch.nonzero(ids == e, as_tuple=True)
        if not token.numel():
            continue
        values = [_exact_values(b[e]) for b in s["blocks"]]
        slot = token * top_k + place
        if case["op"] == "down":
            out.index_add_(0, token, (s["x"][slot].double() @ values[0].T) * s["weights"][token, place].double()[:, None])
            continue
        x = s["x"][token].double()
        if case["op"] == "gemm":
            out[slot] = x @ values[0].T
        else:
            gate = x @ values[0].T
            out[slot] = gate * torch.sigmoid(gate) * (x @ values[1].T)
    return out
