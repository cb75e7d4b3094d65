"""The block-quantized paged key-value cache and the attention that reads it:
what is measured, and each operator in its plain form.

The cache is a pool of pages (uint8 [pages, page bytes]).  A page holds
`page_tokens` tokens (a multiple of 16) of every kv head:

    page = [kv head][tile of 16 tokens]
    tile = K codes [D/32][16 tokens][32 values], K scales [D/32][16] fp16,
           V codes, V scales the same

(the scale of the tile's token r is at place 4 s + r / 4 of its 16, s = r % 4
where r / 4 is even and 3 - r % 4 where it is odd) with one block of 32 values of one token as the unit of the format:
    q8_0  d = max|x| / 127, code = x / d rounded half away from zero, stored
          as code + 128 in one byte; the value is d code
    q4_0  d = -m / 8 with m the value of largest magnitude (the first of
          equals), code = floor(x / d + 8.5) limited to 0 .. 15, the nibbles of
          values i and i + 16 in byte i; the value is d (code - 8)
    f16   the values in fp16, no scales
d, x / d and x / d + 8.5 are fp32; the stored d is its fp16 rounding (at most
65504 in magnitude; NaN, with codes of zero value, for a block that holds a
NaN or an infinity).  A token's place is its slot, page * page_tokens +
offset; a slot outside the pool is skipped when written and reads as zeros.

Attention: sequence b has `rows` new tokens (q rows b rows .. b rows + rows - 1)
at the end of its first kv_lens[b] tokens, which page_table[b] maps to pages.
Row i sees the positions p < kv_lens[b] - (rows - 1 - i), of those the last
`window` ones where window > 0; a row that sees none gives zeros.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
VALUE_BYTES = {"q8_0": 34 / 32, "q4_0": 18 / 32, "f16": 2.0}
TILE = 16


def listed():
    return [
        # a draft's first tokens after a short prompt: one row, latency only
        dict(name="attn_short", op="attn", fmt="q8_0", dtype="f32", page=16, batch=1, rows=1, heads=40, kv_heads=8,
             dim=128, len_lo=197, len_hi=197, empty=0, window=0, fused=True),
        # the width-6 verifier on one sequence of hidden size 5120
        dict(name="attn_verify6", op="attn", fmt="q8_0", dtype="f32", page=64, batch=1, rows=6, heads=40, kv_heads=8,
             dim=128, len_lo=17391, len_hi=17391, empty=0, window=0, fused=True),
        # ordinary serving: a batch of ragged sequences, two of its places unused
        dict(name="attn_batch", op="attn", fmt="q8_0", dtype="bf16", page=32, batch=48, rows=1, heads=40, kv_heads=8,
             dim=128, len_lo=1, len_hi=8192, empty=2, window=0, fused=False),
        # single tokens over two very long caches
        dict(name="attn_long", op="attn", fmt="q4_0", dtype="f16", page=128, batch=2, rows=1, heads=40, kv_heads=8,
             dim=128, len_lo=131071, len_hi=131071, empty=0, window=0, fused=True),
        # the widest verifier with a sliding window and sequences shorter than it
        dict(name="attn_verify17_window", op="attn", fmt="q4_0", dtype="f32", page=16, batch=5, rows=17, heads=20,
             kv_heads=4, dim=256, len_lo=3, len_hi=20001, empty=0, window=4096, fused=False),
        # one kv head for each query head, an unquantized cache, pages that are no power of two
        dict(name="attn_heads_f16", op="attn", fmt="f16", dtype="f16", page=48, batch=12, rows=2, heads=32,
             kv_heads=32, dim=64, len_lo=1, len_hi=4099, empty=1, window=0, fused=False),
        # the verifier step's six new tokens into the cache and back: latency only
        dict(name="write_step", op="write", fmt="q8_0", dtype="f32", page=16, tokens=6, kv_heads=8, dim=128, skip=0,
             fused=True),
        # a long prompt's keys and values
        dict(name="write_prompt", op="write", fmt="q8_0", dtype="bf16", page=64, tokens=17408, kv_heads=8, dim=128,
             skip=0, fused=True),
        # an odd prompt padded in front, wide heads, four bits
        dict(name="write_prompt_q4", op="write", fmt="q4_0", dtype="f32", page=16, tokens=4999, kv_heads=4, dim=256,
             skip=37, fused=False),
        # a short prefix taken out of the cache
        dict(name="read_prefix", op="read", fmt="q4_0", dtype="f32", page=32, tokens=97, kv_heads=8, dim=128, skip=0),
        # a whole long cache read back for a dense pass
        dict(name="read_long", op="read", fmt="q8_0", dtype="bf16", page=128, tokens=131071, kv_heads=8, dim=128,
             skip=3),
    ]


def _spread(rng, lo, hi):
    """A whole number, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _drawn(rng)
    size = "len_hi" if case["op"] == "attn" else "tokens"
    limit = {n: max(work(c)[n] for c in listed() if c["op"] == case["op"]) for n in ("bytes", "flops")}
    while any(work(case)[n] > limit[n] for n in limit):  # no dearer than the dearest listed one
        case[size] = case[size] * 3 // 4
        case["len_lo" if size == "len_hi" else "skip"] = 1 if size == "len_hi" else 0
    return case


def _drawn(rng):
    op = rng.choice(["attn", "attn", "attn", "write", "read"])
    fmt = rng.choice(["q8_0", "q8_0", "q4_0", "q4_0", "f16"])
    dtype = rng.choice(["f32", "f32", "f16", "bf16"])
    page = 16 * rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([64, 96, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 8])
    if op != "attn":
        most = 17408 * 1024 if op == "write" else 131071 * 1024
        tokens = _spread(rng, 1, min(most // (kv_heads * dim), 131071))
        skip = rng.choice([0, 0, min(5, tokens - 1)])
        case = dict(op=op, fmt=fmt, dtype=dtype, page=page, tokens=tokens, kv_heads=kv_heads, dim=dim, skip=skip)
        if op == "write":
            case["fused"] = rng.random() < 0.5
        return case
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 6, 8) if 3 << 10 not in (g * kv_heads * dim, (g + 2) * kv_heads * dim)])
    rows = rng.choice([1, 1, 1, 2, 3, 6, 6, 9, 17])
    batch = _spread(rng, 1, 64)
    # the values of the whole batch's cache, and its scores, stay below the largest listed case's
    cap = int(min(2 * 131071 * 1024 / (batch * kv_heads * dim), 1.2e9 / (batch * kv_heads * group * rows * dim)))
    len_hi = _spread(rng, min(16, cap), min(cap, 131071))
    len_lo = rng.choice([len_hi, 1 + len_hi // 3, min(1 + rows // 2, len_hi)])
    return dict(op=op, fmt=fmt, dtype=dtype, page=page, batch=batch, rows=rows, heads=group * kv_heads,
                kv_heads=kv_heads, dim=dim, len_lo=len_lo, len_hi=len_hi,
                empty=rng.choice([0, 0, 1]) if batch > 2 else 0,
                window=rng.choice([0, 0, 0, 1 + len_hi // 2, 128]), fused=rng.random() < 0.5)


def _lens(case):
    """The sequences' lengths: part of the case, not of the seed."""
    b, lo, hi = case["batch"], case["len_lo"], case["len_hi"]
    r = random.Random(b * 1000003 + lo * 1009 + hi)
    lens = [hi] + [r.randint(lo, hi) for _ in range(b - 1)]
    for i in range(case["empty"]):
        lens[1 + i] = 0
    return lens


# ------------------------------------------------------------------ the plain form: format


def _half_bytes(fmt, dim):
    """Bytes of a tile's codes and scales of K (or of V)."""
    blocks = dim // 32
    if fmt == "f16":
        return blocks * TILE * 64, 0
    return blocks * TILE * (32 if fmt == "q8_0" else 16), blocks * TILE * 2


def _quantize(x, fmt):
    """x [..., D] -> (codes uint8 [..., D/32, code bytes], scales fp16 [..., D/32])."""
    x = x.float().unflatten(-1, (-1, 32))
    if fmt == "f16":
        return x.half().contiguous().view(torch.uint8), None
    mag = x.abs()
    top = mag.amax(-1, keepdim=True)
    fine = torch.isfinite(top)
    if fmt == "q8_0":
        d = top / torch.full_like(top, 127.0)
    else:
        at = torch.where(mag == top, torch.arange(32, device=x.device), 32).amin(-1, keepdim=True).clamp(max=31)
        d = x.gather(-1, at) * -0.125
    y = torch.where((d != 0) & fine, x / torch.where(d != 0, d, torch.ones_like(d)), torch.zeros_like(x))
    scale = torch.where(fine, d.clamp(-65504.0, 65504.0), torch.full_like(d, math.nan))
    if fmt == "q8_0":
        mag = y.abs()
        whole = mag.floor()
        code = (whole + (mag - whole >= 0.5)).clamp(max=127.0) * y.sign() + 128.0
        return code.to(torch.uint8), scale[..., 0].half()
    code = (y + 8.5).floor().clamp(0.0, 15.0).to(torch.uint8)
    return code[..., :16] | (code[..., 16:] << 4), scale[..., 0].half()


def _dequantize(codes, scales, fmt):
    """The inverse of _quantize, in fp32: [..., D/32, bytes] -> [..., D]."""
    if fmt == "f16":
        return codes.view(torch.float16).float().flatten(-2)
    if fmt == "q8_0":
        v = codes.float() - 128.0
    else:
        v = torch.cat([codes & 15, codes >> 4], -1).float() - 8.0
    return (v * scales.float().unsqueeze(-1)).flatten(-2)


def _parts(pool, case):
    """Views of the pool: K codes, K scales, V codes, V scales, each
    [pages, kv heads, tiles, D/32, 16, bytes]."""
    fmt, dim, heads = case["fmt"], case["dim"], case["kv_heads"]
    codes, scales = _half_bytes(fmt, dim)
    half = codes + scales
    t = pool.view(pool.shape[0], heads, case["page"] // TILE, 2 * half)
    views = []
    for at in (0, half):
        views.append(t[..., at:at + codes].unflatten(-1, (dim // 32, TILE, -1)))
        views.append(t[..., at + codes:at + half].unflatten(-1, (dim // 32, TILE, 2)) if scales else None)
    return views


def _place(slots, page):
    return slots // page, slots % page // TILE, slots % TILE


def _scale_place(row):
    """Where the scale of a tile's token stands among its 16."""
    four = row // 4
    return 4 * torch.where(four % 2 == 0, row % 4, 3 - row % 4) + four


def _store(pool, case, k, v, slots):
    at, tile, row = _place(slots, case["page"])
    kc, ks, vc, vs = _parts(pool, case)
    for x, to, scale_to in ((k, kc, ks), (v, vc, vs)):
        codes, scales = _quantize(x, case["fmt"])
        to[at, :, tile, :, row, :] = codes
        if scales is not None:
            scale_to[at, :, tile, :, _scale_place(row), :] = scales.unsqueeze(-1).view(torch.uint8)


def _load(pool, case, slots):
    at, tile, row = _place(slots, case["page"])
    kc, ks, vc, vs = _parts(pool, case)
    got = []
    for codes, scales in ((kc, ks), (vc, vs)):
        s = None if scales is None else scales[at, :, tile, :, _scale_place(row), :].contiguous().view(torch.float16)[..., 0]
        got.append(_dequantize(codes[at, :, tile, :, row, :].contiguous(), s, case["fmt"]))
    return got


# ------------------------------------------------------------------ inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _keys_values(case, tokens, g, dtype):
    """Keys with a few strong channels, as attention layers have, and values
    with a small mean."""
    heads, dim = case["kv_heads"], case["dim"]
    k = torch.randn((tokens, heads, dim), generator=g, device="cuda")
    channel = torch.rand((heads, dim), generator=g, device="cuda")
    k = torch.where(channel < 0.05, 4.0 * k + 3.0, k)
    v = torch.randn((tokens, heads, dim), generator=g, device="cuda") + 0.1
    return k.to(dtype), v.to(dtype)


def _pool(case, pages):
    """Pages that nothing has written: every byte 0xFF, so their scales and
    fp16 values are NaN.  One page more than the program's own, which the
    plain form uses for what it skips."""
    codes, scales = _half_bytes(case["fmt"], case["dim"])
    size = case["kv_heads"] * (case["page"] // TILE) * 2 * (codes + scales)
    return torch.full((pages + 1, size), 255, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    dtype, page, dim = TYPES[case["dtype"]], case["page"], case["dim"]
    state = dict(case=case, dtype=dtype)
    if case["op"] == "attn":
        lens = _lens(case)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        pool = _pool(case, pages)
        table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device="cuda")
        done = 0
        for b, n in enumerate(need):
            table[b, :n] = order[done:done + n].int()
            done += n
        for b, n in enumerate(lens):
            for lo in range(0, n, 32768):  # a bounded piece at a time
                p = torch.arange(lo, min(n, lo + 32768), device="cuda")
                k, v = _keys_values(case, p.numel(), g, torch.float32)
                _store(pool, case, k, v, table[b].long()[p // page] * page + p % page)
        tokens, heads = case["batch"] * case["rows"], case["heads"]
        wide = heads + 2 * case["kv_heads"] if case["fused"] else heads
        q = (2.0 * torch.randn((tokens, wide, dim), generator=g, device="cuda")).to(dtype)
        state.update(pool=pool, cache=pool[:-1], table=table, q=q[:, :heads],
                     lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), longest=max(lens))
        return state
    tokens, skip = case["tokens"], case["skip"]
    used = -(-(tokens + 5) // page)
    pages = used + 2
    order = torch.randperm(pages, generator=g, device="cuda")
    pool = _pool(case, pages)
    p = torch.arange(tokens, device="cuda") + 5  # the first page is partly another's
    slots = order[p // page] * page + p % page
    slots[:skip] = -1
    state.update(pool=pool, cache=pool[:-1], slots=slots)
    k, v = _keys_values(case, tokens, g, dtype if case["op"] == "write" else torch.float32)
    if case["op"] == "read":
        _store(pool, case, k, v, torch.where(slots < 0, pages * page, slots))
        return state
    if case["fused"]:  # slices of one projection's output, queries first
        qkv = torch.zeros((tokens, 7 * case["kv_heads"], dim), dtype=dtype, device="cuda")
        qkv[:, 5 * case["kv_heads"]:6 * case["kv_heads"]] = k
        qkv[:, 6 * case["kv_heads"]:] = v
        k, v = qkv[:, 5 * case["kv_heads"]:6 * case["kv_heads"]], qkv[:, 6 * case["kv_heads"]:]
    state.update(k=k, v=v)
    return state


# ------------------------------------------------------------------ one pass


def _plain_attention(s):
    case = s["case"]
    batch, rows, heads, kv_heads, dim = (case[n] for n in ("batch", "rows", "heads", "kv_heads", "dim"))
    used = -(-max(1, s["longest"]) // case["page"])
    table = s["table"][:, :used].long()
    where = torch.where(table < 0, s["pool"].shape[0] - 1, table)
    kc, ks, vc, vs = _parts(s["pool"], case)
    position = torch.arange(used * case["page"], device="cuda")
    live = (position < s["lens"][:, None])[:, None, :, None]
    kv = []
    for codes, scales in ((kc, ks), (vc, vs)):
        order = _scale_place(torch.arange(TILE, device="cuda"))
        d = None if scales is None else scales[where].contiguous().view(torch.float16)[..., order, 0]
        d = None if d is None else d.movedim(4, -1)
        x = _dequantize(codes[where].movedim(4, -2).contiguous(), d, case["fmt"])
        x = x.movedim(2, 1).reshape(batch, kv_heads, position.numel(), dim)  # [batch, kv head, position, D]
        kv.append(torch.where(live, x, torch.zeros_like(x)))
    q = s["q"].float().view(batch, rows, kv_heads, heads // kv_heads, dim).permute(0, 2, 3, 1, 4)
    score = q.reshape(batch, kv_heads, -1, dim) @ kv[0].transpose(-1, -2) * (1.0 / math.sqrt(dim))
    end = s["lens"][:, None] - (rows - 1) + torch.arange(rows, device="cuda")
    seen = position < end[..., None]
    if case["window"]:
        seen = seen & (position >= end[..., None] - case["window"])
    score = score.view(batch, kv_heads, -1, rows, position.numel())
    score = torch.where(seen[:, None, None], score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = weight.sum(-1, keepdim=True)
    out = weight.flatten(2, 3) @ kv[1]
    out = out.view(batch, kv_heads, -1, rows, dim) / torch.where(total == 0, torch.ones_like(total), total)
    return out.permute(0, 3, 1, 2, 4).reshape(batch * rows, heads, dim).to(s["dtype"])


def run(state):
    case = state["case"]
    fmt, page = case["fmt"], case["page"]
    if own:
        from block_quantized_gemv_quantize_gb300 import ops

        if case["op"] == "attn":
            return ops.attn_paged(state["q"], state["cache"], state["table"], state["lens"], fmt, page,
                                  case["kv_heads"], rows=case["rows"], window=case["window"])
        if case["op"] == "write":
            ops.kv_write(state["cache"], state["k"], state["v"], state["slots"], fmt, page)
        return ops.kv_read(state["cache"], state["slots"], fmt, page, case["kv_heads"], case["dim"],
                           dtype=state["dtype"])
    if case["op"] == "attn":
        return _plain_attention(state)
    spare = (state["pool"].shape[0] - 1) * page
    slots = torch.where(state["slots"] < 0, spare, state["slots"])
    if case["op"] == "write":
        _store(state["pool"], case, state["k"], state["v"], slots)
    live = (state["slots"] >= 0)[:, None, None]
    k, v = _load(state["pool"], case, slots)
    return (torch.where(live, k, torch.zeros_like(k)).to(state["dtype"]),
            torch.where(live, v, torch.zeros_like(v)).to(state["dtype"]))


def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
    values = case["kv_heads"] * case["dim"]
    if case["op"] != "attn":
        n = case["tokens"] - case["skip"]
        held = 2 * n * values * VALUE_BYTES[case["fmt"]]
        out = 2 * case["tokens"] * values * size + 8 * case["tokens"]
        if case["op"] == "read":
            return {"bytes": held + out, "flops": 2 * n * values}
        # read the rows, write the cache, and back
        return {"bytes": 2 * n * values * size + held + held + out, "flops": 8 * n * values}
    held = pairs = 0
    rows, window = case["rows"], case["window"]
    for n in _lens(case):
        ends = [max(0, n - (rows - 1 - i)) for i in range(rows)]
        seen = [min(e, window) if window else e for e in ends]
        pairs += sum(seen)
        first = min([e - c for e, c in zip(ends, seen) if c], default=0)
        held += max(ends) - first
    q = case["batch"] * rows * case["heads"] * case["dim"]
    tables = 4 * case["batch"] + 4 * -(-held // case["page"])
    return {"bytes": 2 * held * values * VALUE_BYTES[case["fmt"]] + 2 * q * size + tables,
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ the definition, in 64 bits


def _exact_codes(x, fmt):
    """The cache's values of x [n, heads, D], by the format's definition: the
    fp32 steps as fp64 operations rounded to fp32 (a quotient or a sum of two
    fp32 numbers rounds to the same fp32 number by way of fp64)."""
    to32 = lambda t: t.to(torch.float32).to(torch.float64)  # noqa: E731
    x = x.to(torch.float64)
    if fmt == "f16":
        return x.to(torch.float16).to(torch.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    if fmt == "q8_0":
        d = to32(b.abs().max(dim=-1, keepdim=True).values / 127)
    else:
        first = b.abs().argmax(dim=-1, keepdim=True)  # a tie's members differ at most in sign
        m = torch.take_along_dim(b, first, dim=-1)
        tie = (b.abs() == m.abs()) & (b != m)
        if bool(tie.any()):
            rank = torch.arange(32, 0, -1, device=b.device) * (b.abs() == m.abs())
            m = torch.take_along_dim(b, rank.argmax(dim=-1, keepdim=True), dim=-1)
        d = to32(-m / 8)
    held = d.clamp(-65504, 65504).to(torch.float16).to(torch.float64)
    y = to32(b / torch.where(d == 0, torch.ones_like(d), d))
    if fmt == "q8_0":
        code = (torch.sign(y) * torch.floor(y.abs() + 0.5)).clamp(-127, 127)
    else:
        code = torch.floor(to32(y + 8.5)).clamp(0, 15) - 8
    code = torch.where(d == 0, torch.zeros_like(code), code)
    return (code * held).reshape(x.shape)


def _exact_tiles(tiles, case):
    """tiles uint8 [n, tile bytes] of one kv head -> K, V fp64 [n 16, D]."""
    dim, fmt = case["dim"], case["fmt"]
    blocks, n = dim // 32, tiles.shape[0]
    halves = []
    for part in tiles.reshape(n, 2, -1).unbind(1):
        part = part.contiguous()
        if fmt == "f16":
            v = part.view(torch.float16).to(torch.float64).reshape(n, blocks, TILE, 32)
        else:
            width = 32 if fmt == "q8_0" else 16
            codes = part[:, :blocks * TILE * width].reshape(n, blocks, TILE, width).to(torch.int64)
            d = part[:, blocks * TILE * width:].contiguous().view(torch.float16).to(torch.float64)
            whole = codes - 128 if fmt == "q8_0" else torch.cat([codes % 16, codes // 16], dim=3) - 8
            order = [4 * (r % 4 if r // 4 % 2 == 0 else 3 - r % 4) + r // 4 for r in range(TILE)]
            v = whole.to(torch.float64) * d.reshape(n, blocks, TILE, 1)[:, :, order]
        halves.append(v.permute(0, 2, 1, 3).reshape(n * TILE, dim))
    return halves


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        live = (s["slots"] >= 0).to(torch.float64)[:, None, None]
        return tuple(_exact_codes(x, case["fmt"]) * live for x in (s["k"], s["v"]))
    kv_heads, per_page = case["kv_heads"], case["page"] // TILE
    pool = s["pool"].reshape(s["pool"].shape[0], kv_heads, per_page, -1)
    if case["op"] == "read":
        out = [torch.zeros((case["tokens"], kv_heads, case["dim"]), dtype=torch.float64, device="cuda")
               for _ in range(2)]
        live = s["slots"] >= 0
        slots = s["slots"][live]
        for h in range(kv_heads):
            both = _exact_tiles(pool[:, h].reshape(-1, pool.shape[-1]), case)
            for o, x in zip(out, both):
                o[live, h] = x[slots]
        return tuple(out)
    rows, heads, dim = case["rows"], case["heads"], case["dim"]
    group = heads // kv_heads
    q = s["q"].to(torch.float64)
    out = torch.zeros((case["batch"] * rows, heads, dim), dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        pages = s["table"][b, :-(-n // case["page"])].to(torch.int64)
        for h in range(kv_heads if n else 0):
            k, v = _exact_tiles(pool[pages, h].reshape(-1, pool.shape[-1]), case)
            for i in range(rows):
                end = n - rows + 1 + i
                begin = max(0, end - case["window"]) if case["window"] else 0
                if end <= 0:
                    continue
                r, hs = b * rows + i, slice(h * group, (h + 1) * group)
                p = torch.softmax(q[r, hs] @ k[begin:end].T / math.sqrt(dim), dim=-1)
                out[r, hs] = p @ v[begin:end]
    return out
