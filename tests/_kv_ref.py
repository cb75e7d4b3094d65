"""The paged key-value cache and the attention over it, plainly, in numpy and
64 bits: the format's definition, the documented layout, and softmax
attention.  Test code only."""
from __future__ import annotations

import numpy as np

TILE = 16
CODE_BYTES = {"f16": 64, "q8_0": 32, "q4_0": 16}
HALF_STEP = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
LEAST = {"float32": 1e-30, "float16": 2.0 ** -25, "bfloat16": 1e-30}  # half a step of the subnormal numbers


def quantize(x: np.ndarray, fmt: str):
    """fp32 values [..., D] -> (block bytes [..., D/32, n], fp16 scales [..., D/32] or None)."""
    x = np.asarray(x, dtype=np.float32).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    with np.errstate(all="ignore"):
        if fmt == "f16":
            return x.astype(np.float16).view(np.uint8), None
        mag = np.abs(x)
        fine = np.isfinite(x).all(-1)
        top = mag.max(-1)
        if fmt == "q8_0":
            d = (top / np.float32(127)).astype(np.float32)
        else:
            d = (np.take_along_axis(x, mag.argmax(-1)[..., None], -1)[..., 0] / np.float32(-8)).astype(np.float32)
        y = np.where((fine & (d != 0))[..., None], x / np.where(d != 0, d, 1)[..., None], 0).astype(np.float32)
        scale = np.where(fine, np.clip(d, -65504, 65504), np.nan).astype(np.float16)
        if fmt == "q8_0":
            y64 = y.astype(np.float64)
            code = np.clip(np.sign(y64) * np.floor(np.abs(y64) + 0.5), -127, 127) + 128
            return code.astype(np.uint8), scale
        code = np.clip(np.floor(y + np.float32(8.5)), 0, 15).astype(np.uint8)
        return code[..., :16] | (code[..., 16:] << 4), scale


def dequantize(code: np.ndarray, scale, fmt: str) -> np.ndarray:
    """The values in fp64 [..., D]."""
    if fmt == "f16":
        v = np.ascontiguousarray(code).view(np.float16).astype(np.float64)
    elif fmt == "q8_0":
        v = (code.astype(np.float64) - 128) * scale.astype(np.float64)[..., None]
    else:
        v = (np.concatenate([code & 15, code >> 4], -1).astype(np.float64) - 8) * scale.astype(np.float64)[..., None]
    return v.reshape(*v.shape[:-2], v.shape[-2] * 32)


def scale_place(r: int) -> int:
    s = r % 4 if (r // 4) % 2 == 0 else 3 - r % 4
    return 4 * s + r // 4


def half_bytes(fmt: str, dim: int) -> int:
    return dim // 32 * TILE * (CODE_BYTES[fmt] + (0 if fmt == "f16" else 2))


def page_bytes(fmt: str, page: int, heads: int, dim: int) -> int:
    return heads * (page // TILE) * 2 * half_bytes(fmt, dim)


def store(cache: np.ndarray, k: np.ndarray, v: np.ndarray, slots, fmt: str, page: int) -> None:
    """k, v [tokens, heads, D] into the bytes of cache [pages, page bytes], one token and head at a time."""
    n, heads, dim = k.shape
    half = half_bytes(fmt, dim)
    cb = CODE_BYTES[fmt]
    parts = [quantize(x, fmt) for x in (k, v)]
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= cache.shape[0] * page:
            continue
        r = slot % TILE
        for h in range(heads):
            at = (h * (page // TILE) + slot % page // TILE) * 2 * half
            for code, scale in parts:
                for b in range(dim // 32):
                    o = at + (b * TILE + r) * cb
                    cache[slot // page, o:o + cb] = code[t, h, b]
                    if scale is not None:
                        o = at + dim // 32 * TILE * cb + (b * TILE + scale_place(r)) * 2
                        cache[slot // page, o:o + 2] = scale[t, h, b:b + 1].view(np.uint8)
                at += half


def attention(q, k, v, length: int, rows: int, window: int, scale: float):
    """One sequence: q [rows, heads, D], k and v [length, kv heads, D], all
    fp64 -> (out, lse [rows, heads], sum p |v|, the largest scale sum |q k|)."""
    heads, kv_heads = q.shape[1], k.shape[1]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    reach = 0.0
    for i in range(rows):
        end = length - (rows - 1 - i)
        begin = max(0, end - window) if window else 0
        if end <= 0:
            continue
        for h in range(heads):
            kk, vv = k[begin:end, h * kv_heads // heads], v[begin:end, h * kv_heads // heads]
            s = kk @ q[i, h] * scale
            reach = max(reach, float((np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)))
            p = np.exp(s - s.max())
            total = p.sum()
            lse[i, h] = s.max() + np.log(total)
            out[i, h] = p @ vv / total
            mag[i, h] = p @ np.abs(vv) / total
    return out, lse, mag, reach


def bounds(out, mag, reach: float, dim: int, length: int, kind: str):
    """(largest error of out, of lse) by the operator's arithmetic: scores of
    operands with 22 bits, products summed in fp32 over dim/16 steps and the
    blocks (each step may cut 2^-22 of what it has); exp2 and the split weights
    2^-19 together; sums over the length in fp32, 16 positions a step; weights of
    one 11-bit term where the type is bf16; one rounding of the output."""
    score = (dim / 16 + 8) * 2.0 ** -22 * reach
    rel = 2 * score + 2.0 ** -19 + length * 2.0 ** -26 + (2.0 ** -11 if kind == "bfloat16" else 0)
    return mag * rel + np.abs(out) * HALF_STEP[kind] + np.abs(out) * rel + LEAST[kind], rel + 2.0 ** -19 * (1 + reach)
