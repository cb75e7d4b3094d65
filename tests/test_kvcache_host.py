"""The paged cache without a GPU: sizes, tile addresses (slots and heads
outside the cache among them), and the calls' refusals, which come before any
CUDA call."""
import ctypes

import pytest

from block_quantized_gemv_quantize_gb300 import build

from . import _kv_ref as R

P, I, L, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
FMT = {"f16": 0, "q8_0": 1, "q4_0": 2}
A = 0x10000  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(build.build())
    lib.kv_page_bytes.restype = S
    lib.kv_page_bytes.argtypes = [I, I, I, I]
    lib.kv_tile_offset.restype = L
    lib.kv_tile_offset.argtypes = [I, L, I, I, I, L, I]
    lib.kv_write.argtypes = [I, I, P, L, L, P, L, L, P, P, L, I, I, I, I, P]
    lib.kv_read.argtypes = [I, I, P, L, I, P, P, L, L, P, L, L, I, I, I, P]
    lib.attn_paged_workspace_bytes.restype = S
    lib.attn_paged_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.attn_paged.argtypes = [I, I, P, L, L, P, L, I, P, L, I, P, P, L, L, P, P, S, I, I, I, I, I, ctypes.c_float, I, P]
    return lib


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("page,heads,dim", [(16, 1, 32), (48, 3, 96), (1024, 8, 512)])
def test_page_bytes(lib, fmt, page, heads, dim):
    assert lib.kv_page_bytes(FMT[fmt], page, heads, dim) == R.page_bytes(fmt, page, heads, dim)


def test_page_bytes_of_refused_sizes(lib):
    for fmt, page, heads, dim in ((3, 16, 1, 32), (-1, 16, 1, 32), (1, 0, 1, 32), (1, 24, 1, 32), (1, 1040, 1, 32),
                                  (1, 16, 0, 32), (1, 16, 1025, 32), (1, 16, 1, 0), (1, 16, 1, 48), (1, 16, 1, 544)):
        assert lib.kv_page_bytes(fmt, page, heads, dim) == 0


@pytest.mark.parametrize("fmt", FMT)
def test_tile_offsets_stay_inside_the_cache(lib, fmt):
    pages, page, heads, dim = 5, 48, 3, 96
    size = R.page_bytes(fmt, page, heads, dim)
    tile = 2 * R.half_bytes(fmt, dim)
    seen = set()
    for slot in range(pages * page):
        for h in range(heads):
            off = lib.kv_tile_offset(FMT[fmt], pages, page, heads, dim, slot, h)
            assert off == slot // page * size + (h * (page // 16) + slot % page // 16) * tile
            assert 0 <= off and off + tile <= pages * size
            seen.add(off)
    assert len(seen) == pages * heads * page // 16
    for slot, h in ((-1, 0), (pages * page, 0), (0, -1), (0, heads), (-(1 << 62), 0), ((1 << 62), 0)):
        assert lib.kv_tile_offset(FMT[fmt], pages, page, heads, dim, slot, h) == -1


def test_tile_offset_past_32_bits(lib):
    pages = 1 << 22
    size = R.page_bytes("q8_0", 128, 8, 128)
    slot = pages * 128 - 1
    want = (pages - 1) * size + (7 * 8 + 7) * 2 * R.half_bytes("q8_0", 128)
    assert lib.kv_tile_offset(1, pages, 128, 8, 128, slot, 7) == want > 1 << 39


def write_args(**over):
    a = dict(fmt=1, type=0, k=A, kt=1024, kh=128, v=A, vt=1024, vh=128, slots=A, cache=A, pages=4, page=16, n=3, heads=8,
             dim=128, stream=None)
    a.update(over)
    return list(a.values())


REFUSED = [(dict(k=None), -1), (dict(v=None), -1), (dict(slots=None), -1), (dict(cache=None), -1), (dict(fmt=3), -1),
           (dict(type=3), -1), (dict(n=-1), -1), (dict(pages=0), -1), (dict(pages=1 << 60), -1), (dict(heads=0), -1),
           (dict(dim=0), -1), (dict(page=0), -1), (dict(kt=-1), -1), (dict(vh=-128), -1), (dict(page=24), -2),
           (dict(dim=80), -2), (dict(cache=A + 8), -3), (dict(slots=A + 4), -3), (dict(k=A + 2), -3),
           (dict(type=1, v=A + 1), -3)]


@pytest.mark.parametrize("over,status", REFUSED)
def test_write_and_read_refusals(lib, over, status):
    w = write_args(**over)
    assert lib.kv_write(*w) == status
    fmt, typ, k, kt, kh, v, vt, vh, slots, cache, pages, page, n, heads, dim, stream = w
    assert lib.kv_read(fmt, typ, cache, pages, page, slots, k, kt, kh, v, vt, vh, n, heads, dim, stream) == status


def test_no_tokens_is_no_work(lib):
    assert lib.kv_write(*write_args(n=0)) == 0


def attn_args(**over):
    a = dict(fmt=1, type=0, q=A, qr=5120, qh=128, cache=A, pages=4, page=16, table=A, ld=4, max_pages=4, lens=A, out=A,
             orow=5120, oh=128, lse=None, ws=A, ws_bytes=1 << 30, batch=1, rows=1, heads=40, kv_heads=8, dim=128,
             scale=0.1, window=0, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,status", [
    (dict(q=None), -1), (dict(cache=None), -1), (dict(table=None), -1), (dict(lens=None), -1), (dict(out=None), -1),
    (dict(ws=None), -1), (dict(fmt=9), -1), (dict(type=-1), -1), (dict(batch=0), -1), (dict(batch=65537), -1),
    (dict(rows=0), -1), (dict(max_pages=0), -1), (dict(ld=3), -1), (dict(scale=float("inf")), -1),
    (dict(scale=float("nan")), -1), (dict(window=-1), -1), (dict(pages=0), -1), (dict(qr=-1), -1),
    (dict(max_pages=1 << 27, ld=1 << 27), -1), (dict(rows=18), -2), (dict(heads=41), -2), (dict(dim=32), -2),
    (dict(dim=160), -2), (dict(page=8), -2), (dict(ws_bytes=1023), -4), (dict(cache=A + 8), -3), (dict(ws=A + 4), -3),
    (dict(q=A + 1), -3), (dict(out=A + 2), -3), (dict(table=A + 2), -3), (dict(lens=A + 1), -3), (dict(lse=A + 2), -3)])
def test_attention_refusals(lib, over, status):
    assert lib.attn_paged(*attn_args(**over)) == status


def test_workspace_sizes(lib):
    w = lib.attn_paged_workspace_bytes
    assert w(0, 1, 40, 8, 128) >= 1024
    for bad in ((3, 1, 40, 8, 128), (0, 0, 40, 8, 128), (0, 18, 40, 8, 128), (0, 1, 41, 8, 128), (0, 1, 40, 0, 128)):
        assert w(*bad) == 0


def test_binding_refuses_what_it_cannot_pass_on():
    import torch

    from block_quantized_gemv_quantize_gb300 import ops

    with pytest.raises(ValueError):
        ops.kv_page_bytes("q5_0", 16, 1, 64)
    cache = torch.zeros(ops.kv_page_bytes("q8_0", 16, 2, 64), dtype=torch.uint8)
    k = torch.zeros((3, 2, 64))
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        ops.kv_write(cache, k, k, slots, "q8_0", 16)  # no CUDA tensors
    with pytest.raises(ValueError):
        ops.kv_write(cache, k.double(), k.double(), slots, "q8_0", 16)
    with pytest.raises(ValueError):
        ops.attn_paged(k[:, 0], cache, slots, slots, "q8_0", 16, 2)
