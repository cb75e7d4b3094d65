"""Sizes and slots past 32 (or 64) bits are refused: passed on as they are, they
would come out of the C interface as other, smaller numbers.  No GPU."""
import pytest

torch = pytest.importorskip("torch")

from block_quantized_gemv_quantize_gb300 import ops  # noqa: E402

from .test_kv_devices_host import Tensor, machine  # noqa: E402, F401

BIG = [1 << 32, (1 << 32) + 16, 1 << 31, -(1 << 31) - 1, 1 << 64]


@pytest.mark.parametrize("n", BIG)
def test_size_queries(n):
    for args in ((n, 2, 64), (16, n, 64), (16, 2, n)):
        with pytest.raises(ValueError):
            ops.kv_page_bytes("q8_0", *args)
    for args in ((n, 4, 2, 64), (1, n, 2, 64), (1, 4, n, 64), (1, 4, 2, n)):
        with pytest.raises(ValueError):
            ops.attn_paged_workspace_bytes(torch.float32, *args)
    for args in ((16, n, 64, 0, 0), (n, 2, 64, 0, 0), (16, 2, n, 0, 0), (16, 2, 64, 0, n)):
        with pytest.raises(ValueError):
            ops.kv_tile_offset("q8_0", 4, *args)


@pytest.mark.parametrize("n", [1 << 63, 1 << 64, -(1 << 63) - 1])
def test_slots_and_pages(n):
    with pytest.raises(ValueError):
        ops.kv_tile_offset("q8_0", 4, 16, 2, 64, n, 0)
    with pytest.raises(ValueError):
        ops.kv_tile_offset("q8_0", n, 16, 2, 64, 0, 0)
    assert ops.kv_tile_offset("q8_0", 4, 16, 2, 64, 1 << 40, 0) == -1


@pytest.mark.parametrize("n", BIG)
def test_calls(machine, n):  # noqa: F811
    cache = Tensor((4, ops.kv_page_bytes("q8_0", 16, 2, 64)), torch.uint8)
    rows, slots = Tensor((3, 2, 64), torch.float32), Tensor((3,), torch.int64)
    q, table, lens = Tensor((3, 4, 64), torch.float32), Tensor((3, 2), torch.int32), Tensor((3,), torch.int32)
    ws = Tensor((1 << 24,), torch.uint8)
    for call in (lambda: ops.kv_write(cache, rows, rows, slots, "q8_0", n),
                 lambda: ops.kv_read(cache, slots, "q8_0", n, 2, 64, k=rows, v=rows),
                 lambda: ops.attn_paged(q, cache, table, lens, "q8_0", n, 2, out=q, ws=ws),
                 lambda: ops.attn_paged(q, cache, table, lens, "q8_0", 16, n, out=q, ws=ws),
                 lambda: ops.attn_paged(q, cache, table, lens, "q8_0", 16, 2, rows=n, out=q, ws=ws),
                 lambda: ops.attn_paged(q, cache, table, lens, "q8_0", 16, 2, window=-abs(n) - 1, out=q, ws=ws)):
        with pytest.raises(ValueError):
            call()
    assert machine.calls == []


def test_a_window_longer_than_any_sequence(machine):  # noqa: F811
    cache = Tensor((4, ops.kv_page_bytes("q8_0", 16, 2, 64)), torch.uint8)
    q, table, lens = Tensor((3, 4, 64), torch.float32), Tensor((3, 2), torch.int32), Tensor((3,), torch.int32)
    for n in (1 << 31, 1 << 40, 1 << 70):
        ops.attn_paged(q, cache, table, lens, "q8_0", 16, 2, window=n, out=q, ws=Tensor((1 << 24,), torch.uint8))
    assert [args[-2] for args in machine.args] == [(1 << 31) - 1] * 3


def test_tokens_past_32_bits(machine):  # noqa: F811
    # (rows with a stride of zero have such lengths without the memory)
    n = (1 << 32) + 3
    cache = Tensor((4, ops.kv_page_bytes("q8_0", 16, 2, 64)), torch.uint8)
    rows, slots = Tensor((n, 2, 64), torch.float32), Tensor((n,), torch.int64)
    with pytest.raises(ValueError):
        ops.kv_write(cache, rows, rows, slots, "q8_0", 16)
    with pytest.raises(ValueError):
        ops.kv_read(cache, slots, "q8_0", 16, 2, 64, k=rows, v=rows)
    assert machine.calls == []
