"""The calls' device, without a GPU: tensors of one device while another is
current.  Stand-ins for the tensors take the ctypes way to a stand-in for the
library, which records the device that was current when it was called."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

from block_quantized_gemv_quantize_gb300 import _lib, ops  # noqa: E402


class Tensor:
    is_cuda = True

    def __init__(self, shape, dtype, device="cuda:1"):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)

    def stride(self, i=None):
        steps, n = [], 1
        for size in reversed(self.shape):
            steps.insert(0, n)
            n *= size
        return tuple(steps) if i is None else steps[i]

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def machine(monkeypatch):
    """Two devices, the first of them current; `calls` gets (name, device, stream) of each call of the library,
    `args` its arguments."""
    state = types.SimpleNamespace(now=0, calls=[], args=[])

    @contextlib.contextmanager
    def device(d):
        before, state.now = state.now, torch.device(d).index
        yield
        state.now = before

    def entry(name):
        def call(*args):
            state.calls.append((name, state.now, args[-1]))
            state.args.append(args)
            return 0
        return call

    names = ("kv_write", "kv_read", "attn_paged")
    fake = types.SimpleNamespace(**{n: entry(n) for n in names}, kv_page_bytes=_lib.LIB.kv_page_bytes,
                                 attn_paged_workspace_bytes=_lib.LIB.attn_paged_workspace_bytes)
    monkeypatch.setattr(_lib, "LIB", fake)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(_lib, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(_lib, "_device_now", lambda: state.now, raising=False)
    return state


def test_the_cache_calls_run_on_their_tensors_device(machine):
    size = ops.kv_page_bytes("q8_0", 16, 2, 64)
    cache = Tensor((4, size), torch.uint8)
    rows, slots = Tensor((3, 2, 64), torch.float32), Tensor((3,), torch.int64)
    ops.kv_write(cache, rows, rows, slots, "q8_0", 16)
    ops.kv_read(cache, slots, "q8_0", 16, 2, 64, k=rows, v=rows)
    q = Tensor((3, 4, 64), torch.float32)
    ops.attn_paged(q, cache, Tensor((3, 2), torch.int32), Tensor((3,), torch.int32), "q8_0", 16, 2, out=q,
                   ws=Tensor((1 << 24,), torch.uint8))
    assert machine.calls == [(n, 1, 101) for n in ("kv_write", "kv_read", "attn_paged")]
    assert machine.now == 0


def test_the_other_calls_refuse_tensors_of_another_device(machine):
    assert _lib._stream(Tensor((3,), torch.float32, "cuda:0")) == 100
    with pytest.raises(ValueError, match="cuda:1"):
        _lib._stream(Tensor((3,), torch.float32))
