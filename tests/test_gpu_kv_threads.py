"""The compiled call of the attention does not hold the interpreter while it
launches: a launch may wait for room in the stream's queue, and what it waits for
may be a callback in Python."""
import ctypes
import threading
import time

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from .test_gpu_kvcache import attention_case, ops  # noqa: E402, F401


def test_other_threads_run_while_a_call_waits(ops):  # noqa: F811
    if not hasattr(ops._CALLS, "init"):
        pytest.skip("no compiled calls")
    args, _, _ = attention_case(ops, "q8_0", "float32", [40], 1, 4, 2, 64, 16, 0)
    want = ops.attn_paged(**args)
    entries = {n: ctypes.cast(getattr(ops.LIB, n), ctypes.c_void_p).value
               for n in ("kv_write", "kv_read", "attn_paged", "kv_page_bytes", "attn_paged_workspace_bytes")}
    # in place of the library's call one that waits: sleep(fmt), a second, and returns 0
    sleep = ctypes.cast(ctypes.CDLL(None).sleep, ctypes.c_void_p).value
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.wait(0.01):
            ticks.append(time.monotonic())

    thread = threading.Thread(target=tick)
    try:
        ops._CALLS.init(*{**entries, "attn_paged": sleep}.values())
        thread.start()
        begin = time.monotonic()
        ops.attn_paged(**args)
        end = time.monotonic()
    finally:
        ops._CALLS.init(*entries.values())
        stop.set()
        thread.join()
    assert end - begin > 0.9
    assert sum(begin + 0.1 < t < end - 0.1 for t in ticks) >= 10
    assert torch.equal(ops.attn_paged(**args), want)
