"""The many-row products' bounded waits, made to run out without any GPU fault.

A test-only switch has one CTA not announce its first rows of x, so that the
warps that wait for them give up after about a second, and with them the other
roles of both CTAs of the pair.  The launch completes, the timeouts are counted, and
until the count has been taken every call is refused; afterwards the same call
gives the same result as before.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from .test_gpu_mxfp4 import Layer, ops  # noqa: E402, F401

QGEMV_WAIT_TIMEOUT = -6


# (short and long K: the roles are all done, or all waiting, when the wait runs out)
@pytest.mark.parametrize("kind,K", [("bfloat16", 64), ("bfloat16", 4096), ("float32", 2048), ("float16", 1056)])
def test_rows_that_are_never_announced(ops, kind, K):  # noqa: F811
    c = Layer(ops, kind, 300, 2, 3, K, 272)
    x = c.rows(300)
    call = lambda: ops.qgemm_mxfp4(c.packs[0], x, c.offsets, 272, order=c.order, top_k=2)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    assert ops.qgemv_take_wait_timeouts() == 0
    assert ops.qgemv_debug_drop_next_copy() == 0
    call()
    torch.cuda.synchronize()
    for refused in (call, lambda: ops.quantize_mxfp4(x[:, :K // 32 * 32]), lambda: ops.moe_route(x[:, :64].contiguous(), 2),
                    lambda: ops.moe_group(c.ids.contiguous(), 3)):
        with pytest.raises(ops.QgemvError) as e:
            refused()
        assert e.value.status == QGEMV_WAIT_TIMEOUT
    assert ops.qgemv_take_wait_timeouts() >= 1 and ops.qgemv_take_wait_timeouts() == 0
    assert torch.equal(call(), want)
