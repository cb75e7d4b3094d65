"""The attention's bounded waits, made to run out without any GPU fault.

A test-only switch has the attention's copying warp leave out the copy of the first
tile, so that the warps that wait for it give up after about a second, and the
copying warp, where its ring is not emptied any more, after a few.  The launch
completes, the rows of that kv head are NaN and no others, the timeouts are counted,
and until the count has been taken every call is refused.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from .test_gpu_kvcache import ops  # noqa: E402, F401

QGEMV_WAIT_TIMEOUT = -6


# With 120000 tokens a split has more tiles than its ring: the copying warp waits
# for room.  With 3000 it has issued all its copies when the others give up.
@pytest.mark.parametrize("length", [3000, 120000])
@pytest.mark.parametrize("fmt,rows,heads", [("q8_0", 1, 4), ("q4_0", 6, 12), ("f16", 2, 8)])
def test_a_copy_that_never_comes(ops, fmt, rows, heads, length):  # noqa: F811
    pages = -(-length // 32)
    cache = torch.zeros((pages, ops.kv_page_bytes(fmt, 32, 2, 128)), dtype=torch.uint8, device="cuda:0")
    g = torch.Generator(device="cuda:0").manual_seed(1)
    k, v, q = (torch.randn((n, h, 128), generator=g, device="cuda:0")
               for n, h in ((length, 2), (length, 2), (rows, heads)))
    ops.kv_write(cache, k, v, torch.arange(length, device="cuda:0"), fmt, 32)
    args = dict(q=q, cache=cache, page_table=torch.arange(pages, dtype=torch.int32, device="cuda:0")[None], fmt=fmt,
                kv_lens=torch.tensor([length], dtype=torch.int32, device="cuda:0"), page_tokens=32, n_kv_heads=2,
                rows=rows)
    want = ops.attn_paged(**args)
    torch.cuda.synchronize()
    assert ops.qgemv_take_wait_timeouts() == 0
    assert ops.qgemv_debug_drop_next_copy() == 0
    got = ops.attn_paged(**args)
    torch.cuda.synchronize()
    first = heads // 2  # the heads of kv head 0
    assert bool(torch.isnan(got[:, :first]).all()) and torch.equal(got[:, first:], want[:, first:])
    out = torch.full_like(want, 7.0)
    with pytest.raises(ops.QgemvError) as e:
        ops.attn_paged(**args, out=out)
    assert e.value.status == QGEMV_WAIT_TIMEOUT
    slots = torch.zeros(1, dtype=torch.int64, device=out.device)
    with pytest.raises(ops.QgemvError):
        ops.kv_read(args["cache"], slots, fmt, 32, 2, 128)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
    assert ops.qgemv_take_wait_timeouts() >= 1 and ops.qgemv_take_wait_timeouts() == 0
    assert torch.equal(ops.attn_paged(**args), want)
