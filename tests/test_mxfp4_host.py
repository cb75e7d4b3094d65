"""The MXFP4 calls' host side, without a GPU: sizes, refusals before anything is
enqueued, and the pins of the plain implementation that the GPU tests use."""
import ctypes
import math

import pytest
import torch

from block_quantized_gemv_quantize_gb300 import build
from tests import _mx_ref as R

INVALID, UNSUPPORTED, MISALIGNED, TOO_SMALL = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    build.build()
    from block_quantized_gemv_quantize_gb300 import _lib

    return _lib.LIB


@pytest.fixture(scope="module")
def ops(lib):
    from block_quantized_gemv_quantize_gb300 import ops as o

    return o


def test_sizes(lib):
    assert lib.mxfp4_bytes(3, 64) == 3 * 2 * 17
    assert lib.mxfp4_bytes(0, 64) == 0 and lib.mxfp4_bytes(3, 48) == 0 and lib.mxfp4_bytes(1 << 40, 32) == 0
    # 16-row tiles, units of 64 values, 16 bytes a tile
    assert lib.mxfp4_pack_bytes(2, 17, 96) == 2 * 2 * (2 * 544 + 16)
    assert lib.mxfp4_pack_bytes(64, 1408, 5120) == 64 * 88 * (80 * 544 + 16)
    for bad in ((0, 16, 32), (1025, 16, 32), (1, 0, 32), (1, 16, 33), (1, 16, 32800), (1, (1 << 24) + 1, 32)):
        assert lib.mxfp4_pack_bytes(*bad) == 0
    assert lib.moe_route_workspace_bytes(1, 64, 6) == 0
    assert lib.moe_route_workspace_bytes(100000, 64, 8) > 0
    assert lib.moe_route_workspace_bytes(1 << 28, 64, 8) == 0
    assert lib.moe_down_mxfp4_workspace_bytes(2, 5, 3, 8, 64, 10) >= 5 * 3 * 10 * 4
    assert lib.moe_down_mxfp4_workspace_bytes(7, 5, 3, 8, 64, 10) == 0


P = 4096  # an address that nothing reads: every call below is refused before a launch


def test_refusals_of_the_format_calls(lib):
    q, d, pack = lib.quantize_mxfp4, lib.dequantize_mxfp4, lib.qpack_mxfp4
    assert q(0, None, 64, P, 1, 64, None) == INVALID
    assert q(0, P, 64, None, 1, 64, None) == INVALID
    assert q(3, P, 64, P, 1, 64, None) == INVALID
    assert q(0, P, 63, P, 1, 64, None) == INVALID
    assert q(0, P, 64, P, 0, 64, None) == INVALID
    assert q(0, P, 64, P, 1, 48, None) == UNSUPPORTED
    assert q(0, P, 64, P + 8, 1, 64, None) == MISALIGNED
    assert q(0, P + 2, 64, P, 1, 64, None) == MISALIGNED
    assert q(1, P + 1, 64, P, 1, 64, None) == MISALIGNED
    assert q(0, P, 64, P, 1 << 31, 64, None) == INVALID
    assert d(0, P, None, 64, 1, 64, None) == INVALID
    assert d(0, P, P, 32, 1, 64, None) == INVALID
    assert d(2, P + 4, P, 64, 1, 64, None) == MISALIGNED
    assert pack(None, P, 1, 16, 32, None) == INVALID
    assert pack(P, P, 0, 16, 32, None) == INVALID
    assert pack(P, P, 1, 16, 40, None) == UNSUPPORTED
    assert pack(P, P + 4, 1, 16, 32, None) == MISALIGNED


def test_refusals_of_the_router(lib):
    def route(type=0, logits=P, ld=64, ids=P, weights=P, offsets=P, order=P, ws=None, n=0, tokens=4, experts=64, top_k=6,
              score=0, scale=1.0):
        return lib.moe_route(type, logits, ld, ids, weights, offsets, order, ws, n, tokens, experts, top_k, score, 1, scale,
                             None)

    for bad in (dict(type=3), dict(logits=None), dict(ld=63), dict(ids=None), dict(weights=None), dict(offsets=None),
                dict(order=None), dict(tokens=-1), dict(experts=0), dict(experts=1025, ld=2000), dict(top_k=0),
                dict(top_k=65), dict(top_k=33), dict(score=2), dict(scale=math.inf), dict(scale=math.nan),
                dict(tokens=1 << 28, top_k=8), dict(tokens=10000)):
        assert route(**bad) == INVALID, bad
    assert route(tokens=10000, ws=P, n=100) == TOO_SMALL
    assert route(ids=P + 2) == MISALIGNED
    assert route(logits=P + 2) == MISALIGNED
    assert route(tokens=10000, ws=P + 8, n=1 << 30) == MISALIGNED
    group = lib.moe_group
    assert group(None, P, P, None, 0, 4, 8, 2, None) == INVALID
    assert group(P, P, P, None, 0, 4, 8, 0, None) == INVALID
    assert group(P, P, P, None, 0, 4, 8, 33, None) == INVALID
    assert group(P, P, P + 1, None, 0, 4, 8, 2, None) == MISALIGNED


def test_refusals_of_the_products(lib):
    def gemm(type=2, w=P, x=P, ldx=64, offsets=P, order=P, y=P, ldy=16, ws=P, n=1 << 30, tokens=4, top_k=2, experts=3, K=64,
             N=16):
        return lib.qgemm_mxfp4(type, w, x, ldx, offsets, order, y, ldy, ws, n, tokens, top_k, experts, K, N, None)

    for bad in (dict(type=-1), dict(w=None), dict(x=None), dict(offsets=None), dict(y=None), dict(ldx=63), dict(ldy=15),
                dict(order=None), dict(tokens=-1), dict(top_k=0), dict(top_k=33), dict(experts=0), dict(N=0), dict(K=0),
                dict(K=1 << 16, ldx=1 << 17), dict(tokens=1 << 30)):
        assert gemm(**bad) == INVALID, bad
    assert gemm(K=48) == UNSUPPORTED
    assert gemm(w=P + 8) == MISALIGNED
    assert gemm(x=P + 1) == MISALIGNED
    assert gemm(offsets=P + 2) == MISALIGNED
    assert lib.moe_gate_up_mxfp4(2, P, None, P, 64, P, P, P, 16, P, 1 << 30, 4, 2, 3, 64, 16, None) == INVALID
    assert lib.moe_down_mxfp4(2, P, P, 64, P, P, None, P, 16, P, 1 << 30, 4, 2, 3, 64, 16, None) == INVALID
    assert lib.moe_down_mxfp4(2, P, P, 64, P, P, P, P, 16, P, 8, 4, 2, 3, 64, 16, None) == TOO_SMALL
    assert lib.moe_down_mxfp4(2, P, P, 64, P, P, P, P, 16, None, 0, 4, 2, 3, 64, 16, None) == INVALID
    assert gemm(tokens=0, x=None, y=None) == 0


def test_the_binding_refuses_what_it_cannot_pass_on(ops):
    cpu = torch.zeros((4, 64))
    blocks = torch.zeros((4, 2, 17), dtype=torch.uint8)
    whole = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: ops.quantize_mxfp4(cpu), lambda: ops.dequantize_mxfp4(blocks),
                 lambda: ops.qpack_mxfp4(blocks, 1, 4, 64), lambda: ops.moe_route(cpu, 2),
                 lambda: ops.moe_route(cpu, 2, score="tanh"), lambda: ops.moe_group(whole.view(2, 2), 3),
                 lambda: ops.qgemm_mxfp4(blocks, cpu, whole, 4),
                 lambda: ops.moe_down_mxfp4(blocks, cpu, whole, 4, whole, torch.zeros((3, 1))),
                 lambda: ops.mxfp4_pack_bytes(1 << 32, 16, 64), lambda: ops.mxfp4_bytes(4, 1 << 40)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the plain implementation


def test_plain_quantizer_by_hand():
    x = torch.zeros((1, 32))
    x[0, :8] = torch.tensor([4.0, -6.0, 0.25, 0.75, 5.0, -2.5, 7.0, 0.3])
    b = R.quantize(x)[0, 0]
    assert b[0] == 127  # the largest, 7, is below 8 = 2 * 4: scale 1
    low = [int(v) & 15 for v in b[1:9]]
    # 4; -6; 0.25 -> 0; 0.75 -> 1; 5 -> 4; -2.5 -> -2; 7 -> 6; 0.3 -> 0.5
    assert low == [6, 8 | 7, 0, 2, 6, 8 | 4, 7, 1]
    v = R.values(b[None])
    assert v[:8].tolist() == [4.0, -6.0, 0.0, 1.0, 4.0, -2.0, 6.0, 0.5]
    assert bool((v[8:] == 0).all())


def test_plain_quantizer_is_nearest():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((6, 64), generator=g).double()
    v = R.values(R.quantize(x.float())).view(6, 2, 32)
    x = x.float().double().view(6, 2, 32)
    unit = torch.exp2(torch.floor(torch.log2(x.abs().amax(-1, keepdim=True))) - 2)
    y = (x / unit).abs()
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    off = ((x - v) / unit).abs()
    assert bool(((off <= step / 2) | (y > 6)).all())


def test_plain_group_and_route_by_hand():
    offsets, order = R.group(torch.tensor([[1, 0], [-1, 1], [2, 1]]), 3)
    assert offsets.tolist() == [0, 1, 4, 5] and order.tolist() == [1, 0, 3, 5, 4, 2]
    ids, w = R.route(torch.tensor([[0.0, math.log(3.0), -math.inf]]), 3, "softmax", False, 2.0)
    assert ids.tolist() == [[1, 0, -1]]
    assert torch.allclose(w, torch.tensor([[1.5, 0.5, 0.0]], dtype=torch.float64))
    ids, w = R.route(torch.tensor([[0.0, 0.0]]), 1, "sigmoid", False, 1.0)
    assert ids.tolist() == [[0]] and float(w) == 0.5


def test_signatures_match_the_header(lib):
    for name in ("quantize_mxfp4", "moe_route", "qgemm_mxfp4", "moe_gate_up_mxfp4", "moe_down_mxfp4"):
        assert getattr(lib, name).restype is ctypes.c_int
