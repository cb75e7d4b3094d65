"""What the sparse layer's calls refuse, by the compiled short way and by ctypes: the same exception."""
import types

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from .test_gpu_mxfp4 import ops  # noqa: E402, F401


@pytest.fixture(params=["compiled", "ctypes"])
def way(request, ops, monkeypatch):  # noqa: F811
    if request.param == "ctypes":
        monkeypatch.setattr(ops, "_CALLS", types.SimpleNamespace(
            **{n: lambda *args: None for n in ("quantize_mxfp4", "dequantize_mxfp4", "moe_route", "product")}))
    return ops


def test_an_unknown_score(way):
    logits = torch.zeros((4, 8), device="cuda")
    for score in ("tanh", "", None, 1):
        with pytest.raises(ValueError, match="softmax, sigmoid"):
            way.moe_route(logits, 2, score=score)


def test_sizes_and_scale_of_the_router(way):
    for experts, top_k, scale in ((2000, 2, 1.0), (64, 33, 1.0), (8, 2, float("inf")), (8, 2, float("nan")), (8, 2, 1e39)):
        with pytest.raises((way.QgemvError, OverflowError)):
            way.moe_route(torch.zeros((4, experts), device="cuda"), top_k, scale=scale)
    for top_k in (0, 9, -1):
        with pytest.raises(ValueError):
            way.moe_route(torch.zeros((4, 8), device="cuda"), top_k)


def test_the_other_calls(way):
    pack = way.qpack_mxfp4(torch.zeros((16, 2, 17), dtype=torch.uint8, device="cuda"), 1, 16, 64)
    x, offsets = torch.zeros((4, 64), device="cuda"), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for bad in (dict(N=17), dict(x=torch.zeros((4, 96), device="cuda")), dict(x=x.int()), dict(top_k=2), dict(offsets=offsets.long()), dict(offsets=offsets[:1])):
        with pytest.raises(ValueError):
            way.qgemm_mxfp4(**{**dict(w_pack=pack, x=x, offsets=offsets, N=16), **bad})
    for bad in (x[:, :40], x.int(), x.cpu(), x[0]):
        with pytest.raises(ValueError):
            way.quantize_mxfp4(bad)
    with pytest.raises(ValueError):
        way.dequantize_mxfp4(torch.zeros((4, 2, 16), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        way.dequantize_mxfp4(torch.zeros((4, 2, 17), dtype=torch.uint8, device="cuda"), dtype=torch.int32)
