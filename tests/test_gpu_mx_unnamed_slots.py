"""Products whose order names some slots not at all (entries out of range are skipped): such a
slot is no term of the down product's sum and leaves its row of the others as it was,
whatever the workspace holds."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import _mx_ref as R  # noqa: E402

from .test_gpu_mxfp4 import TYPES, Layer, gen, ops  # noqa: E402, F401


def holes(c, every):
    """The layer's order with every `every`-th entry out of range, and the slots that it still names in a range."""
    n = c.order.numel()
    order = c.order.clone()
    at = torch.arange(0, n, every, device="cuda")
    order[at] = torch.tensor([-1, n, 1 << 30, -(1 << 31)], dtype=torch.int32, device="cuda")[torch.arange(at.numel(), device="cuda") % 4]
    named = torch.zeros(n, dtype=torch.bool, device="cuda")
    named[order[(order >= 0) & (order < n)].long()] = True
    return order, named


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens,top_k,experts,every", [(1, 2, 2, 2), (7, 3, 6, 2), (40, 2, 4, 3), (300, 2, 5, 7)])
def test_down(ops, kind, tokens, top_k, experts, every):  # noqa: F811
    c = Layer(ops, kind, tokens, top_k, experts, 128, 72)
    h = c.rows(tokens * top_k)
    weights = torch.rand((tokens, top_k), generator=gen(1)).cuda()
    order, named = holes(c, every)
    y, bound = R.product(c.w[0], h, c.ids, lambda s: s)
    y[~named], bound[~named] = 0.0, 0.0
    want, bound = R.down(y, bound, weights)
    need = max(16, ops.LIB.moe_down_mxfp4_workspace_bytes(ops._TYPES[c.dtype], tokens, top_k, experts, 128, 72))
    first = None
    for fill in (0, 255, 1, "places", "a call before"):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        if fill == "places":  # each slot's number, and partial results that are NaN
            ws.view(torch.int32)[:] = -1
            ws.view(torch.int32)[tokens * top_k * 72:][:tokens * top_k] = torch.arange(tokens * top_k, dtype=torch.int32, device="cuda")
        elif fill == "a call before":
            ops.moe_down_mxfp4(c.packs[0], h, c.offsets, 72, c.order, weights, ws=ws)
        else:
            ws.fill_(fill)
        got = ops.moe_down_mxfp4(c.packs[0], h, c.offsets, 72, order, weights, ws=ws)
        R.close(got, want, R.rounded(want, bound, c.dtype))
        first = got if first is None else first
        assert torch.equal(got, first)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens", [7, 300])
def test_rows_stay_as_they_were(ops, kind, tokens):  # noqa: F811
    c = Layer(ops, kind, tokens, 2, 5, 128, 72, weights=2)
    x = c.rows(tokens) * 0.5
    order, named = holes(c, 3)
    for call in (lambda o, y: ops.qgemm_mxfp4(c.packs[0], x, c.offsets, 72, order=o, top_k=2, y=y),
                 lambda o, y: ops.moe_gate_up_mxfp4(*c.packs, x, c.offsets, 72, o, 2, h=y)):
        want = call(c.order, None)
        held = torch.full((2 * tokens, 72), 3.0, dtype=c.dtype, device="cuda")
        call(order, held)
        assert torch.equal(held[named], want[named]) and bool((held[~named] == 3.0).all())
