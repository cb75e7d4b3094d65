"""Weights whose blocks' scales are far apart, as another writer of the format may have
them: a block of zeros has no part in a row whatever its scale byte says."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import _mx_ref as R  # noqa: E402

from .test_gpu_mxfp4 import TYPES, Layer, gen, ops  # noqa: E402, F401


def set_blocks(c, i, blocks):
    """Weight i of the layer from these blocks."""
    c.blocks[i] = blocks
    c.w[i] = R.values(blocks)
    c.packs[i] = c.ops.qpack_mxfp4(blocks, c.experts, c.N, 32 * blocks.shape[-2])


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens,top_k,experts,K,N", [(5, 2, 3, 160, 40), (5, 1, 1, 1056, 33), (200, 2, 4, 160, 40), (90, 1, 1, 1056, 130)])
@pytest.mark.parametrize("byte", [254, 190, 149, 128])
def test_blocks_of_zeros_with_a_large_scale(ops, kind, tokens, top_k, experts, K, N, byte):  # noqa: F811
    c = Layer(ops, kind, tokens, top_k, experts, K, N, weights=2)
    g = gen(byte)
    for i in range(2):
        blocks = c.blocks[i].clone()
        zero = (torch.rand(blocks.shape[:-1], generator=g) < 0.3).cuda()
        zero[..., 0] |= ~zero.any(-1)
        blocks[..., 0] = torch.where(zero, byte, blocks[..., 0])
        blocks[..., 1:] = torch.where(zero[..., None], blocks[..., 1:] & 0x88, blocks[..., 1:])  # (zeros of both signs)
        set_blocks(c, i, blocks)
    x = c.rows(tokens)
    c.gemm(x)
    c.gate_up(x * 0.5)
    c.down(c.rows(tokens * top_k), torch.rand((tokens, top_k), generator=g).cuda())


def test_a_weight_of_zeros(ops):  # noqa: F811
    for tokens in (3, 90):
        c = Layer(ops, "float32", tokens, 1, 2, 96, 40)
        blocks = c.blocks[0].clone()
        blocks[..., 0] = 254
        blocks[..., 1:] &= 0x88
        set_blocks(c, 0, blocks)
        assert bool((c.gemm(c.rows(tokens)) == 0).all())


def product(w, x, ids, rows_of):
    """R.product, its bound without what zeros of x (exact ones) would add: a row's elements enter to
    2^-38 of its largest, but a zero enters as zero."""
    y, bound = R.product(w, x, ids, rows_of)
    x64 = x.double()
    for e in range(w.shape[0]):
        s = torch.nonzero(ids.flatten() == e)[:, 0]
        if s.numel():
            xe = x64[rows_of(s)]
            top = xe.abs().amax(-1, keepdim=True)
            bound[s] -= top * w[e].abs().sum(-1) * 2.0 ** -38
            mag = xe.abs() @ w[e].abs().T
            roundings = 2.0 ** -23 + 32 * 2.0 ** -23 + (x.shape[1] / 32 + 16) * 2.0 ** -24
            bound[s] = mag * roundings + top * ((xe != 0).double() @ w[e].abs().T) * 2.0 ** -38
    return y, bound


DISTANCES = [0, 1, 26, 27, 28, 29, 30, 31, 32, 33, 60, 63, 64, 65, 95, 96, 99, 100, 125, 126, 127, 128, 129, 191, 192, 249, 253, 254]


def far_blocks(kind, K, N, distances, g):
    """An expert a distance l: its rows' first block (and others) at scale T, their second at T - l, which
    is 2^0 where a byte has it.  (blocks, the power of two that brings the second's products to about 1)"""
    blocks = R.random_blocks(g, len(distances), N, K)
    powers = []
    for j, l in enumerate(distances):
        top = min(254, 127 + l)
        blocks[j, :, :, 0] = top - torch.randint(0, min(20, l + 1), (N, K // 32), generator=g).to(torch.uint8)
        blocks[j, :, 0, 0] = top
        blocks[j, :, 0, 1] |= 0x11
        blocks[j, :, 1, 0] = top - l
        blocks[j, :, 1, 1] |= 0x11
        powers.append(127.0 - (top - l))
    return blocks.cuda(), torch.tensor(powers, dtype=torch.float64)


def second_block_only(c, rows, ids, powers, g):
    """Rows of x that are zero but in the second block, of such size that products are about 1."""
    x = torch.zeros((rows, 32 * c.blocks[0].shape[-2]), dtype=torch.float64)
    x[:, 32:64] = torch.randn((rows, 32), generator=g, dtype=torch.float64) * 2.0 ** powers[ids.cpu().long(), None]
    return x.to(c.dtype).cuda()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("each,K,N", [(1, 96, 40), (3, 160, 20), (20, 160, 20), (40, 1056, 33), (170, 128, 260)])
def test_a_block_at_every_distance(ops, kind, each, K, N):  # noqa: F811
    """The one block that x meets is 2^-l of the row's largest scale."""
    distances = [l for l in DISTANCES if kind != "float16" or l <= 128]
    E, g = len(distances), gen(each)
    ids = (torch.arange(E * each, dtype=torch.int32) % E)[:, None]
    c = Layer(ops, kind, E * each, 1, E, K, N, ids=ids, weights=2)
    made = [far_blocks(kind, K, N, distances, g) for _ in range(2)]
    for i in range(2):
        set_blocks(c, i, made[i][0])
    x = second_block_only(c, E * each, c.ids.flatten(), made[0][1], g)
    y, bound = product(c.w[0], x, c.ids, lambda s: s)
    assert 0.05 < float(y.abs().median()) < 500
    R.close(ops.qgemm_mxfp4(c.packs[0], x, c.offsets, N, order=c.order), y, R.rounded(y, bound, c.dtype))
    weights = torch.rand((E * each, 1), generator=g).cuda()
    want, bound = R.down(y, bound, weights)
    R.close(ops.moe_down_mxfp4(c.packs[0], x, c.offsets, N, c.order, weights), want, R.rounded(want, bound, c.dtype))
    x = x * 0.125
    gate, gb = product(c.w[0], x, c.ids, lambda s: s)
    up, ub = product(c.w[1], x, c.ids, lambda s: s)
    want, bound = R.gate_up(gate, gb, up, ub)
    R.close(ops.moe_gate_up_mxfp4(*c.packs, x, c.offsets, N, c.order), want, R.rounded(want, bound, c.dtype))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens,top_k,experts,K,N", [(6, 2, 4, 224, 50), (3, 1, 1, 5120, 70), (150, 2, 3, 224, 50), (300, 1, 1, 1056, 300)])
def test_some_rows_with_far_blocks(ops, kind, tokens, top_k, experts, K, N):  # noqa: F811
    """One row in five has blocks at any distance up to 60, and x zeros in half of its blocks; the other
    rows' results are those of a weight without such rows, bit for bit."""
    g = gen(K + tokens)
    c = Layer(ops, kind, tokens, top_k, experts, K, N, weights=2)
    near = [b.clone() for b in c.blocks]
    some = torch.arange(N) % 5 == 3
    x = c.rows(tokens) * 0.5
    x = torch.where((torch.rand(K // 32, generator=g) < 0.5).repeat_interleave(32).cuda(), x, torch.zeros_like(x))
    clean = (ops.qgemm_mxfp4(c.packs[0], x, c.offsets, N, order=c.order, top_k=top_k),
             ops.moe_gate_up_mxfp4(*c.packs, x, c.offsets, N, c.order, top_k))
    for i in range(2):
        blocks = near[i].clone()
        drop = torch.randint(0, 61, (experts, N, K // 32), generator=g).to(torch.uint8).cuda()
        blocks[..., 0] = torch.where(some[:, None].cuda(), 140 - drop, blocks[..., 0])
        set_blocks(c, i, blocks)
    y, bound = product(c.w[0], x, c.ids, lambda s: s // top_k)
    got = ops.qgemm_mxfp4(c.packs[0], x, c.offsets, N, order=c.order, top_k=top_k)
    fine = y.abs() < torch.finfo(c.dtype).max / 2
    assert bool(fine[:, ~some].all())  # (fp16 holds the others' only in part: scales of 2^13)
    R.close(got[fine], y[fine], R.rounded(y, bound, c.dtype)[fine])
    assert torch.equal(got[:, ~some], clean[0][:, ~some])
    got = ops.moe_gate_up_mxfp4(*c.packs, x, c.offsets, N, c.order, top_k)
    assert torch.equal(got[:, ~some], clean[1][:, ~some])
    if kind != "float16":
        up, ub = product(c.w[1], x, c.ids, lambda s: s // top_k)
        want, bound = R.gate_up(y, bound, up, ub)
        R.close(got, want, R.rounded(want, bound, c.dtype))


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("tokens", [4, 100])
def test_values_that_are_not_finite_in_a_far_block(ops, kind, tokens):  # noqa: F811
    c = Layer(ops, kind, tokens, 1, 1, 96, 24, ids=torch.zeros((tokens, 1), dtype=torch.int32))
    for l in (40, 200):
        blocks = c.blocks[0].clone()
        blocks[..., 0] = 250
        blocks[:, :, 1, 0] = 250 - l
        blocks[0, :, 1, 1:] &= 0x77  # (of one sign: an infinity's sign is that of x)
        blocks[0, :, 1, 1:] |= 0x11
        blocks[0, 7, 2, 0] = 255
        set_blocks(c, 0, blocks)
        x = c.rows(tokens).float() * 2.0 ** -100
        x[0, 40] = torch.inf
        x[1, 41] = -torch.inf
        x[2, 42] = torch.nan
        x = x.to(c.dtype)
        want = (x.double()[:, None, :] * c.w[0][0]).sum(-1)
        got = ops.qgemm_mxfp4(c.packs[0], x, c.offsets, 24)
        assert torch.equal(got[:3].isnan(), want[:3].isnan()) and bool(got[:, 7].isnan().all())
        inf = want[:2].isinf()
        assert torch.equal(got[:2][inf].double(), want[:2][inf])
