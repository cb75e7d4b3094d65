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
