"""Sums of 16-bit rows of one sign, which lose the most to an accumulator that cuts: at most
2^-23 of the sum for each product of 16 values (include/qgemv.h), whatever the number of rows."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import _mx_ref as R  # noqa: E402

from .test_gpu_mxfp4 import gen, ops  # noqa: E402, F401


@pytest.mark.parametrize("kind", ["float16", "bfloat16"])
@pytest.mark.parametrize("tokens,K", [(3, 5120), (3, 16384), (3, 32768), (90, 256), (90, 5120), (90, 16384), (200, 32768)])
def test_sums_of_one_sign(ops, kind, tokens, K):  # noqa: F811
    N, dtype = 40, getattr(torch, kind)
    blocks = R.random_blocks(gen(K), N, K, lo=115, hi=121)
    blocks[..., 1:] &= 0x77
    x = (torch.rand((tokens, K), generator=gen(tokens)) / 64).to(dtype).cuda()
    pack = ops.qpack_mxfp4(blocks.cuda(), 1, N, K)
    want = x.double() @ R.values(blocks.cuda()).T
    assert float(want.max()) < 6e4
    got = ops.qgemm_mxfp4(pack, x, torch.tensor([0, tokens], dtype=torch.int32, device="cuda"), N)
    # (and a fused multiply-add a block, where the blocks' sums are apart)
    R.close(got, want, R.rounded(want, want * (K / 16 * 2.0 ** -23 + K / 32 * 2.0 ** -24), dtype))
    # roundings to the output's type are as often up as down: their mean is near zero, a cut's is not
    off = ((got.double() - want) / want).mean()
    noise = 6 * R.HALF_STEP[dtype] / (3 * want.numel()) ** 0.5  # six deviations of a mean of even ones
    assert -(K / 16 * 2.0 ** -23) - noise <= float(off) <= noise + 2.0 ** -20
