"""Products of rows of x whose largest magnitude is near the end of fp32's range or
subnormal, with weights that bring them back: what include/qgemv.h says of
rows holds for them too (22 bits or all of theirs, to no less than 2^-38 of the row's largest)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import _mx_ref as R  # noqa: E402

from .test_gpu_mxfp4 import Layer, gen, ops  # noqa: E402, F401

POWERS = [-90, -98, -105, -112, -120, -124, -126, -127, -130, -137, -141, -145]


def small_rows(dtype, tokens, K, seed):
    """Rows of 2^p, p from POWERS in turn (as far as the type goes), a few elements far below their row's."""
    g = gen(seed)
    x = torch.randn((tokens, K), generator=g, dtype=torch.float64)
    x = torch.where(torch.rand((tokens, K), generator=g) < 0.2, x * 2.0 ** -12, x)
    powers = [p for p in POWERS if dtype == torch.float32 or p >= -130]
    power = torch.tensor(powers, dtype=torch.float64)[torch.arange(tokens) % len(powers), None]
    return torch.ldexp(x, power).to(dtype).cuda()


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("tokens", [7, 96])
def test_every_element_of_small_rows(ops, kind, tokens):  # noqa: F811
    """Weights with one code a row: an output is one product, so that it shows what is left of
    its element: 2^-23 of it (fp32; bf16: nothing) and 2^-38 of the row's largest."""
    dtype, K = getattr(torch, kind), 64
    blocks = torch.zeros((K, 2, 17), dtype=torch.uint8)
    n = torch.arange(K)
    blocks[n, n // 32, 0] = 127 + 108
    blocks[n, n // 32, 1 + n % 16] = torch.where(n % 32 < 16, 2, 2 << 4).to(torch.uint8)  # code 1
    w = R.values(blocks)
    assert torch.equal(w, torch.eye(K, dtype=torch.float64) * 2.0 ** 108)
    pack = ops.qpack_mxfp4(blocks.cuda(), 1, K, K)
    x = small_rows(dtype, tokens, K, 1)
    assert bool((x != 0).any(-1).all())
    got = ops.qgemm_mxfp4(pack, x, torch.tensor([0, tokens], dtype=torch.int32, device="cuda"), K)
    want = x.double() * 2.0 ** 108
    own = 2.0 ** -23 if kind == "float32" else 0.0
    R.close(got, want, R.rounded(want, want.abs() * own + want.abs().amax(-1, keepdim=True) * 2.0 ** -38, dtype))


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("tokens,K,lo", [(7, 256, 205), (7, 256, 245), (96, 256, 205), (96, 256, 245), (96, 1056, 225)])
def test_products_of_small_rows(ops, kind, tokens, K, lo):  # noqa: F811
    c = Layer(ops, kind, tokens, 1, 1, K, 48, ids=torch.zeros((tokens, 1), dtype=torch.int32), weights=2, scales=(lo, lo + 5))
    x = small_rows(c.dtype, tokens, K, 2)
    c.gemm(x)
    y, bound = R.product(c.w[0], x, c.ids, lambda s: s)
    weights = torch.rand((tokens, 1), generator=gen(3)).cuda()
    want, bound = R.down(y, bound, weights)
    R.close(ops.moe_down_mxfp4(c.packs[0], x, c.offsets, 48, c.order, weights), want, R.rounded(want, bound, c.dtype))


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("tokens", [7, 96])
def test_rows_of_the_smallest_numbers(ops, kind, tokens):  # noqa: F811
    """A row's one element is the type's smallest; large weights make it a normal number."""
    dtype = getattr(torch, kind)
    tiny = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133}[kind]
    blocks = torch.zeros((16, 1, 17), dtype=torch.uint8)
    blocks[:, 0, 0] = 254 - torch.arange(16).to(torch.uint8)
    blocks[:, 0, 1] = 7 | 3 << 4  # 6 x[0] + 1.5 x[16]
    x = torch.zeros((tokens, 32), dtype=torch.float64)
    x[:, 16] = tiny
    x[1::2, 0] = tiny
    x[2::3] = 0.0
    pack = ops.qpack_mxfp4(blocks.cuda(), 1, 16, 32)
    got = ops.qgemm_mxfp4(pack, x.to(dtype).cuda(), torch.tensor([0, tokens], dtype=torch.int32, device="cuda"), 16)
    assert torch.equal(got.cpu().double(), x @ R.values(blocks).T)


@pytest.mark.parametrize("tokens", [6, 96])
@pytest.mark.parametrize("shift", [-103, -106, -107, -109, -112, -118])
def test_subnormal_outputs_round_once(ops, tokens, shift):  # noqa: F811
    """Outputs between 2^-122 and 2^-139, each one product of an element that two halves hold
    exactly (23 bits): the fp32 number nearest to it, of two the even one."""
    K = 64
    blocks = torch.zeros((K, 2, 17), dtype=torch.uint8)
    n = torch.arange(1, K)
    blocks[n, n // 32, 0] = 127 + shift
    blocks[n, n // 32, 1 + n % 16] = torch.where(n % 32 < 16, 2, 2 << 4).to(torch.uint8)  # code 1
    pack = ops.qpack_mxfp4(blocks.cuda(), 1, K, K)
    x = torch.randint(1 << 22, 1 << 23, (tokens, K), generator=gen(5)).double() * 2.0 ** -42  # [2^-20, 2^-19)
    x[:, 0] = 2.0 ** -4  # the row's largest, which no weight meets
    x[:, 1::3] *= -1
    got = ops.qgemm_mxfp4(pack, x.float().cuda(), torch.tensor([0, tokens], dtype=torch.int32, device="cuda"), K)
    want = x * 2.0 ** shift
    want[:, 0] = 0.0
    assert torch.equal(got.cpu(), want.float())
