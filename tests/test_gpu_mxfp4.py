"""The MXFP4 format and the sparse layer on a GPU against a plain 64-bit
implementation (tests/_mx_ref.py): bytes, ids and order exactly, products
within bounds derived from their arithmetic."""
import math

import pytest
import torch

from tests import _mx_ref as R

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]
TINY = {"float32": 2.0 ** -149, "float16": 2.0 ** -24, "bfloat16": 2.0 ** -133}


@pytest.fixture(scope="module")
def ops():
    from block_quantized_gemv_quantize_gb300 import ops as o

    return o


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ format


def special_rows(dtype):
    """Blocks at the borders of the format: ties, saturation, both zeros, ends of the type."""
    big = torch.finfo(dtype).max
    tiny = TINY[str(dtype)[6:]]
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]
    rows = [
        [4.0] + ties + [-t for t in ties] + [0.2499, 0.2501, 0.7499, 0.7501, 4.999, 5.001, 6.999, 7.999, -0.0, 0.0] + [0.5] * 5,
        [0.0] * 32,
        [-0.0] * 31 + [tiny],
        [tiny * i for i in range(32)],
        [big] + [big / 2, -big / 4, big / 8, 1.0] * 7 + [0.0] * 3,
        [math.inf] + [1.0] * 31,
        [1.0] * 31 + [math.nan],
        [0.0] * 31 + [-math.inf],
        [7.9, 7.51, 7.49, 6.01, 5.99] + [0.1] * 27,
        [2.0 ** -i for i in range(32)],
    ]
    return torch.tensor(rows, dtype=torch.float64).to(dtype)


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_special_blocks(ops, kind):
    x = special_rows(getattr(torch, kind))
    blocks = ops.quantize_mxfp4(x.cuda())
    assert torch.equal(blocks.cpu(), R.quantize(x))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("N,K,pad", [(1, 32, 0), (3, 96, 0), (7, 1056, 8), (33, 64, 3), (5, 5120, 0), (600, 32, 1)])
def test_quantize_and_back(ops, kind, N, K, pad):
    dtype = getattr(torch, kind)
    g = gen(N * K + pad)
    wide = (torch.randn((N, K + pad), generator=g) * torch.exp2(torch.randint(-12, 8, (N, 1), generator=g).float())).to(dtype)
    x = wide.cuda()[:, pad:]
    blocks = ops.quantize_mxfp4(x)
    want = R.quantize(x.cpu())
    assert torch.equal(blocks.cpu(), want)
    exact = R.values(want)
    for out_kind in TYPES:
        out_type = getattr(torch, out_kind)
        back = ops.dequantize_mxfp4(blocks, dtype=out_type)
        assert torch.equal(back.cpu().double(), exact.to(out_type).double())
    held = torch.full((N, K + pad), 5.0, dtype=dtype, device="cuda")
    ops.dequantize_mxfp4(blocks, out=held[:, pad:])
    assert torch.equal(held[:, pad:].cpu().double(), exact.to(dtype).double())
    assert bool((held[:, :pad] == 5.0).all())


def test_dequantize_every_code_and_scale(ops):
    blocks = torch.zeros((256, 1, 17), dtype=torch.uint8)
    blocks[:, 0, 0] = torch.arange(256)
    blocks[:, 0, 1:] = torch.arange(16) | (15 - torch.arange(16)) << 4
    want = R.values(blocks)
    for kind in TYPES:
        got = ops.dequantize_mxfp4(blocks.cuda(), dtype=getattr(torch, kind)).cpu()
        want_t = want.float().to(getattr(torch, kind))  # (6 * 2^127 and more: infinite in fp32 as well)
        assert torch.equal(got.nan_to_num(nan=-7.0, posinf=-8.0, neginf=-9.0), want_t.nan_to_num(nan=-7.0, posinf=-8.0, neginf=-9.0))


def test_quantize_many_rows(ops):
    """More runs than the grid takes at a time, a row a block."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((400_001, 32), generator=g, device="cuda")
    blocks = ops.quantize_mxfp4(x)
    at = torch.randint(0, x.shape[0], (50,))
    assert torch.equal(blocks[at.cuda()].cpu(), R.quantize(x[at.cuda()].cpu()))
    back = ops.dequantize_mxfp4(blocks)
    assert torch.equal(back.double(), R.values(blocks))


# ------------------------------------------------------------------ router


def check_route(ops, logits, top_k, score, renormalize, scale):
    ids, weights, offsets, order = ops.moe_route(logits.cuda(), top_k, score=score, renormalize=renormalize, scale=scale)
    want_ids, want = R.route(logits, top_k, score, renormalize, scale)
    assert torch.equal(ids.cpu(), want_ids)
    want_offsets, want_order = R.group(want_ids, logits.shape[1])
    assert torch.equal(offsets.cpu(), want_offsets)
    assert torch.equal(order.cpu(), want_order)
    # a difference of logits in fp32 (2^-24 of 128 at most: 2^-17 of the weight
    # covers it for these), exp, a sum of up to 1024, a quotient, a product
    tol = 2.0 ** -24 * (8 + logits.shape[1] / 32 + 2 * float(logits.double().nan_to_num(0, 0, 0).abs().max())) * 2
    R.close(weights.cpu(), want, want.abs() * tol + 1e-37)
    return ids, weights, offsets, order


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 64, 6), (7, 33, 5), (6, 8, 8), (17, 256, 8),
                                                  (64, 1000, 32), (257, 60, 4), (2049, 1, 1), (1500, 128, 8), (700, 1024, 3)])
@pytest.mark.parametrize("score,renormalize,scale", [("softmax", True, 1.0), ("softmax", False, 2.5), ("sigmoid", True, 1.0),
                                                     ("sigmoid", False, -0.5)])
def test_route(ops, kind, tokens, experts, top_k, score, renormalize, scale):
    g = gen(tokens + experts)
    logits = (3 * torch.randn((tokens, experts), generator=g)).to(getattr(torch, kind))
    check_route(ops, logits, top_k, score, renormalize, scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [40, 900])
def test_route_masks_ties_and_nan(ops, score, tokens):
    g = gen(3)
    logits = torch.randint(-2, 3, (tokens, 48), generator=g).float()  # many ties
    logits[:, 7] = -math.inf
    logits[1::5] = -math.inf  # rows that leave nothing
    logits[2::5, 4:] = -math.inf  # rows that leave fewer than top_k
    logits[3::5, 3] = math.nan
    logits[4::5] = math.nan
    logits[0, :] = -0.0
    logits[0, 9] = 0.0
    logits[0, 7] = torch.finfo(torch.float32).min  # the lowest number is one
    ids, weights, _, _ = check_route(ops, logits, 6, score, True, 1.0)
    assert ids[0].tolist() == [0, 1, 2, 3, 4, 5]
    assert bool((ids[1::5] == -1).all()) and bool((weights[1::5] == 0).all())


def test_route_far_sigmoid_logits_keep_their_ratio(ops):
    logits = torch.tensor([[-200.0, -201.0, -300.0, 200.0], [-200.0, -201.0, -300.0, -math.inf]])
    _, w, _, _ = ops.moe_route(logits.cuda(), 3, score="sigmoid")
    assert abs(float(w[1, 0]) - 1 / (1 + math.exp(-1))) < 1e-6
    assert float(w[0, 0]) == 1.0


def test_route_rows_with_strides(ops):
    g = gen(8)
    wide = torch.randn((50, 70), generator=g).bfloat16()
    check = wide[:, 3:63].clone()
    got = ops.moe_route(wide.cuda()[:, 3:63], 4)
    want = ops.moe_route(check.cuda(), 4)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("tokens,top_k,experts", [(1, 1, 1), (5, 3, 4), (3000, 2, 17), (211, 32, 1024), (9000, 7, 300),
                                                  (40000, 8, 1024)])
def test_group(ops, tokens, top_k, experts):
    g = gen(tokens)
    ids = torch.randint(-2, experts + 2, (tokens, top_k), generator=g, dtype=torch.int32)
    offsets, order = ops.moe_group(ids.cuda(), experts)
    want_offsets, want_order = R.group(ids, experts)
    assert torch.equal(offsets.cpu(), want_offsets) and torch.equal(order.cpu(), want_order)


def test_no_tokens(ops):
    ids, weights, offsets, order = ops.moe_route(torch.empty((0, 16), device="cuda"), 4)
    assert ids.shape == (0, 4) and order.numel() == 0 and offsets.tolist() == [0] * 17
    offsets, order = ops.moe_group(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 5)
    assert offsets.tolist() == [0] * 6
    pack = ops.qpack_mxfp4(torch.zeros((16 * 16, 2, 17), dtype=torch.uint8, device="cuda"), 16, 16, 64)
    x = torch.empty((0, 64), device="cuda")
    none = torch.zeros(17, dtype=torch.int32, device="cuda")
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    assert ops.qgemm_mxfp4(pack, x, none, 16, order=empty, top_k=4).shape == (0, 16)
    assert ops.moe_down_mxfp4(pack, x, none, 16, empty, torch.empty((0, 4), device="cuda")).shape == (0, 16)


# ------------------------------------------------------------------ products


class Layer:
    """Weights, ids and rows of a random case, on the GPU."""

    def __init__(self, ops, kind, tokens, top_k, experts, K, N, ids="random", seed=0, pad=0, weights=1, scales=(118, 124)):
        self.ops, self.dtype = ops, getattr(torch, kind)
        self.N, self.top_k, self.tokens, self.experts = N, top_k, tokens, experts
        g = gen(seed + tokens * 7 + K)
        self.blocks = [R.random_blocks(g, experts, N, K, lo=scales[0], hi=scales[1]).cuda() for _ in range(weights)]
        self.w = [R.values(b) for b in self.blocks]
        self.packs = [ops.qpack_mxfp4(b, experts, N, K) for b in self.blocks]
        if ids == "random":  # some experts popular, some without a row, some slots without an expert
            p = torch.exp(1.5 * torch.randn(experts + 1, generator=g))
            ids = torch.multinomial(p, tokens * top_k, replacement=True, generator=g).view(tokens, top_k).int() - 1
        elif ids == "one":
            ids = torch.full((tokens, top_k), experts - 1, dtype=torch.int32)
        self.ids = ids.cuda()
        self.offsets, self.order = ops.moe_group(self.ids.contiguous(), experts)
        self.rows = lambda n: (torch.randn((n, K + pad), generator=g) * torch.where(
            torch.rand(K + pad, generator=g) < 0.02, 20.0, 1.0)).to(self.dtype).cuda()[:, pad:]

    def gemm(self, x):
        y, bound = R.product(self.w[0], x, self.ids, lambda s: s // self.top_k)
        got = self.ops.qgemm_mxfp4(self.packs[0], x, self.offsets, self.N, order=self.order, top_k=self.top_k)
        R.close(got, y, R.rounded(y, bound, self.dtype))
        return got

    def gate_up(self, x):
        g, gb = R.product(self.w[0], x, self.ids, lambda s: s // self.top_k)
        u, ub = R.product(self.w[1], x, self.ids, lambda s: s // self.top_k)
        h, bound = R.gate_up(g, gb, u, ub)
        got = self.ops.moe_gate_up_mxfp4(*self.packs, x, self.offsets, self.N, self.order, self.top_k)
        R.close(got, h, R.rounded(h, bound, self.dtype))
        return got

    def down(self, h, weights):
        y, bound = R.product(self.w[0], h, self.ids, lambda s: s)
        out, bound = R.down(y, bound, weights)
        got = self.ops.moe_down_mxfp4(self.packs[0], h, self.offsets, self.N, self.order, weights)
        R.close(got, out, R.rounded(out, bound, self.dtype))
        return got


SHAPES = [  # tokens, top_k, experts, K, N
    (1, 1, 1, 32, 1),
    (1, 6, 64, 512, 96),
    (1, 2, 4, 5120, 48),
    (6, 6, 16, 1408, 200),
    (7, 2, 3, 96, 33),
    (17, 1, 1, 1056, 144),
    (40, 4, 8, 768, 72),
    (100, 2, 5, 224, 260),
    (333, 3, 4, 160, 129),
    (900, 2, 3, 512, 272),
    (64, 8, 256, 128, 16),
]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gemm(ops, kind, shape):
    c = Layer(ops, kind, *shape)
    c.gemm(c.rows(shape[0]))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gate_up(ops, kind, shape):
    c = Layer(ops, kind, *shape, weights=2)
    c.gate_up(c.rows(shape[0]) * 0.5)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_down(ops, kind, shape):
    c = Layer(ops, kind, *shape)
    g = gen(1)
    c.down(c.rows(shape[0] * shape[1]), torch.rand((shape[0], shape[1]), generator=g).cuda())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("pad", [1, 8, 40])
@pytest.mark.parametrize("tokens", [5, 200])
def test_rows_with_strides_and_given_outputs(ops, kind, pad, tokens):
    c = Layer(ops, kind, tokens, 2, 4, 256, 80, pad=pad)
    x = c.rows(tokens)
    want = c.gemm(x)
    held = torch.full((2 * tokens, 80 + pad), 3.0, dtype=c.dtype, device="cuda")
    ops.qgemm_mxfp4(c.packs[0], x, c.offsets, 80, order=c.order, top_k=2, y=held[:, pad:])
    assert torch.equal(held[:, pad:], want) and bool((held[:, :pad] == 3.0).all())
    h = c.rows(2 * tokens)
    w = torch.rand((tokens, 2), generator=gen(4)).cuda()
    want = c.down(h, w)
    held = torch.full((tokens, 80 + pad), 3.0, dtype=c.dtype, device="cuda")
    ops.moe_down_mxfp4(c.packs[0], h, c.offsets, 80, c.order, w, out=held[:, pad:])
    assert torch.equal(held[:, pad:], want) and bool((held[:, :pad] == 3.0).all())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("counts", [[0, 5, 0, 200, 1, 0], [0, 0, 0], [33], [1] * 40, [8, 9, 16, 17, 127, 128, 129, 0]])
def test_sorted_rows_without_an_order(ops, kind, counts):
    ids = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).int()[:, None]
    ids = torch.cat([ids, torch.full((3, 1), -1, dtype=torch.int32)])  # rows behind the last expert's
    c = Layer(ops, kind, ids.shape[0], 1, len(counts), 288, 100, ids=ids)
    x = c.rows(ids.shape[0])
    want = c.gemm(x)
    assert torch.equal(ops.qgemm_mxfp4(c.packs[0], x, c.offsets, 100), want)
    assert bool((want[-3:] == 0).all())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens", [3, 150])
def test_every_slot_one_expert_or_none(ops, kind, tokens):
    c = Layer(ops, kind, tokens, 2, 5, 128, 64, ids="one")
    c.gemm(c.rows(tokens))
    c = Layer(ops, kind, tokens, 2, 5, 128, 64, ids=torch.full((tokens, 2), -1, dtype=torch.int32))
    assert bool((c.gemm(c.rows(tokens)) == 0).all())
    assert bool((c.down(c.rows(2 * tokens), torch.ones((tokens, 2), device="cuda")) == 0).all())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens", [2, 160])
def test_infinities_and_nan(ops, kind, tokens):
    """A NaN in a row of x or a NaN block of a weight's row makes what it enters
    NaN and nothing else; an infinity what the formula has."""
    ids = torch.arange(tokens * 2).view(tokens, 2).int() % 3
    c = Layer(ops, kind, tokens, 2, 3, 192, 48, ids=ids)
    c.blocks[0][1, 5, 2, 0] = 255
    c.blocks[0][2, 6, 0, 1:] = 0  # zeros that meet an infinity
    c.w[0] = R.values(c.blocks[0])
    c.packs[0] = ops.qpack_mxfp4(c.blocks[0], 3, 48, 192)
    x = c.rows(tokens)
    x[0, 3] = math.inf
    x[1, 100] = math.nan
    want = torch.zeros((tokens * 2, 48), dtype=torch.float64, device="cuda")
    for s in range(tokens * 2):
        want[s] = (x[s // 2].double() * c.w[0][int(c.ids.flatten()[s])]).sum(-1)
    got = ops.qgemm_mxfp4(c.packs[0], x, c.offsets, 48, order=c.order, top_k=2)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.isinf() & (got > 0), want.isinf() & (want > 0))
    assert torch.equal(got.isinf() & (got < 0), want.isinf() & (want < 0))
    fine = want.isfinite()
    _, bound = R.product(c.w[0].nan_to_num(0), x.nan_to_num(0, 0, 0), c.ids, lambda s: s // 2)
    assert bool(((got.double() - want).abs() <= R.rounded(want, bound, c.dtype))[fine].all())


@pytest.mark.parametrize("kind,power", [("float32", 100), ("float32", -100), ("bfloat16", 100), ("bfloat16", -100),
                                        ("float16", 10), ("float16", -10)])
@pytest.mark.parametrize("tokens", [2, 160])
def test_rows_and_scales_far_from_one(ops, kind, power, tokens):
    """Large rows against small weights and the other way: products that fp32 holds."""
    c = Layer(ops, kind, tokens, 1, 2, 256, 32, scales=(122 - power, 126 - power))
    x = torch.ldexp(c.rows(tokens).float(), torch.tensor(power)).to(c.dtype)
    c.gemm(x)


@pytest.mark.parametrize("tokens", [2, 160])
def test_scales_far_apart_in_a_row(ops, tokens):
    c = Layer(ops, "float32", tokens, 1, 2, 512, 32, scales=(60, 180))
    c.gemm(c.rows(tokens))


@pytest.mark.parametrize("tokens", [3, 150])
def test_outputs_repeat_bit_for_bit(ops, tokens):
    c = Layer(ops, "bfloat16", tokens, 4, 9, 640, 112)
    h = c.rows(tokens * 4)
    w = torch.rand((tokens, 4), generator=gen(2)).cuda()
    first = c.down(h, w)
    for _ in range(5):
        assert torch.equal(ops.moe_down_mxfp4(c.packs[0], h, c.offsets, 112, c.order, w), first)


def test_offsets_and_order_that_do_not_fit_touch_nothing_else(ops):
    """Entries out of range are cut or skipped."""
    c = Layer(ops, "bfloat16", 40, 2, 4, 64, 32)
    x = c.rows(40)
    held = torch.full((82, 32), 3.0, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([-5, 30, 1 << 30, 20, 1 << 30], dtype=torch.int32, device="cuda")
    order = torch.randint(-100, 200, (80,), generator=gen(1), dtype=torch.int32).cuda()
    ops.qgemm_mxfp4(c.packs[0], x, offsets, 32, order=order, top_k=2, y=held[1:81])
    torch.cuda.synchronize()
    assert bool((held[0] == 3.0).all()) and bool((held[81] == 3.0).all())


# ------------------------------------------------------------------ a layer


def layer_weights(ops, E, K, N, seed):
    g = gen(seed)
    made = []
    for n, k in ((N, K), (N, K), (K, N)):
        w = torch.randn((E * n, k), generator=g) / math.sqrt(k)
        blocks = ops.quantize_mxfp4(w.cuda())
        made.append((R.values(blocks).view(E, n, k), ops.qpack_mxfp4(blocks, E, n, k)))
    return made


def run_layer(ops, made, x, logits, top_k):
    N, K = made[0][0].shape[1:]
    ids, weights, offsets, order = ops.moe_route(logits, top_k)
    h = ops.moe_gate_up_mxfp4(made[0][1], made[1][1], x, offsets, N, order, top_k)
    return ids, weights, h, ops.moe_down_mxfp4(made[2][1], h, offsets, K, order, weights)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens,E,K,N,top_k", [(1, 16, 256, 160, 4), (6, 8, 512, 96, 2), (190, 6, 128, 224, 3)])
def test_a_sparse_layer_from_router_to_sum(ops, kind, tokens, E, K, N, top_k):
    dtype = getattr(torch, kind)
    made = layer_weights(ops, E, K, N, tokens)
    g = gen(tokens + 1)
    x = torch.randn((tokens, K), generator=g).to(dtype).cuda()
    logits = torch.randn((tokens, E), generator=g).to(dtype).cuda()
    logits[tokens // 2 + 1:tokens // 2 + 3] = -math.inf  # padding
    ids, weights, h, out = run_layer(ops, made, x, logits, top_k)
    gate, gb = R.product(made[0][0], x, ids, lambda s: s // top_k)
    up, ub = R.product(made[1][0], x, ids, lambda s: s // top_k)
    want, bound = R.gate_up(gate, gb, up, ub)
    R.close(h, want, R.rounded(want, bound, dtype))
    y, bound = R.product(made[2][0], h, ids, lambda s: s)  # (from the h that the layer made)
    want, bound = R.down(y, bound, weights)
    R.close(out, want, R.rounded(want, bound, dtype))


def test_a_captured_layer_serves_new_routes(ops):
    """Counts are read on the device: one graph, any routing; a second graph of
    the same buffers and an eager call between the replays change nothing."""
    tokens, E, K, N, top_k = 24, 12, 256, 128, 4
    made = layer_weights(ops, E, K, N, 3)
    x = torch.zeros((tokens, K), dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros((tokens, E), device="cuda")
    run_layer(ops, made, x, logits, top_k)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run_layer(ops, made, x, logits, top_k))
        graphs.append(graph)
    g = gen(9)
    for i in range(4):
        new_x = torch.randn((tokens, K), generator=g).bfloat16().cuda()
        new_logits = (8.0 * i * torch.randn((1, E), generator=g) + torch.randn((tokens, E), generator=g)).cuda()
        x.copy_(new_x)
        logits.copy_(new_logits)
        graphs[i % 2].replay()
        want = run_layer(ops, made, new_x, new_logits, top_k)
        for a, b in zip(outs[i % 2], want):
            assert torch.equal(a, b)


def test_two_streams_at_once(ops):
    made = layer_weights(ops, 8, 512, 256, 5)
    g = gen(2)
    xs = [torch.randn((60, 512), generator=g).bfloat16().cuda() for _ in range(2)]
    logits = [torch.randn((60, 8), generator=g).cuda() for _ in range(2)]
    want = [run_layer(ops, made, x, l, 2)[3].clone() for x, l in zip(xs, logits)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run_layer(ops, made, xs[i], logits[i], 2)[3])
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert torch.equal(out, want[i])
