"""The sparse layer's calls at the ends of their ranges: most experts, longest
rows, most places a token, many slots, offsets past 32 bits, subnormal halves,
workspaces with anything in them, threads, and the ctypes way of a call."""
import threading
import types

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import _mx_ref as R  # noqa: E402

from .test_gpu_mxfp4 import TYPES, Layer, gen, layer_weights, ops, run_layer  # noqa: E402, F401


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens", [3, 1200])
def test_most_experts_and_places(ops, kind, tokens):  # noqa: F811
    """1024 experts, 32 places a token: up to 8 slots an expert, and more."""
    c = Layer(ops, kind, tokens, 32, 1024, 64, 48, weights=2)
    x = c.rows(tokens)
    c.gemm(x)
    c.gate_up(x * 0.5)
    c.down(c.rows(tokens * 32), torch.rand((tokens, 32), generator=gen(1)).cuda())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens,K", [(2, 16384), (2, 16416), (2, 32768), (40, 32768)])
def test_longest_rows(ops, kind, tokens, K):  # noqa: F811
    c = Layer(ops, kind, tokens, 1, 2, K, 40)
    c.gemm(c.rows(tokens))


@pytest.mark.parametrize("kind", TYPES)
def test_many_slots(ops, kind):  # noqa: F811
    c = Layer(ops, kind, 60_001, 4, 16, 32, 24)
    c.gemm(c.rows(60_001))
    g = gen(2)
    c.down(c.rows(4 * 60_001), torch.rand((60_001, 4), generator=g).cuda())


@pytest.mark.parametrize("tokens", [2, 160])
def test_subnormal_halves(ops, tokens):  # noqa: F811
    """fp16 rows below 2^-14 go in as they are."""
    c = Layer(ops, "float16", tokens, 1, 2, 128, 32, scales=(130, 134))
    x = (c.rows(tokens).float() * 2.0 ** -19).half()
    assert bool((x.abs() < 2.0 ** -14).any()) and bool((x != 0).any())
    c.gemm(x)


def test_outputs_past_32_bits(ops):  # noqa: F811
    """4.6e9 outputs; rows from all over them."""
    tokens, K, N = 70_000, 32, 65_536
    c = Layer(ops, "bfloat16", tokens, 1, 2, K, N)
    x = c.rows(tokens)
    y = ops.qgemm_mxfp4(c.packs[0], x, c.offsets, N, order=c.order)
    at = torch.cat([torch.tensor([0, 1, tokens - 2, tokens - 1]), torch.randint(0, tokens, (60,), generator=gen(3))]).cuda()
    want, bound = R.product(c.w[0], x[at], c.ids[at], lambda s: s)
    R.close(y[at], want, R.rounded(want, bound, torch.bfloat16))


@pytest.mark.parametrize("tokens", [3, 80])
def test_weights_past_32_bits(ops, tokens):  # noqa: F811
    """A pack of 4.7e9 bytes: the first, a middle and the last expert."""
    E, N, K = 1024, 16_384, 512
    blocks = torch.randint(0, 256, (E * N, K // 32, 17), dtype=torch.uint8, device="cuda")
    blocks[..., 0] = 120
    pack = ops.qpack_mxfp4(blocks, E, N, K)
    assert pack.numel() > 1 << 32
    ids = (torch.arange(tokens) % 3)[:, None]
    real = torch.tensor([0, 611, E - 1], dtype=torch.int32)[ids].cuda()
    offsets, order = ops.moe_group(real.contiguous(), E)
    x = torch.randn((tokens, K), generator=gen(1)).bfloat16().cuda()
    y = ops.qgemm_mxfp4(pack, x, offsets, N, order=order)
    for t in range(3):
        rows = ids[:, 0].cuda() == t
        w = R.values(blocks[int(real[t]) * N:(int(real[t]) + 1) * N])
        zero = torch.zeros((int(rows.sum()), 1), dtype=torch.int64, device="cuda")
        want, bound = R.product(w[None], x[rows], zero, lambda s: s)
        R.close(y[rows], want, R.rounded(want, bound, torch.bfloat16))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens", [5, 90])
def test_workspaces_hold_anything(ops, kind, tokens):  # noqa: F811
    made = layer_weights(ops, 6, 128, 96, 2)
    dtype = getattr(torch, kind)
    g = gen(tokens)
    x = torch.randn((tokens, 129), generator=g).to(dtype).cuda()[:, 1:]  # (rows off 16-byte boundaries)
    logits = torch.randn((tokens, 6), generator=g).cuda()
    ids, weights, h, out = run_layer(ops, made, x, logits, 2)
    _, _, offsets, order = ops.moe_route(logits, 2)
    code = ops._TYPES[dtype]
    for fill in (0, 255):
        def ws(need):
            return torch.full((max(need, 16),), fill, dtype=torch.uint8, device="cuda")

        got = ops.moe_route(logits, 2, ws=ws(ops.moe_route_workspace_bytes(tokens, 6, 2)))
        assert torch.equal(got[0], ids) and torch.equal(got[2], offsets) and torch.equal(got[3], order)
        need = ops.LIB.moe_gate_up_mxfp4_workspace_bytes(code, tokens, 2, 6, 128, 96)
        assert torch.equal(ops.moe_gate_up_mxfp4(made[0][1], made[1][1], x, offsets, 96, order, 2, ws=ws(need)), h)
        need = ops.LIB.moe_down_mxfp4_workspace_bytes(code, tokens, 2, 6, 96, 128)
        assert torch.equal(ops.moe_down_mxfp4(made[2][1], h, offsets, 128, order, weights, ws=ws(need)), out)
        with pytest.raises(ops.QgemvError):
            ops.moe_down_mxfp4(made[2][1], h, offsets, 128, order, weights, ws=ws(need)[:need - 16])


def test_weights_of_slots_without_an_expert_are_not_read(ops):  # noqa: F811
    made = layer_weights(ops, 4, 64, 64, 1)
    for tokens in (3, 100):
        ids = torch.randint(0, 4, (tokens, 2), generator=gen(1), dtype=torch.int32)
        ids[::2, 1] = -1
        offsets, order = ops.moe_group(ids.cuda(), 4)
        h = torch.randn((tokens * 2, 64), generator=gen(2)).cuda()
        weights = torch.rand((tokens, 2), generator=gen(3)).cuda()
        want = ops.moe_down_mxfp4(made[2][1], h, offsets, 64, order, weights)
        weights[::2, 1] = float("nan")
        h[1::4] = float("nan")
        assert torch.equal(ops.moe_down_mxfp4(made[2][1], h, offsets, 64, order, weights), want)


def test_threads_call_at_once(ops):  # noqa: F811
    made = layer_weights(ops, 8, 256, 128, 5)
    g = gen(2)
    cases = [(torch.randn((n, 256), generator=g).bfloat16().cuda(), torch.randn((n, 8), generator=g).cuda()) for n in (4, 70, 9, 200)]
    want = [run_layer(ops, made, x, logits, 2)[3].clone() for x, logits in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i, stream):
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = run_layer(ops, made, *cases[i], 2)[3]
                stream.synchronize()
                if not torch.equal(got, want[i]):
                    wrong.append(i)

    one = torch.cuda.Stream()
    threads = [threading.Thread(target=work, args=(i, one if i < 2 else torch.cuda.Stream())) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []


@pytest.mark.parametrize("tokens", [4, 100])
def test_the_ctypes_way_gives_the_same(ops, tokens, monkeypatch):  # noqa: F811
    made = layer_weights(ops, 5, 96, 64, 7)
    g = gen(tokens)
    x = torch.randn((tokens, 96), generator=g).cuda()
    logits = torch.randn((tokens, 5), generator=g).cuda()

    def everything():
        blocks = ops.quantize_mxfp4(x)
        back = torch.empty_like(x)
        ops.dequantize_mxfp4(blocks, out=back)
        out = torch.empty((tokens, 64), device="cuda")
        offsets = torch.tensor([0, tokens, tokens, tokens, tokens, tokens], dtype=torch.int32, device="cuda")
        ops.qgemm_mxfp4(made[0][1], x, offsets, 64, y=out)
        return (blocks, back, ops.dequantize_mxfp4(blocks, dtype=torch.float16), out, *run_layer(ops, made, x, logits, 2))

    fast = everything()
    monkeypatch.setattr(ops, "_CALLS", types.SimpleNamespace(
        **{n: lambda *args: None for n in ("quantize_mxfp4", "dequantize_mxfp4", "moe_route", "product")}))
    for a, b in zip(fast, everything()):
        assert torch.equal(a, b)


def test_refusals_of_device_tensors(ops):  # noqa: F811
    c = Layer(ops, "bfloat16", 6, 2, 3, 64, 32)
    x = c.rows(6)
    bad = [
        dict(x=x.t()), dict(x=x.expand(2, 6, 64)), dict(x=x[:1].expand(6, 64)), dict(x=x.int()), dict(order=c.order[:5]),
        dict(order=c.order.long()), dict(offsets=c.offsets[:3]), dict(offsets=c.offsets.cpu()), dict(w_pack=c.packs[0][:-16]),
        dict(N=33), dict(top_k=3), dict(y=torch.empty((12, 31), dtype=torch.bfloat16, device="cuda")),
        dict(y=torch.empty((12, 32), device="cuda")), dict(ws=torch.empty(64, device="cuda"))]
    for change in bad:
        args = dict(w_pack=c.packs[0], x=x, offsets=c.offsets, N=32, order=c.order, top_k=2)
        args.update(change)
        with pytest.raises(ValueError):
            ops.qgemm_mxfp4(**args)
    with pytest.raises(ValueError):
        ops.moe_down_mxfp4(c.packs[0], x, c.offsets, 32, c.order, torch.ones((6, 2), device="cuda"))
    with pytest.raises(ValueError):
        ops.moe_route(x, 65)
    with pytest.raises(ValueError):
        ops.quantize_mxfp4(x[:, :40])
    with pytest.raises(ValueError):
        ops.dequantize_mxfp4(c.blocks[0].view(3, 32, 2, 17)[..., :16])
    with pytest.raises(ops.QgemvError):
        ops.moe_route(torch.zeros((4, 2000), device="cuda"), 2)


@pytest.mark.parametrize("tokens", [5, 90])
def test_offsets_that_fall_count_as_the_largest_before(ops, tokens):  # noqa: F811
    c = Layer(ops, "float32", tokens, 2, 6, 64, 48)
    x, h = c.rows(tokens), c.rows(tokens * 2)
    weights = torch.rand((tokens, 2), generator=gen(1)).cuda()
    n = 2 * tokens
    for offsets in ([n // 2, 0, n, 0, n, 3, 1], [1, n // 2, 2, n // 3, n - 2, 0, 0], [5, 4, 3, 2, 1, 0, -1]):
        falling = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        rising = torch.cummax(falling.clamp(0, n), 0).values
        assert torch.equal(ops.qgemm_mxfp4(c.packs[0], x, falling, 48, order=c.order, top_k=2),
                           ops.qgemm_mxfp4(c.packs[0], x, rising, 48, order=c.order, top_k=2))
        assert torch.equal(ops.moe_down_mxfp4(c.packs[0], h, falling, 48, c.order, weights),
                           ops.moe_down_mxfp4(c.packs[0], h, rising, 48, c.order, weights))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("tokens", [1, 40])
def test_silu_far_below_zero(ops, kind, tokens):  # noqa: F811
    """g = -80, -88 (e^88 is still an fp32 number, its sum's quotient small), -96 (e^96 is none); h near 1.

    The exponential of |g| has (2 + 1.2 |g|) 2^-23 for 16-bit outputs and 2^-22
    for fp32, or two steps where it is subnormal: 2^-149 of e^-96 = 2^-138.5, so 2^-9.5; then
    three roundings of 2^-23 and the output's own."""
    dtype = getattr(torch, kind)
    N, sums = 3, (80, 88, 96)
    blocks = torch.zeros((2, N, 1, 17), dtype=torch.uint8)
    blocks[0, :, 0, 0] = 127 + 3
    for n, total in enumerate(sums):  # eighths: ten, eleven, twelve of them as codes -6 (15), -4 (14), -1 (10), -2 (12)
        for i, code in enumerate({80: (15, 14), 88: (15, 14, 10), 96: (15, 14, 12)}[total]):
            blocks[0, n, 0, 1 + i] = code
    powers = torch.tensor([109, 120, 127])  # up: 2^p from code 1 (2) of scale p
    blocks[1, :, 0, 0] = (127 + powers).to(torch.uint8)
    blocks[1, :, 0, 1] = 2
    gate, up = (ops.qpack_mxfp4(blocks[i].cuda(), 1, N, 32) for i in range(2))
    x = torch.ones((tokens, 32), dtype=dtype, device="cuda")
    offsets = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    got = ops.moe_gate_up_mxfp4(gate, up, x, offsets, N)
    g = -torch.tensor(sums, dtype=torch.float64)
    want = g / (1 + torch.exp(-g)) * 2.0 ** powers.double()
    exp = (2 + 1.2 * g.abs()) * 2.0 ** -23 if kind != "float32" else torch.full((3,), 2.0 ** -22, dtype=torch.float64)
    exp = torch.maximum(exp, 2 * 2.0 ** -149 / torch.exp(g))
    R.close(got.cpu(), want.expand(tokens, N), R.rounded(want, want.abs() * (exp + 3 * 2.0 ** -23), dtype))


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("lo", [20, 60, 118, 170, 235])
@pytest.mark.parametrize("tokens", [5, 90])
def test_powers_of_rows_and_weights_far_apart(ops, kind, lo, tokens):  # noqa: F811
    """Rows of 2^-110 to 2^110 in one call with weights of 2^-107 to 2^112: only the
    product of the two has to be an fp32 number."""
    c = Layer(ops, kind, tokens, 1, 2, 64, 40, scales=(lo, lo + 5))
    power = torch.tensor([-110, -40, 0, 50, 110], dtype=torch.float64)[torch.arange(tokens) % 5, None].cuda()
    x = (c.rows(tokens).double() * 2.0 ** power).to(c.dtype)
    y, bound = R.product(c.w[0], x, c.ids, lambda s: s)
    most = torch.finfo(c.dtype).max
    assert not bool(((y.abs() > most / 4) & (y.abs() < most * 4)).any())
    y = torch.where(y.abs() > most, y.sign() * torch.inf, y)
    got = ops.qgemm_mxfp4(c.packs[0], x, c.offsets, c.N, order=c.order)
    bound = torch.where(y.isinf(), 0.0, R.rounded(y, bound, c.dtype))
    R.close(got, y, bound)


@pytest.mark.parametrize("tokens,K", [(90, 256), (90, 320), (90, 5120), (200, 16384), (2, 32768)])
def test_sums_of_fp32_rows_of_one_sign(ops, tokens, K):  # noqa: F811
    """Sums that only grow lose the most to an accumulator that cuts: one of 256 values has 32
    products (two terms of x), each cut by 2^-23 at most; then a rounding for each of them, x's
    own (2^-23) and the output's."""
    N = 40
    blocks = R.random_blocks(gen(K), N, K)
    blocks[..., 1:] &= 0x77
    x = torch.rand((tokens, K), generator=gen(tokens)).cuda()
    pack = ops.qpack_mxfp4(blocks.cuda(), 1, N, K)
    want = x.double() @ R.values(blocks.cuda()).T
    got = ops.qgemm_mxfp4(pack, x, torch.tensor([0, tokens], dtype=torch.int32, device="cuda"), N)
    R.close(got, want, want * (33 * 2.0 ** -23 + (K / 256 + 1) * 2.0 ** -24))
