"""The paged cache and the attention over it on the GPU, against the plain
implementation in 64 bits (tests/_kv_ref.py): bytes and values exactly,
attention within the bounds that its arithmetic gives."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from . import _kv_ref as R  # noqa: E402

DEV = "cuda:0"
FMTS = ["q8_0", "q4_0", "f16"]
TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_gemv_quantize_gb300 import build

    build.build()
    from block_quantized_gemv_quantize_gb300 import ops as o

    return o


def random_kv(rng, n, heads, dim):
    k = rng.standard_normal((n, heads, dim)).astype(np.float32)
    k[..., ::17] = 4 * k[..., ::17] + 3
    return k, rng.standard_normal((n, heads, dim)).astype(np.float32)


def edge_rows(heads, dim):
    """Blocks at which a quantizer can go wrong, as rows [n, heads, dim]."""
    rng = np.random.default_rng(9)
    x = rng.standard_normal((14, heads, dim)).astype(np.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2, ..., 5] = np.nan
    x[3, ..., 33 % dim] = np.inf
    x[4, ..., 31] = -np.inf
    x[5] = 1e-42  # the scale is subnormal
    x[6] = 3e38   # it passes fp16's range
    x[7] = np.tile(np.repeat(np.arange(16, dtype=np.float32) - 7.5, 2), dim // 32)  # halves and equal magnitudes
    x[7, ..., 0::32] = 127.0
    x[8] = 0.5
    x[8, ..., 0::32] = -8.0
    x[9] = -1.0
    x[9, ..., 3::32] = 1.0  # the largest magnitude with both signs: the first counts
    x[10] *= 1e-6
    x[11] *= 1e6
    x[12] = 65520.0
    x[13, ..., 1::2] = 0.0
    return x


def cache_of(ops, fmt, pages, page, heads, dim):
    size = ops.kv_page_bytes(fmt, page, heads, dim)
    return torch.full((pages, size), 255, dtype=torch.uint8, device=DEV)  # scales and fp16 values NaN


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("heads,dim,page,layout", [(1, 32, 16, "rows"), (3, 96, 48, "slice"), (2, 128, 32, "odd"),
                                                   (8, 64, 16, "heads first"), (1, 512, 64, "rows")])
def test_write_and_read(ops, fmt, kind, heads, dim, page, layout):
    rng = np.random.default_rng(heads * dim)
    n, pages = 37, 5
    k, v = random_kv(rng, n, heads, dim)
    e = edge_rows(heads, dim)
    k[:14], v[3:17] = e, e[::-1]
    kt, vt = (torch.from_numpy(x).to(DEV).to(TYPES[kind]) for x in (k, v))
    if layout == "slice":  # slices of one projection
        both = torch.cat([kt, torch.ones_like(kt), vt], 1)
        kt, vt = both[:, :heads], both[:, 2 * heads:]
    elif layout == "odd":  # rows that start on no 16-byte boundary
        pad = [torch.zeros((n, heads, dim + 1), dtype=x.dtype, device=DEV) for x in (kt, vt)]
        for p, x in zip(pad, (kt, vt)):
            p[..., 1:] = x
        kt, vt = pad[0][..., 1:], pad[1][..., 1:]
    elif layout == "heads first":
        kt, vt = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (kt, vt))
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    slots[[2, 20]] = -1
    slots[21] = pages * page  # one past the cache
    slots[22] = 1 << 40
    cache = cache_of(ops, fmt, pages, page, heads, dim)
    want = cache.cpu().numpy().copy()
    R.store(want, kt.float().cpu().numpy(), vt.float().cpu().numpy(), slots, fmt, page)
    st = torch.from_numpy(slots).to(DEV)
    ops.kv_write(cache, kt, vt, st, fmt, page)
    got = cache.cpu().numpy()
    if fmt == "f16":
        np.testing.assert_array_equal(got.view(np.float16), want.view(np.float16))  # any NaN is a NaN
    else:
        a, b = got.copy(), want.copy()
        nan = (a.reshape(-1, 2).view(np.uint16) & 0x7fff) > 0x7c00
        same = (a.reshape(-1, 2) == b.reshape(-1, 2)).all(1) | (nan[:, 0] & ((b.reshape(-1, 2).view(np.uint16)[:, 0] & 0x7fff) > 0x7c00))
        assert same.all(), np.flatnonzero(~same)[:10]
    gk, gv = ops.kv_read(cache, st, fmt, page, heads, dim, dtype=TYPES[kind])
    live = (slots >= 0) & (slots < pages * page)
    for x, g in ((kt, gk), (vt, gv)):
        code, scale = R.quantize(x.float().cpu().numpy(), fmt)
        with np.errstate(all="ignore"):
            w = R.dequantize(code, scale, fmt)
        w[~live] = 0
        w = torch.from_numpy(w).to(torch.float32).to(TYPES[kind])  # exact in fp32, rounded once
        np.testing.assert_array_equal(g.float().cpu().numpy(), w.float().numpy())
    # into given tensors with other strides
    buf = torch.zeros((n, heads + 1, 2 * dim), dtype=TYPES[kind], device=DEV)
    ops.kv_read(cache, st, fmt, page, heads, dim, k=buf[:, :heads, :dim], v=buf[:, :heads, dim:])
    assert torch.equal(torch.nan_to_num(buf[:, :heads, :dim]), torch.nan_to_num(gk)) and not bool(buf[:, heads].any())


def border_rows(fmt, kind, n, dim, seed):
    """Rows of blocks whose values lie on or next to where the code changes, for
    scales of every size that a type holds."""
    rng = np.random.default_rng(seed)
    blocks = n * dim // 32
    lo, hi = {"float32": (-120, 110), "float16": (-12, 14), "bfloat16": (-120, 110)}[kind]
    top = np.ldexp(1 + rng.random(blocks), rng.integers(lo, hi, blocks)).astype(np.float32)
    top[::7] = np.ldexp(1.0, rng.integers(lo, hi, top[::7].size))  # powers of two: exact halves
    top[3::11] = np.nextafter(2 * top[3::11], np.float32(0)) if kind == "float32" else top[3::11]  # mantissas near all ones
    steps = 127 if fmt == "q8_0" else 8
    at = rng.integers(-steps, steps, (blocks, 32)) + 0.5
    x = (top[:, None].astype(np.float64) * at / steps).astype(np.float32)
    off = rng.integers(-3, 4, x.shape)  # units of the last place
    bits = x.view(np.int32) + np.where(x != 0, off, 0).astype(np.int32)
    x = np.where(rng.random(x.shape) < 0.5, bits.view(np.float32), x)
    x[:, 0] = top
    x[::2, 0] *= -1
    x = torch.from_numpy(x.reshape(n, 1, dim)).to(TYPES[kind])
    return x


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("kind", TYPES)
def test_codes_next_to_a_border(ops, fmt, kind):
    n, dim, page = 16384, 128, 64
    k, v = (border_rows(fmt, kind, n, dim, seed) for seed in (1, 2))
    slots = torch.arange(n, device=DEV)
    cache = cache_of(ops, fmt, n // page, page, 1, dim)
    ops.kv_write(cache, k.to(DEV), v.to(DEV), slots, fmt, page)
    for x, g in zip((k, v), ops.kv_read(cache, slots, fmt, page, 1, dim)):
        with np.errstate(all="ignore"):
            want = R.dequantize(*R.quantize(x.float().numpy(), fmt), fmt).astype(np.float32)
        np.testing.assert_array_equal(g.cpu().numpy(), want)


def attention_case(ops, fmt, kind, lens, rows, heads, kv_heads, dim, page, window, seed=0, plant=None, spread=2.0,
                   spare_table=2):
    """(ops arguments, reference): a cache of randomly placed pages, its
    unwritten places 0xFF, one table row a sequence."""
    rng = np.random.default_rng(seed + dim + rows)
    need = [-(-max(0, n) // page) for n in lens]
    pages = sum(need) + 2
    order = rng.permutation(pages)
    cache = np.full((pages, R.page_bytes(fmt, page, kv_heads, dim)), 255, dtype=np.uint8)
    table = np.full((len(lens), max(need) + spare_table), -7, dtype=np.int32)
    kv, at = [], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        k, v = random_kv(rng, max(0, n), kv_heads, dim)
        if plant:
            plant(b, k, v)
        p = np.arange(max(0, n))
        R.store(cache, k, v, table[b, p // page].astype(np.int64) * page + p % page, fmt, page)
        with np.errstate(all="ignore"):
            kv.append([R.dequantize(*R.quantize(x, fmt), fmt) for x in (k, v)])
    q = torch.from_numpy((spread * rng.standard_normal((len(lens) * rows, heads, dim))).astype(np.float32))
    q = q.to(TYPES[kind])
    args = dict(q=q.to(DEV), cache=torch.from_numpy(cache).to(DEV), page_table=torch.from_numpy(table).to(DEV),
                kv_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), fmt=fmt, page_tokens=page,
                n_kv_heads=kv_heads, rows=rows, window=window)
    return args, q.double().numpy(), kv


def check_attention(ops, args, q, kv, lens, scale=None):
    rows, window = args["rows"], args["window"]
    kind = str(args["q"].dtype).replace("torch.", "")
    n, heads, dim = args["q"].shape
    lse = torch.full((n, heads), 7.0, device=DEV)
    out = ops.attn_paged(**args, lse=lse, scale=scale)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, length in enumerate(lens):
        r = slice(b * rows, (b + 1) * rows)
        want, wlse, mag, reach = R.attention(q[r], *kv[b], length, rows, window, dim ** -0.5 if scale is None else scale)
        tol, ltol = R.bounds(want, mag, reach, dim, max(length, 0), kind)
        err = np.abs(got[r] - want)
        assert np.isfinite(got[r]).all(), (b, length)
        assert (err <= tol).all(), (b, length, float((err / tol).max()))
        empty = np.isinf(wlse)
        assert (np.isneginf(glse[r]) == empty).all()
        assert (np.abs(np.where(empty, 0, glse[r] - np.where(empty, 0, wlse))) <= ltol).all()
        assert not got[r][empty].any()
    return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("lens,rows,heads,kv_heads,dim,page,window", [
    ([1], 1, 1, 1, 64, 16, 0),
    ([0, 5, 16, 17, 33], 1, 4, 4, 64, 16, 0),
    ([197], 1, 40, 8, 128, 16, 0),
    ([300, 0, 1, 47, 48, 49], 2, 6, 2, 96, 48, 0),
    ([70, 3, 6, 7], 6, 10, 2, 128, 32, 0),
    ([129, 16, 500], 17, 5, 1, 128, 64, 100),
    ([1000, 2, 640], 3, 8, 1, 256, 128, 33),
    ([2500], 6, 20, 4, 256, 16, 0),
    ([35, 36], 4, 9, 3, 64, 16, 1),
])
def test_attention(ops, fmt, kind, lens, rows, heads, kv_heads, dim, page, window):
    args, q, kv = attention_case(ops, fmt, kind, lens, rows, heads, kv_heads, dim, page, window)
    check_attention(ops, args, q, kv, lens)


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_long_sequences_are_split_and_joined(ops, kind):
    lens = [9001, 1, 4096]
    args, q, kv = attention_case(ops, "q8_0", kind, lens, 1, 4, 1, 128, 64, 0, spread=4.0)
    out = check_attention(ops, args, q, kv, lens)
    for _ in range(3):
        assert torch.equal(ops.attn_paged(**args), out)


@pytest.mark.parametrize("fmt,kind", [("q8_0", "float32"), ("q4_0", "float16"), ("f16", "bfloat16"), ("q8_0", "bfloat16")])
def test_more_rows_than_the_warps_of_a_cta_hold(ops, fmt, kind):
    lens = [300, 0, 77]
    args, q, kv = attention_case(ops, fmt, kind, lens, 17, 32, 2, 64, 16, 0)  # 272 rows a kv head
    check_attention(ops, args, q, kv, lens)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page,window", [(48, 0), (48, 130), (16, 300), (1024, 33), (80, 640)])
def test_pages_and_windows_that_cut_pairs_of_tiles(ops, fmt, page, window):
    lens = [1333, 15, 16, 17, 31, 32, 33, 47, 48, 49, 641]
    args, q, kv = attention_case(ops, fmt, "float32", lens, 2, 6, 2, 96, page, window)
    check_attention(ops, args, q, kv, lens)


def test_one_kv_head_over_all_splits(ops):
    lens = [40000]
    args, q, kv = attention_case(ops, "q4_0", "float32", lens, 1, 3, 1, 64, 32, 0, spread=5.0)
    out = check_attention(ops, args, q, kv, lens)
    for _ in range(3):
        assert torch.equal(ops.attn_paged(**args), out)


def test_the_workspace_may_hold_anything(ops):
    lens = [500, 3, 90]
    args, q, kv = attention_case(ops, "q8_0", "float32", lens, 2, 4, 2, 64, 16, 0)
    want = ops.attn_paged(**args)
    ws = torch.full((ops.attn_paged_workspace_bytes(torch.float32, 2, 4, 2, 64),), 255, dtype=torch.uint8, device=DEV)
    for fill in (255, 127, 1, 0):
        ws.fill_(fill)
        assert torch.equal(ops.attn_paged(**args, ws=ws), want)


def test_many_short_sequences(ops):
    lens = [int(n) for n in np.random.default_rng(3).integers(0, 40, 300)]
    args, q, kv = attention_case(ops, "q4_0", "float16", lens, 2, 4, 2, 64, 16, 0)
    check_attention(ops, args, q, kv, lens)


@pytest.mark.parametrize("fmt", FMTS)
def test_scale_and_sharp_scores(ops, fmt):
    lens = [777]
    args, q, kv = attention_case(ops, fmt, "float32", lens, 2, 4, 2, 128, 16, 0, spread=30.0)
    check_attention(ops, args, q, kv, lens)
    check_attention(ops, args, q, kv, lens, scale=-0.01)
    check_attention(ops, args, q, kv, lens, scale=0.0)


def test_scales_far_apart(ops):
    # blocks whose scales differ by many powers of two, growing along the cache
    def plant(b, k, v):
        v *= (2.0 ** np.linspace(-20, 12, v.shape[0], dtype=np.float32))[:, None, None]
        k[:, :, 32:64] *= 1e-4

    for fmt in FMTS:
        args, q, kv = attention_case(ops, fmt, "float32", [401], 2, 4, 2, 128, 16, 0, plant=plant)
        check_attention(ops, args, q, kv, [401])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_masked_places_never_reach_a_row(ops, fmt, value):
    # the newest token is bad: only the last row sees it; and the oldest one:
    # only the rows whose window reaches it do
    lens, rows, window = [50, 23], 3, 21

    def plant(b, k, v):
        for x in (k, v):
            x[-1] = value
            x[lens[b] - rows + 1 - window] = value  # position begin(0): row 0 alone sees it

    args, q, kv = attention_case(ops, fmt, "float32", lens, rows, 4, 2, 64, 16, window, plant=plant)
    out = ops.attn_paged(**args).cpu().numpy().reshape(2, rows, 4, 64)
    for b, n in enumerate(lens):
        want, _, mag, reach = R.attention(q[b * rows:(b + 1) * rows], *kv[b], n, rows, window, 0.125)
        tol, _ = R.bounds(want, mag, 50.0, 64, n, "float32")
        assert np.isnan(out[b, [0, 2]]).all()
        assert (np.abs(out[b, 1] - want[1]) <= tol[1]).all()


def test_infinite_values_of_one_row_only(ops):
    # fp16 values of infinity in V alone: where seen, the output is infinite as the formula has it
    def plant(b, k, v):
        v[-1, :, 7] = np.inf
        v[-2, :, 9] = -np.inf

    for kind in ("float32", "bfloat16"):
        args, q, kv = attention_case(ops, "f16", kind, [20], 2, 4, 2, 64, 16, 0, plant=plant)
        out = ops.attn_paged(**args).float().cpu().numpy()
        assert np.isposinf(out[1, :, 7]).all() and np.isfinite(out[0, :, 7]).all()
        assert np.isneginf(out[:, :, 9]).all()
        other = [d for d in range(64) if d not in (7, 9)]
        assert np.isfinite(out[:, :, other]).all()


def test_bad_pages_and_lengths_give_nan_and_nothing_else(ops):
    # every address comes from the checked tile_offset (tests/test_kvcache_host.py)
    lens = [40, 40, 40, 40]
    args, q, kv = attention_case(ops, "q8_0", "float32", lens, 2, 4, 2, 64, 16, 0, spare_table=0)
    good = ops.attn_paged(**args)
    pages = args["cache"].shape[0]
    args["page_table"][1, 1] = -1
    args["page_table"][2, 2] = pages
    args["kv_lens"][3] = 49  # three pages of 16 hold 48
    out = ops.attn_paged(**args)
    assert torch.equal(out[:2], good[:2]) and bool(torch.isnan(out[2:]).all())
    args["kv_lens"][:] = torch.tensor([-(1 << 31), (1 << 31) - 1, -1, 0], dtype=torch.int32)
    out = ops.attn_paged(**args)
    assert bool(torch.isnan(out[2:4]).all()) and not bool(out[[0, 1, 4, 5, 6, 7]].any())


@pytest.mark.parametrize("kind", TYPES)
def test_strides_and_orders(ops, kind):
    lens = [100, 37]
    args, q, kv = attention_case(ops, "q8_0", kind, lens, 3, 10, 2, 128, 16, 0)
    want = ops.attn_paged(**args)
    wide = torch.zeros((6, 14, 128 + 1), dtype=args["q"].dtype, device=DEV)
    for part in (wide[:, 2:12, :128], wide[:, 2:12, 1:], wide.transpose(0, 1)[2:12, :, :128].transpose(0, 1)):
        part.copy_(args["q"])
        out = torch.zeros_like(wide)
        ops.attn_paged(**{**args, "q": part}, out=out[:, 1:11, 1:])
        assert torch.equal(out[:, 1:11, 1:], want)
        out[:, 1:11, 1:] = 0
        assert not bool(out.any())
    heads_first = args["q"].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(ops.attn_paged(**{**args, "q": heads_first}), want)
    table = torch.full((2, 50), -1, dtype=torch.int32, device=DEV)
    table[:, :args["page_table"].shape[1]] = args["page_table"]
    assert torch.equal(ops.attn_paged(**{**args, "page_table": table}), want)


def test_offsets_past_32_bits(ops):
    page, heads, dim = 64, 8, 128
    size = ops.kv_page_bytes("q8_0", page, heads, dim)
    pages = (9 << 29) // size + 3  # above 4.5 GB
    cache = torch.empty((pages, size), dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(1)
    k, v = random_kv(rng, 130, heads, dim)
    p = np.arange(130)
    table = np.array([pages - 1, 0, pages - 2], dtype=np.int64)
    slots = torch.from_numpy(table[p // page] * page + p % page).to(DEV)
    ops.kv_write(cache, torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), slots, "q8_0", page)
    kv = [R.dequantize(*R.quantize(x, "q8_0"), "q8_0") for x in (k, v)]
    gk, gv = ops.kv_read(cache, slots, "q8_0", page, heads, dim)
    assert np.array_equal(gk.cpu().numpy(), kv[0].astype(np.float32))
    assert np.array_equal(gv.cpu().numpy(), kv[1].astype(np.float32))
    q = torch.randn((1, 16, dim), device=DEV)
    args = dict(q=q, cache=cache, page_table=torch.from_numpy(table).to(DEV).int()[None], fmt="q8_0", page_tokens=page,
                kv_lens=torch.tensor([130], dtype=torch.int32, device=DEV), n_kv_heads=heads, rows=1, window=0)
    check_attention(ops, args, q.double().cpu().numpy(), [kv], [130])


@pytest.mark.parametrize("short_way", [True, False])
def test_threads_on_one_stream(ops, short_way, monkeypatch):
    # the two kernels of a call and the workspace between them, with calls of other threads
    import threading

    if not short_way:
        monkeypatch.setattr(ops._CALLS, "attn_paged", lambda *a: None)
    cases = [attention_case(ops, "q8_0", "float32", [900 + 100 * i, 30], 2, 8, 2, 64, 16, 0, seed=i)[0] for i in range(4)]
    wants = [ops.attn_paged(**c) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        for _ in range(100):
            if not torch.equal(ops.attn_paged(**cases[i]), wants[i]):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_the_short_way_and_ctypes_agree(ops, monkeypatch):
    args, q, kv = attention_case(ops, "q4_0", "bfloat16", [100, 37], 3, 10, 2, 128, 16, 20)
    cache, slots = args["cache"].clone(), torch.arange(40, device=DEV)
    rows = torch.randn((40, 2, 128), device=DEV).bfloat16()

    def both():
        c = cache.clone()
        ops.kv_write(c, rows, rows, slots, "q4_0", 16)
        return (c, *ops.kv_read(c, slots, "q4_0", 16, 2, 128, dtype=torch.float16), ops.attn_paged(**args, scale=0.1))

    first = both()
    for name in ("kv_write", "kv_read", "attn_paged"):
        monkeypatch.setattr(ops._CALLS, name, lambda *a: None)
    for a, b in zip(first, both()):
        assert a.dtype == b.dtype and a.shape == b.shape
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


def test_another_stream_and_a_graph(ops):
    lens = [333, 20]
    args, q, kv = attention_case(ops, "q4_0", "float16", lens, 2, 8, 2, 128, 32, 0)
    want = ops.attn_paged(**args)
    n, heads = 4, 2
    rows = torch.randn((n, heads, 128), device=DEV).half()
    slots = torch.arange(n, device=DEV)
    scratch = cache_of(ops, "q4_0", 1, 32, heads, 128)
    ops.kv_write(scratch, rows, rows, slots, "q4_0", 32)
    want_kv = ops.kv_read(scratch, slots, "q4_0", 32, heads, 128)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = ops.attn_paged(**args)
    s.synchronize()
    assert torch.equal(other, want)
    g = torch.cuda.CUDAGraph()
    scratch.fill_(255)
    with torch.cuda.graph(g):
        ops.kv_write(scratch, rows, rows, slots, "q4_0", 32)
        got_kv = ops.kv_read(scratch, slots, "q4_0", 32, heads, 128)
        out = ops.attn_paged(**args)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(got_kv, want_kv))
    args["kv_lens"][:] = torch.tensor([1, 300], dtype=torch.int32)  # new lengths, the same graph
    args["page_table"][1] = args["page_table"][0]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ops.attn_paged(**args))
