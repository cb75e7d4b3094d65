"""The attention over the paged cache where V's scales differ widely: between the
blocks of a token, between tokens of much and of little weight, and between tokens
that a row sees and those that it does not.  Every row and block of 32 channels
stays within the bounds of its own arithmetic (tests/_kv_ref.py and one term more),
which know nothing of the other scales."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from . import _kv_ref as R  # noqa: E402
from .test_gpu_kvcache import FMTS, attention_case, ops  # noqa: E402, F401

SHAPES = [(3, 4, 2, 64), (3, 8, 1, 96), (2, 4, 2, 128), (6, 8, 2, 128), (3, 8, 1, 256), (17, 4, 1, 256)]
HUGE = {"q8_0": 6e6, "q4_0": 4e5, "f16": 6e4}  # scales of about 47000 and 50000, or the largest values


def largest_products(q, k, v, length, rows):
    """Of each row, head and block: the largest weight times the block's largest value."""
    heads, dim = q.shape[1:]
    out = np.zeros(q.shape)
    for i in range(rows):
        end = length - (rows - 1 - i)
        for h in range(heads if end > 0 else 0):
            kv_head = h * k.shape[1] // heads
            s = k[:end, kv_head] @ q[i, h] * dim ** -0.5
            p = np.exp(s - s.max())
            most = np.abs(v[:end, kv_head]).reshape(end, dim // 32, 32).max(-1)
            out[i, h] = np.repeat((p[:, None] * most).max(0) / p.sum(), 32)
    return out


def check(ops, args, q, kv, lens):  # noqa: F811
    """Within the bounds of tests/_kv_ref.py, and for every token 2^-26 of the
    largest product of the row and block: scales as far apart as here (2^20 and more)
    have their products rounded to less."""
    rows, dim = args["rows"], q.shape[2]
    kind = str(args["q"].dtype).replace("torch.", "")
    got = ops.attn_paged(**args).double().cpu().numpy()
    for b, length in enumerate(lens):
        r = slice(b * rows, (b + 1) * rows)
        want, _, mag, reach = R.attention(q[r], *kv[b], length, rows, 0, dim ** -0.5)
        tol = R.bounds(want, mag, reach, dim, length, kind)[0]
        tol = tol + length * 2.0 ** -26 * largest_products(q[r], *kv[b], length, rows)
        assert np.isfinite(got[r]).all()
        err = np.abs(got[r] - want)
        assert (err <= tol).all(), (b, length, float((err / tol).max()))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("rows,heads,kv_heads,dim", SHAPES)
def test_a_huge_value_that_earlier_rows_do_not_see(ops, fmt, kind, rows, heads, kv_heads, dim):  # noqa: F811
    def plant(b, k, v):
        v *= 2.0 ** -8
        v[-1] *= (6e4 if kind == "float16" else HUGE[fmt]) / np.abs(v[-1]).max()

    lens = [50, 333]
    args, q, kv = attention_case(ops, fmt, kind, lens, rows, heads, kv_heads, dim, 16, 0, plant=plant, spread=0.7)
    check(ops, args, q, kv, lens)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,heads,kv_heads,dim", SHAPES)
def test_blocks_of_a_token_far_apart(ops, fmt, rows, heads, kv_heads, dim):  # noqa: F811
    def plant(b, k, v):
        for n in range(dim // 32):
            v[..., 32 * n:32 * n + 32] *= (2.0 ** 12, 2.0 ** -12, 1.0)[n % 3]

    args, q, kv = attention_case(ops, fmt, "float32", [401], rows, heads, kv_heads, dim, 16, 0, plant=plant, spread=0.7)
    check(ops, args, q, kv, [401])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("at", [0, 150, 299])
@pytest.mark.parametrize("rows,heads,kv_heads,dim", SHAPES)
def test_a_huge_value_of_no_weight(ops, fmt, at, rows, heads, kv_heads, dim):  # noqa: F811
    # scores of about -70 at that token (a weight of 1e-30), 0 +- 1 elsewhere
    def plant(b, k, v):
        k *= 0.1
        k[at] = -70.0 / (0.56 * np.sqrt(dim))
        v *= 2.0 ** -8
        v[at] *= HUGE[fmt] / np.abs(v[at]).max()

    args, q, kv = attention_case(ops, fmt, "float32", [300], rows, heads, kv_heads, dim, 32, 0, plant=plant, spread=0.7)
    args["q"] = args["q"].abs()
    check(ops, args, np.abs(q), kv, [300])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("rows,heads,kv_heads,dim", SHAPES)
def test_scores_that_rise_while_values_fall(ops, fmt, rising, rows, heads, kv_heads, dim):  # noqa: F811
    # scores from 0 to 60 along the cache, values from 2^10 to 2^-14; or the other way round
    def plant(b, k, v):
        x = np.linspace(0, 1, k.shape[0], dtype=np.float32)[:, None, None]
        x = x if rising else x[::-1]
        k *= 0.1
        k += 60.0 / (0.56 * np.sqrt(dim)) * x
        v *= 2.0 ** (10 - 24 * x)

    args, q, kv = attention_case(ops, fmt, "float32", [500], rows, heads, kv_heads, dim, 48, 0, plant=plant, spread=0.7)
    args["q"] = args["q"].abs()
    check(ops, args, np.abs(q), kv, [500])


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("at", [0, 150, 299])
@pytest.mark.parametrize("rows,heads,kv_heads,dim", SHAPES)
def test_all_weight_on_a_token_of_zeros(ops, fmt, at, rows, heads, kv_heads, dim):  # noqa: F811
    # a score of about 20 at a token whose values are zero: the others' weights, of
    # 1e-9, are all that the output has.  (An f16 cache, which has no scales, keeps
    # weights to 2^-36 of the row's largest.)
    def plant(b, k, v):
        k *= 0.1
        k[at] = 20.0 / (0.56 * np.sqrt(dim))
        v[at] = 0

    args, q, kv = attention_case(ops, fmt, "float32", [300], rows, heads, kv_heads, dim, 32, 0, plant=plant, spread=0.7)
    args["q"] = args["q"].abs()
    check(ops, args, np.abs(q), kv, [300])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_values_of_zero(ops, fmt, kind):  # noqa: F811
    def plant(b, k, v):
        v[:] = 0

    args, q, kv = attention_case(ops, fmt, kind, [333, 1], 3, 4, 2, 128, 16, 0, plant=plant)
    assert not bool(ops.attn_paged(**args).any())
