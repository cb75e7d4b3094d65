"""Infinities and NaN in the paged cache and in q: what the attention's formula
makes of them, wherever in the sequence they stand and however many rows share a
kv head.  f16 caches hold infinities (kv_write's rounding of values past 65504
among them); a key of which a row's score is minus infinity has no weight in it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from . import _kv_ref as R  # noqa: E402
from .test_gpu_kvcache import FMTS, attention_case, ops  # noqa: E402, F401

LENGTH = 700
ROWS = [(2, 4, 2), (6, 4, 2), (17, 10, 2)]  # rows, heads, kv heads: 4, 12 and 85 rows a kv head
KINDS = ["float32", "float16", "bfloat16"]


def reference(args, q, kv, finite):
    """(want, tolerance) of one sequence; `finite`: the keys and values with the
    infinities as zeros, for the sizes that the tolerance goes by."""
    rows, n = args["rows"], q.shape[0]
    dim, kind = q.shape[2], str(args["q"].dtype).replace("torch.", "")
    with np.errstate(all="ignore"):
        want = R.attention(q, *kv, LENGTH, rows, 0, dim ** -0.5)[0]
    _, _, mag, reach = R.attention(q, *finite, LENGTH, rows, 0, dim ** -0.5)
    return want, R.bounds(np.where(np.isfinite(want), want, 0), mag, reach, dim, LENGTH, kind)[0]


def same(got, want, tol):
    """Infinities and NaN in the same places, the rest within the tolerance."""
    assert (np.isnan(got) == np.isnan(want)).all()
    assert (np.isposinf(got) == np.isposinf(want)).all() and (np.isneginf(got) == np.isneginf(want)).all()
    fine = np.isfinite(want)
    assert (np.abs(got - want)[fine] <= tol[fine]).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,heads,kv_heads", ROWS)
@pytest.mark.parametrize("at", [1, 300, 520, LENGTH - 1])
def test_infinite_values(ops, kind, rows, heads, kv_heads, at):  # noqa: F811
    def plant(b, k, v):
        v[at, :, 7] = np.inf
        v[at - 1, :, 9] = -np.inf
        v[at, :, 11], v[at - 1, :, 11] = np.inf, -np.inf

    args, q, kv = attention_case(ops, "f16", kind, [LENGTH], rows, heads, kv_heads, 64, 16, 0, plant=plant, spread=1.0)
    (k, v), = kv
    got = ops.attn_paged(**args).double().cpu().numpy()
    same(got, *reference(args, q, (k, v), (k, np.where(np.isfinite(v), v, 0))))
    if at != LENGTH - 1:
        assert np.isposinf(got[:, :, 7]).all() and np.isneginf(got[:, :, 9]).all() and np.isnan(got[:, :, 11]).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,heads,kv_heads", ROWS)
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("at", [0, 300, LENGTH - 1])
def test_infinite_keys(ops, kind, rows, heads, kv_heads, dim, at):  # noqa: F811
    # heads with a positive q there have a score of minus infinity, of no weight;
    # the others one of plus infinity, and no softmax
    def plant(b, k, v):
        k[at, :, 5] = -np.inf

    args, q, kv = attention_case(ops, "f16", kind, [LENGTH], rows, heads, kv_heads, dim, 32, 0, plant=plant, spread=1.0)
    q[:, :, 5] = np.where(np.arange(heads) % 4 < 3, 1.0, -1.0) * (np.abs(q[:, :, 5]) + 0.25)
    args["q"] = torch.from_numpy(q).to(args["q"])
    q = args["q"].double().cpu().numpy()
    (k, v), = kv
    got = ops.attn_paged(**args).double().cpu().numpy()
    want, tol = reference(args, q, (k, v), (np.where(np.isfinite(k), k, 0), v))
    same(got, want, tol)
    if at < LENGTH - rows:  # (rows before the newest one do not see that)
        assert np.isfinite(got[:, :3]).all() and np.isnan(got[:, 3]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,heads,kv_heads", ROWS)
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_a_row_of_q_that_is_not_finite_is_nan_and_no_other(ops, fmt, kind, rows, heads, kv_heads, value):  # noqa: F811
    args, q, kv = attention_case(ops, fmt, kind, [LENGTH], rows, heads, kv_heads, 64, 16, 0)
    want, tol = reference(args, q, kv[0], kv[0])
    args["q"][rows - 2, 1, 33] = value
    lse = torch.zeros(want.shape[:2], device=args["q"].device)
    got = ops.attn_paged(**args, lse=lse).double().cpu().numpy()
    want[rows - 2, 1] = np.nan
    same(got, want, tol)
    assert bool(torch.isnan(lse[rows - 2, 1])) and int(torch.isnan(lse).sum()) == 1
