"""Infinities and NaN in the paged cache: what the attention's formula makes of
them, wherever in the sequence they stand and however many rows share a kv head.
f16 caches hold infinities (kv_write's rounding of values past 65504 among them)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from . import _kv_ref as R  # noqa: E402
from .test_gpu_kvcache import attention_case, ops  # noqa: E402, F401

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
