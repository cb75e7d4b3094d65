"""bf16 rows of the attention over the paged cache lose nothing but the one
rounding of the output: it is the rounding of a number within the fp32 rows'
bounds of the 64-bit result, which for most elements leaves one value."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from . import _kv_ref as R  # noqa: E402
from .test_gpu_kvcache import FMTS, attention_case, ops  # noqa: E402, F401


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,rows,heads,kv_heads,dim", [([7, 9, 33], 1, 40, 8, 128), ([7, 9, 33], 2, 32, 8, 64),
                                                          ([9, 33], 6, 10, 2, 128), ([21, 40], 17, 5, 1, 256)])
def test_one_rounding(ops, fmt, lens, rows, heads, kv_heads, dim):  # noqa: F811
    # flat scores over few tokens, values about 3: the bounds are far below a step
    # of the type, and roundings of the weights to fewer bits do not average out
    def plant(b, k, v):
        v += 3

    args, q, kv = attention_case(ops, fmt, "bfloat16", lens, rows, heads, kv_heads, dim, 16, 0, plant=plant, spread=0.1)
    got = ops.attn_paged(**args).double().cpu().numpy()
    for b, length in enumerate(lens):
        r = slice(b * rows, (b + 1) * rows)
        want, _, mag, reach = R.attention(q[r], *kv[b], length, rows, 0, dim ** -0.5)
        # the rows' own arithmetic: the fp32 bound without its rounding of the output
        tol = R.bounds(want, mag, reach, dim, length, "float32")[0] - np.abs(want) * R.HALF_STEP["float32"]
        lo, hi = (torch.from_numpy(x).bfloat16().double().numpy() for x in (want - tol, want + tol))
        assert ((lo <= got[r]) & (got[r] <= hi)).all(), int(((got[r] < lo) | (got[r] > hi)).sum())
        assert (lo == hi).mean() > 0.9  # (the test says something)
