"""The paged cache's kernels in the bounds-checking build (compiled with
-DQGEMV_BOUNDS_CHECK): right results and no failed index check, in a child
process, since the binding picks the library when it is imported."""
import json
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_paged_cache_stays_in_bounds():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_gemv_quantize_gb300 import build

    build.build(debug=True)
    env = dict(os.environ, QGEMV_BOUNDS_CHECK="1")
    p = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "_kv_bounds_child.py")], env=env, cwd=ROOT,
                       capture_output=True, text=True, timeout=1200)
    assert p.returncode == 0, p.stderr[-3000:]
    res = json.loads(p.stdout.strip().splitlines()[-1])
    assert res["bounds_build"] is True
    assert res["fail"] == [], res["fail"]
    assert res["cases"] >= 50 and res["timeouts"] == 0
