"""The sparse layer's example runs from its graph and agrees with a dense layer."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# Of the largest output: fp32 sums of 1024 and 352 products carry some 2^-20;
# 16-bit types round the inner rows and the outputs, by half a step each, and
# 352 rounded inner values add up to no more than a few such steps.
@pytest.mark.parametrize("kind,tokens,bound", [("float32", 6, 2.0 ** -17), ("float32", 150, 2.0 ** -17),
                                               ("float16", 6, 2.0 ** -9), ("bfloat16", 150, 2.0 ** -6)])
def test_the_example_agrees_with_a_dense_layer(kind, tokens, bound):
    spec = importlib.util.spec_from_file_location("sparse_layer", os.path.join(ROOT, "examples", "sparse_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.run(getattr(torch, kind), steps=2, tokens=tokens) <= bound
