"""Child process of test_gpu_mx_bounds (run with QGEMV_BOUNDS_CHECK=1, so that
the binding loads the bounds-checking library): the MXFP4 and sparse-layer
calls on ragged and odd cases, each followed by a read of the bounds records.
Prints one JSON line.  Test code only."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from block_quantized_gemv_quantize_gb300 import ops  # noqa: E402
from tests import test_gpu_mxfp4 as T  # noqa: E402


def main():
    res = {"bounds_build": ops.qgemv_bounds_check_build(), "cases": 0, "fail": []}
    ops.qgemv_take_bounds_errors()

    def case(f, *args):
        f(ops, *args)
        T.torch.cuda.synchronize()
        count, site = ops.qgemv_take_bounds_errors()
        res["cases"] += 1
        if count:
            res["fail"].append([f.__name__, str(args), count, site])

    for kind in T.TYPES:
        case(T.test_quantize_and_back, kind, 7, 1056, 8)
        case(T.test_quantize_and_back, kind, 33, 64, 3)
        for shape in T.SHAPES:
            case(T.test_gemm, kind, shape)
            case(T.test_gate_up, kind, shape)
            case(T.test_down, kind, shape)
        for tokens in (5, 200):
            case(T.test_rows_with_strides_and_given_outputs, kind, 1, tokens)
        case(T.test_sorted_rows_without_an_order, kind, [8, 9, 16, 17, 127, 128, 129, 0])
    case(T.test_offsets_and_order_that_do_not_fit_touch_nothing_else)
    res["timeouts"] = ops.qgemv_take_wait_timeouts()
    print(json.dumps(res))


if __name__ == "__main__":
    main()
