"""Child process of test_gpu_sparse_bounds (run with QGEMV_BOUNDS_CHECK=1, so that
the binding loads the bounds-checking library): the router and its sorting by one CTA and by many,
products with odd orders and scales, each followed by a read of the bounds records.
Prints one JSON line.  Test code only."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from block_quantized_gemv_quantize_gb300 import ops  # noqa: E402
from tests import test_gpu_mx_scales as S  # noqa: E402
from tests import test_gpu_mx_small_rows as X  # noqa: E402
from tests import test_gpu_mx_unnamed_slots as U  # noqa: E402
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

    # (tokens: one CTA up to 64, ranges of one round of warps up to 16384, of two beyond)
    for tokens in (1, 63, 64, 65, 16384, 16385):
        for experts, top_k in ((1, 1), (33, 32), (1024, 3)):
            case(T.test_group, tokens, top_k, experts)
    for kind in T.TYPES:
        for tokens, experts, top_k in ((1, 1, 1), (64, 1000, 32), (65, 64, 6), (700, 1024, 32), (2049, 1, 1)):
            case(T.test_route, kind, tokens, experts, top_k, "softmax", True, 1.0)
            case(T.test_route, kind, tokens, experts, top_k, "sigmoid", False, 2.0)
        case(U.test_down, kind, 7, 3, 6, 2)
        case(U.test_down, kind, 300, 2, 5, 7)
        case(S.test_a_block_at_every_distance, kind, 3, 160, 20)
        case(S.test_a_block_at_every_distance, kind, 40, 1056, 33)
    for kind in ("float32", "bfloat16"):
        case(X.test_products_of_small_rows, kind, 7, 256, 205)
        case(X.test_products_of_small_rows, kind, 96, 1056, 225)
    case(T.test_route_rows_with_strides)
    case(T.test_route_masks_ties_and_nan, "softmax", 900)
    case(T.test_no_tokens)
    res["timeouts"] = ops.qgemv_take_wait_timeouts()
    print(json.dumps(res))


if __name__ == "__main__":
    main()
