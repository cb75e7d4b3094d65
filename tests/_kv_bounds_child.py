"""Child process of test_gpu_kv_bounds (run with QGEMV_BOUNDS_CHECK=1, so that
the binding loads the bounds-checking library): the paged cache's calls on
ragged, odd and refused-slot cases, each followed by a read of the bounds
records.  Prints one JSON line.  Test code only."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from block_quantized_gemv_quantize_gb300 import ops  # noqa: E402
from tests import test_gpu_kvcache as T  # noqa: E402


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

    for fmt in T.FMTS:
        for kind in T.TYPES:
            case(T.test_write_and_read, fmt, kind, 3, 96, 48, "slice")
            case(T.test_write_and_read, fmt, kind, 2, 128, 32, "odd")
            case(T.test_attention, fmt, kind, [300, 0, 1, 47, 48, 49], 2, 6, 2, 96, 48, 0)
            case(T.test_attention, fmt, kind, [1000, 2, 640], 3, 8, 1, 256, 128, 33)
            case(T.test_attention, fmt, kind, [35, 36], 4, 9, 3, 64, 16, 1)
        case(T.test_pages_and_windows_that_cut_pairs_of_tiles, fmt, 48, 130)
    case(T.test_more_rows_than_the_warps_of_a_cta_hold, "q4_0", "float16")
    case(T.test_bad_pages_and_lengths_give_nan_and_nothing_else)
    case(T.test_many_short_sequences)
    res["timeouts"] = ops.qgemv_take_wait_timeouts()
    print(json.dumps(res))


if __name__ == "__main__":
    main()
