"""Stores of the sparse layer's kernels whose place is computed from data have a check in the
bounds-checking build.  No GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_gemv_quantize_gb300", "csrc")
STORES = {
    "moe_route.cu": r"\ba\.(?:ids|weights|order|counts)\[.*\] = |\bcounts\[.*\] = ",
    "mx_gemm.cuh": r"\ba\.place_of\[.*\] = ",
    "mx_gemm_tc.cuh": r"\ba\.place_of\[.*\] = ",
}


def test_every_such_store_is_checked():
    for name, store in STORES.items():
        lines = open(os.path.join(CSRC, name)).read().split("\n")
        at = [i for i, line in enumerate(lines) if re.search(store, line)]
        assert at, name
        for i in at:  # (the check stands on the line, or opens the statement or block that the store is in)
            assert any("QG_OK(" in line for line in lines[max(0, i - 2):i + 1]), f"{name}:{i + 1}: {lines[i].strip()}"


def test_sites_are_numbered_apart():
    seen = {}
    for name in sorted(os.listdir(CSRC)):
        for site in re.findall(r"QG_OK\([^;{]*?(?:status|a\.status),\s*(\d+)\)", open(os.path.join(CSRC, name)).read(), re.S):
            if int(site) >= 300:
                assert site not in seen, f"{site}: {name}, {seen.get(site)}"
                seen[site] = name
    assert len(seen) >= 15
