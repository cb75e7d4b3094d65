"""The row tiles of the experts' products with many rows, by the kernel's own arithmetic
compiled for the host: N of a tcgen05.mma over a pair of SMs with M = 256 goes in
steps of 32 (kind::f16), every row is in one tile, and no tile is empty.  No GPU."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_gemv_quantize_gb300", "csrc")

MAIN = r"""
#include <cstdio>
#include <initializer_list>
#include "mx_row_tile.cuh"
int main()
{
    for (int most : {96, 160})
        for (int all = 1; all <= 20000; ++all) {
            const int tiles = (all + most - 1) / most;
            int next = 0;
            for (int i = 0; i < tiles; ++i) {
                const qgemv::MxRowTile t = qgemv::mxt_row_tile(all, tiles, i, most);
                if (t.first != next || t.cnt < 1 || t.n < t.cnt || t.n % 32 || t.n < 32 || t.n > most) {
                    std::printf("most %d, %d rows, tile %d: first %d, cnt %d, n %d\n", most, all, i, t.first, t.cnt, t.n);
                    return 1;
                }
                next += t.cnt;
            }
            if (next != all) {
                std::printf("most %d: %d rows of %d\n", most, next, all);
                return 1;
            }
        }
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("row_tiles")
    (at / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-x", "c++", str(at / "main.cpp"), "-o", str(at / "main")], check=True)
    return str(at / "main")


def test_row_tiles(program):
    r = subprocess.run([program], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_the_kernel_takes_these_tiles():
    src = open(os.path.join(CSRC, "mx_gemm_tc.cuh")).read()
    assert "mxt_row_tile(" in src and "tc_idesc(__shfl_sync(~0u, walk.n, 0))" in src
