// Row tiles of the experts' products with many rows (plain arithmetic, for host compilers too).
#pragma once

#ifdef __CUDACC__
#define MX_BOTH __host__ __device__ __forceinline__
#else
#define MX_BOTH inline
#endif

namespace qgemv {

// N of a tcgen05.mma: the PTX ISA's shapes of kind::f16 over a pair of SMs (cta_group::2)
// with M = 256 are N = 32, 64 .. 256.
constexpr int MXT_N_STEP = 32;

MX_BOTH int mxt_round_n(int rows) { return (rows + MXT_N_STEP - 1) / MXT_N_STEP * MXT_N_STEP; }

// Row tile i of an expert's `all` rows in `tiles` of even size, at most `most` rows each (a
// multiple of the step): its first row, its rows, the product's N.
struct MxRowTile {
    int first, cnt, n;
};
MX_BOTH MxRowTile mxt_row_tile(int all, int tiles, int i, int most)
{
    int each = mxt_round_n((all + tiles - 1) / tiles);
    if (each > most) each = most;
    MxRowTile t;
    t.first = i * each;
    t.cnt = all - t.first < each ? all - t.first : each;
    t.n = mxt_round_n(t.cnt);
    return t;
}

}  // namespace qgemv
