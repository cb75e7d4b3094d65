// attn_paged: the workspace's size and the choice of the kernel (one
// translation unit a cache format).
#include "attn_paged.cuh"

namespace qgemv {

// Counters, then two partial results for every CTA: at most one item that
// began before the CTA's piece and one that goes on after it.
size_t attn_workspace_bytes(int type, int rows, int heads, int kv_heads, int head_dim)
{
    const bool two = type != QGEMV_BF16;
    const int per_tile = two ? 8 : 16, most = AttnShape<QGEMV_KV_F16, 2, true>::MAX_WARPS;
    const int tiles = (rows * (heads / kv_heads) + per_tile - 1) / per_tile;
    const int groups = (tiles + most - 1) / most, wr = (tiles + groups - 1) / groups;
    const size_t part = (size_t)((head_dim / QK) * 4 * (two ? 2 : 4) + 2 * (two ? 1 : 2)) * 32 * sizeof(float);
    return ATTN_COUNTER_BYTES + (size_t)2 * ATTN_GRID * wr * part;
}

int launch_attn_paged(int fmt, int type, const AttnArgs& a, cudaStream_t s)
{
    if (fmt == QGEMV_KV_F16) return launch_attn_f16(type, a, s);
    if (fmt == QGEMV_KV_Q8_0) return launch_attn_q8_0(type, a, s);
    return launch_attn_q4_0(type, a, s);
}

}  // namespace qgemv
