// attn_paged: the workspace's size and the choice of the kernel (one
// translation unit a cache format).
#include "attn_paged.cuh"

namespace qgemv {

// Counters, then two partial results for every split and for every CTA: at
// most one item that began before its piece and one that goes on after it.
size_t attn_workspace_bytes(int type, int rows, int heads, int kv_heads, int head_dim)
{
    const int n = rows * (heads / kv_heads), nb = head_dim / QK, mode = attn_mode(type, n);
    const int per_tile = mode == ATTN_PAIR ? 8 : 16, most = attn_warps(nb);
    const int tiles = (n + per_tile - 1) / per_tile, groups = (tiles + most - 1) / most, wr = (tiles + groups - 1) / groups;
    const size_t part = (size_t)(nb * 4 * (per_tile / 4) + 2 * (per_tile / 8)) * 32 * sizeof(float);
    return ATTN_COUNTER_BYTES + (size_t)2 * ATTN_GRID * (most / wr + 1) * wr * part;
}

int launch_attn_paged(int fmt, int type, const AttnArgs& a, cudaStream_t s)
{
    if (fmt == QGEMV_KV_F16) return launch_attn_f16(type, a, s);
    if (fmt == QGEMV_KV_Q8_0) return launch_attn_q8_0(type, a, s);
    return launch_attn_q4_0(type, a, s);
}

}  // namespace qgemv
