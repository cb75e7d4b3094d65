// attn_paged: the workspace's size and the choice of the kernel (a translation
// unit for each cache format and type of the rows).
#include "attn_paged.cuh"

namespace qgemv {

int launch_attn_f16_f32(const AttnArgs& a, cudaStream_t s);
int launch_attn_f16_f16(const AttnArgs& a, cudaStream_t s);
int launch_attn_f16_bf16(const AttnArgs& a, cudaStream_t s);
int launch_attn_q8_0_f32(const AttnArgs& a, cudaStream_t s);
int launch_attn_q8_0_f16(const AttnArgs& a, cudaStream_t s);
int launch_attn_q8_0_bf16(const AttnArgs& a, cudaStream_t s);
int launch_attn_q4_0_f32(const AttnArgs& a, cudaStream_t s);
int launch_attn_q4_0_f16(const AttnArgs& a, cudaStream_t s);
int launch_attn_q4_0_bf16(const AttnArgs& a, cudaStream_t s);

// Records, then two partial results for every split: of an item that began
// before its piece, and of one that goes on after it.
size_t attn_workspace_bytes(int rows, int heads, int kv_heads, int head_dim)
{
    const int n = rows * (heads / kv_heads), nb = head_dim / QK, mode = attn_mode(n);
    const int per_tile = mode == ATTN_PAIR ? 8 : 16, most = ATTN_WARPS;
    const int tiles = (n + per_tile - 1) / per_tile, groups = (tiles + most - 1) / most, wr = (tiles + groups - 1) / groups;
    const size_t part = (size_t)(nb * 4 * (per_tile / 4) + 2 * (per_tile / 8)) * 32 * sizeof(float);
    return ATTN_RECORD_BYTES + (size_t)2 * ATTN_GRID * (most / wr) * wr * part;
}

int launch_attn_paged(int fmt, int type, const AttnArgs& a, cudaStream_t s)
{
    static_assert(QGEMV_KV_F16 == 0 && QGEMV_KV_Q8_0 == 1 && QGEMV_KV_Q4_0 == 2, "the order of the table");
    static_assert(QGEMV_F32 == 0 && QGEMV_F16 == 1 && QGEMV_BF16 == 2, "the order of the table");
    constexpr decltype(&launch_attn_f16_f32) by[3][3] = {{launch_attn_f16_f32, launch_attn_f16_f16, launch_attn_f16_bf16},
                                                         {launch_attn_q8_0_f32, launch_attn_q8_0_f16, launch_attn_q8_0_bf16},
                                                         {launch_attn_q4_0_f32, launch_attn_q4_0_f16, launch_attn_q4_0_bf16}};
    return by[fmt][type](a, s);
}

}  // namespace qgemv
