// The block-quantized paged key-value cache: its layout (include/qgemv.h has
// the definition) and the element types of the rows that go in and out.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.cuh"

namespace qgemv {

constexpr int KV_TILE = 16;  // tokens per tile
constexpr int KV_MAX_PAGE = 1024, KV_MAX_HEADS = 1024, KV_MAX_DIM = 512;
constexpr int64_t KV_MAX_SLOTS = INT64_C(1) << 35;

// Bytes of one block's codes (32 values of one token) and of its scale.
__host__ __device__ constexpr int kv_code_bytes(int fmt)
{
    return fmt == QGEMV_KV_F16 ? 64 : (fmt == QGEMV_KV_Q8_0 ? 32 : 16);
}
__host__ __device__ constexpr int kv_scale_bytes(int fmt) { return fmt == QGEMV_KV_F16 ? 0 : 2; }

// K (or V) of one tile: codes [nb][16][block], then scales [nb][16].
__host__ __device__ constexpr int kv_half_bytes(int fmt, int nb)
{
    return nb * KV_TILE * (kv_code_bytes(fmt) + kv_scale_bytes(fmt));
}
__host__ __device__ constexpr int kv_tile_bytes(int fmt, int nb) { return 2 * kv_half_bytes(fmt, nb); }

// Where the scale of a tile's token r stands among the block's 16, so that a
// lane of the attention (whose four tokens are 4 i + (s ^ 3 (i & 1))) finds
// its four scales next to one another.
__host__ __device__ constexpr int kv_scale_place(int r) { return 4 * ((r & 3) ^ (3 * ((r >> 2) & 1))) + (r >> 2); }

struct KvLayout {
    int64_t n_pages;
    int page_tokens, heads, nb, tile_bytes;
    __host__ __device__ int tiles() const { return page_tokens / KV_TILE; }
    __host__ __device__ int64_t bytes() const { return n_pages * heads * tiles() * (int64_t)tile_bytes; }
    // byte offset of tile t of head h of a page; -1 outside the cache
    __host__ __device__ int64_t tile_offset(int64_t page, int h, int t) const
    {
        if (page < 0 || page >= n_pages || h < 0 || h >= heads || t < 0 || t >= tiles()) return -1;
        return ((page * heads + h) * tiles() + t) * (int64_t)tile_bytes;
    }
    // Where a slot is; page -1 outside the cache.  A cache has at most
    // KV_MAX_SLOTS of them, so that its tiles count in 31 bits.
    struct Slot {
        int64_t page;
        int tile, row;
    };
    __host__ __device__ Slot slot(int64_t s) const
    {
        if (s < 0 || s >= n_pages * page_tokens) return {-1, 0, 0};
        const uint32_t tile = (uint32_t)(s / KV_TILE), page = tile / (uint32_t)tiles();
        return {page, (int)(tile - page * (uint32_t)tiles()), (int)(s & (KV_TILE - 1))};
    }
    // byte offset of the tile that holds a slot
    __host__ __device__ int64_t slot_offset(int64_t s, int h) const
    {
        const Slot at = slot(s);
        return tile_offset(at.page, h, at.tile);
    }
};

inline __host__ __device__ KvLayout kv_layout(int fmt, int64_t n_pages, int page_tokens, int heads, int head_dim)
{
    KvLayout L;
    L.n_pages = n_pages;
    L.page_tokens = page_tokens;
    L.heads = heads;
    L.nb = head_dim / QK;
    L.tile_bytes = kv_tile_bytes(fmt, L.nb);
    return L;
}

// ---- rows of fp32, fp16 or bf16 values -------------------------------------

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N consecutive values; `wide`: p is aligned to N values (or to 16 bytes).
template <int N, typename T>
__device__ __forceinline__ void store_values(T* p, bool wide, const float (&v)[N])
{
    constexpr int BYTES = N * (int)sizeof(T), VEC = BYTES < 16 ? BYTES : 16, PER = VEC / (int)sizeof(T);
    static_assert(VEC == 8 || VEC == 16, "two or four words at a time");
    if (wide) {
#pragma unroll
        for (int i = 0; i < N / PER; ++i) {
            alignas(16) T t[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) t[k] = from_f32<T>(v[i * PER + k]);
            if constexpr (VEC == 16) reinterpret_cast<uint4*>(p)[i] = *reinterpret_cast<uint4*>(t);
            else reinterpret_cast<uint2*>(p)[i] = *reinterpret_cast<uint2*>(t);
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) p[k] = from_f32<T>(v[k]);
    }
}

// Rows (t, h) of one tensor: base + t * token + h * head elements.
struct KvRows {
    void* base;
    int64_t token, head;
    // every row starts on a 16-byte boundary
    template <typename T>
    __host__ __device__ bool wide() const
    {
        return ((reinterpret_cast<uintptr_t>(base) | (uintptr_t)(token * (int64_t)sizeof(T)) |
                 (uintptr_t)(head * (int64_t)sizeof(T))) & 15u) == 0;
    }
};

struct KvArgs {
    KvRows k, v;
    const int64_t* slots;
    uint8_t* cache;
    KvLayout L;
    int n_tokens;
    uint32_t head_bytes;  // of a page, for one head
    // ceil(2^32 / nb), nb > 1: the high word of n times it is n / nb (n below
    // 2^16 and nb below 2^5 leave an error below 2^-11)
    uint32_t nb_inverse;
};

int launch_kv_write(int fmt, int type, const KvArgs& a, cudaStream_t s);
int launch_kv_read(int fmt, int type, const KvArgs& a, cudaStream_t s);

// ---- attention ---------------------------------------------------------------

constexpr int ATTN_MAX_SPLITS = 2048;
constexpr size_t ATTN_RECORD_BYTES = (size_t)ATTN_MAX_SPLITS * 8;  // of the workspace, before the partial results

struct AttnRecord;

struct AttnArgs {
    const void* q;
    int64_t q_row, q_head;
    void* out;
    int64_t o_row, o_head;
    float* lse;
    const uint8_t* cache;
    KvLayout L;
    const int32_t* table;
    int64_t ld_table;
    const int32_t* lens;
    int max_pages;
    int batch, rows, heads, group;  // group: q heads per kv head
    float scale;
    int window;
    AttnRecord* records;
    float* partials;
};

size_t attn_workspace_bytes(int rows, int heads, int kv_heads, int head_dim);
int launch_attn_paged(int fmt, int type, const AttnArgs& a, cudaStream_t s);

// The positions that the rows of a sequence of `len` tokens see: row i sees
// [begin(i), end(i)), all of them [first, last).  A sequence longer than its
// page table is bad (its rows get NaN) and spans nothing.
struct AttnSpan {
    int len, rows, window;
    bool bad;
    __host__ __device__ AttnSpan(const AttnArgs& a, int kv_len) : rows(a.rows), window(a.window)
    {
        bad = kv_len > (int64_t)a.max_pages * a.L.page_tokens;
        len = bad || kv_len < 0 ? 0 : kv_len;
    }
    __host__ __device__ int end(int i) const { return len - (rows - 1 - i); }  // <= 0: the row sees nothing
    __host__ __device__ int begin(int i) const
    {
        const int e = end(i);
        return window > 0 && e > window ? e - window : 0;
    }
    __host__ __device__ int first() const { return begin(0); }  // no row sees further back than row 0
    __host__ __device__ int last() const { return len; }
};

}  // namespace qgemv
