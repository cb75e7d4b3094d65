// C ABI entry points of the paged key-value cache and the attention over it:
// host-side validation, then one enqueue on the caller's stream.
#include "kvcache.cuh"

#include <cmath>

using namespace qgemv;

namespace {

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
uintptr_t type_bytes(int type) { return type == QGEMV_F32 ? 4 : 2; }

int check_layout(int fmt, int page_tokens, int n_kv_heads, int head_dim)
{
    if (fmt != QGEMV_KV_F16 && fmt != QGEMV_KV_Q8_0 && fmt != QGEMV_KV_Q4_0) return QGEMV_INVALID_ARG;
    if (page_tokens < 1 || page_tokens > KV_MAX_PAGE || n_kv_heads < 1 || n_kv_heads > KV_MAX_HEADS || head_dim < 1 ||
        head_dim > KV_MAX_DIM)
        return QGEMV_INVALID_ARG;
    if (page_tokens % KV_TILE || head_dim % QK) return QGEMV_UNSUPPORTED_SHAPE;
    return QGEMV_OK;
}

// so that every offset in the cache is within 62 bits (a token of a cache has at
// most 2^21 bytes)
bool pages_fit(int64_t n_pages, int page_tokens)
{
    return n_pages >= 1 && n_pages <= KV_MAX_SLOTS / page_tokens;
}

int check_type(int type) { return type == QGEMV_F32 || type == QGEMV_F16 || type == QGEMV_BF16 ? QGEMV_OK : QGEMV_INVALID_ARG; }

// (write: k and v are read; read: written)
int kv_call(bool write, int fmt, int type, const void* k, int64_t k_token, int64_t k_head, const void* v,
            int64_t v_token, int64_t v_head, const int64_t* slots, const void* cache, int64_t n_pages, int page_tokens,
            int n_tokens, int n_kv_heads, int head_dim, void* stream)
{
    if (wait_timeouts_pending()) return QGEMV_WAIT_TIMEOUT;
    if (!k || !v || !slots || !cache || n_tokens < 0) return QGEMV_INVALID_ARG;
    int st = check_layout(fmt, page_tokens, n_kv_heads, head_dim);
    if (st) return st;
    st = check_type(type);
    if (st) return st;
    if (k_token < 0 || k_head < 0 || v_token < 0 || v_head < 0) return QGEMV_INVALID_ARG;
    if (!pages_fit(n_pages, page_tokens)) return QGEMV_INVALID_ARG;
    if (!aligned_to(cache, 16) || !aligned_to(slots, 8) || !aligned_to(k, type_bytes(type)) ||
        !aligned_to(v, type_bytes(type)))
        return QGEMV_MISALIGNED;
    if (n_tokens == 0) return QGEMV_OK;
    KvArgs a{};
    a.k = {const_cast<void*>(k), k_token, k_head};
    a.v = {const_cast<void*>(v), v_token, v_head};
    a.slots = slots;
    a.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
    a.L = kv_layout(fmt, n_pages, page_tokens, n_kv_heads, head_dim);
    a.n_tokens = n_tokens;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return write ? launch_kv_write(fmt, type, a, s) : launch_kv_read(fmt, type, a, s);
}

}  // namespace

extern "C" {

size_t kv_page_bytes(int fmt, int page_tokens, int n_kv_heads, int head_dim)
{
    if (check_layout(fmt, page_tokens, n_kv_heads, head_dim) != QGEMV_OK) return 0;
    return (size_t)n_kv_heads * (page_tokens / KV_TILE) * (size_t)kv_tile_bytes(fmt, head_dim / QK);
}

int64_t kv_tile_offset(int fmt, int64_t n_pages, int page_tokens, int n_kv_heads, int head_dim, int64_t slot, int head)
{
    const size_t page = kv_page_bytes(fmt, page_tokens, n_kv_heads, head_dim);
    if (!page || !pages_fit(n_pages, page_tokens)) return -1;
    return kv_layout(fmt, n_pages, page_tokens, n_kv_heads, head_dim).slot_offset(slot, head);
}

int kv_write(int fmt, int type, const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
             int64_t v_head, const int64_t* slots, void* cache, int64_t n_pages, int page_tokens, int n_tokens,
             int n_kv_heads, int head_dim, void* stream)
{
    return kv_call(true, fmt, type, k, k_token, k_head, v, v_token, v_head, slots, cache, n_pages, page_tokens,
                   n_tokens, n_kv_heads, head_dim, stream);
}

int kv_read(int fmt, int type, const void* cache, int64_t n_pages, int page_tokens, const int64_t* slots, void* k,
            int64_t k_token, int64_t k_head, void* v, int64_t v_token, int64_t v_head, int n_tokens, int n_kv_heads,
            int head_dim, void* stream)
{
    return kv_call(false, fmt, type, k, k_token, k_head, v, v_token, v_head, slots, cache, n_pages, page_tokens,
                   n_tokens, n_kv_heads, head_dim, stream);
}

size_t attn_paged_workspace_bytes(int type, int rows, int n_heads, int n_kv_heads, int head_dim)
{
    if (check_type(type) || rows < 1 || rows > QGEMV_MAX_M || n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads ||
        head_dim < QK || head_dim % QK)
        return 0;
    return attn_workspace_bytes(rows, n_heads, n_kv_heads, head_dim);
}

int attn_paged(int fmt, int type, const void* q, int64_t q_row, int64_t q_head, const void* cache, int64_t n_pages,
               int page_tokens, const int32_t* page_table, int64_t ld_table, int max_pages, const int32_t* kv_lens,
               void* out, int64_t o_row, int64_t o_head, float* lse, void* workspace, size_t ws_bytes, int batch,
               int rows, int n_heads, int n_kv_heads, int head_dim, float scale, int window, void* stream)
{
    if (wait_timeouts_pending()) return QGEMV_WAIT_TIMEOUT;
    if (!q || !cache || !page_table || !kv_lens || !out || !workspace) return QGEMV_INVALID_ARG;
    int st = check_layout(fmt, page_tokens, n_kv_heads, head_dim);
    if (st) return st;
    st = check_type(type);
    if (st) return st;
    if (batch < 1 || batch > 65536 || rows < 1 || max_pages < 1 || ld_table < max_pages || n_heads < 1 ||
        n_heads > (1 << 16) || !std::isfinite(scale) || window < 0 || q_row < 0 || q_head < 0 || o_row < 0 ||
        o_head < 0)
        return QGEMV_INVALID_ARG;
    if (rows > QGEMV_MAX_M || n_heads % n_kv_heads ||
        (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 256))
        return QGEMV_UNSUPPORTED_SHAPE;
    if (!pages_fit(n_pages, page_tokens) ||
        (int64_t)max_pages * page_tokens > (INT64_C(1) << 30))
        return QGEMV_INVALID_ARG;
    if (ws_bytes < attn_paged_workspace_bytes(type, rows, n_heads, n_kv_heads, head_dim))
        return QGEMV_WORKSPACE_TOO_SMALL;
    if (!aligned_to(cache, 16) || !aligned_to(workspace, 16) || !aligned_to(q, type_bytes(type)) ||
        !aligned_to(out, type_bytes(type)) || !aligned_to(page_table, 4) || !aligned_to(kv_lens, 4) ||
        !aligned_to(lse, 4))
        return QGEMV_MISALIGNED;
    AttnArgs a{};
    a.q = q;
    a.q_row = q_row;
    a.q_head = q_head;
    a.out = out;
    a.o_row = o_row;
    a.o_head = o_head;
    a.lse = lse;
    a.cache = static_cast<const uint8_t*>(cache);
    a.L = kv_layout(fmt, n_pages, page_tokens, n_kv_heads, head_dim);
    a.table = page_table;
    a.ld_table = ld_table;
    a.lens = kv_lens;
    a.max_pages = max_pages;
    a.batch = batch;
    a.rows = rows;
    a.heads = n_heads;
    a.group = n_heads / n_kv_heads;
    a.scale = scale;
    a.window = window;
    a.records = static_cast<AttnRecord*>(workspace);
    a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ATTN_RECORD_BYTES);
    return launch_attn_paged(fmt, type, a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
