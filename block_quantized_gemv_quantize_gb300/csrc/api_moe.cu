// C ABI entry points of the MXFP4 format and of the sparse layer on it:
// host-side validation, then the launches on the caller's stream.
#include "mxfp4.cuh"

#include <cmath>

using namespace qgemv;

namespace {

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
uintptr_t type_bytes(int type) { return type == QGEMV_F32 ? 4 : 2; }
bool known_type(int type) { return type == QGEMV_F32 || type == QGEMV_F16 || type == QGEMV_BF16; }

int check_blocks(int64_t N, int K)
{
    if (N < 1 || K < 1 || K > MX_MAX_K) return QGEMV_INVALID_ARG;
    if (K % 32) return QGEMV_UNSUPPORTED_SHAPE;
    return N <= INT32_MAX / (K / 32) ? QGEMV_OK : QGEMV_INVALID_ARG;
}

int check_pack(int experts, int N, int K)
{
    if (experts < 1 || experts > MX_MAX_EXPERTS || N < 1 || N > MX_MAX_N || K < 1 || K > MX_MAX_K) return QGEMV_INVALID_ARG;
    return K % 32 ? QGEMV_UNSUPPORTED_SHAPE : QGEMV_OK;
}

int check_slots(int tokens, int top_k)
{
    return tokens < 0 || top_k < 1 || top_k > MX_MAX_TOP_K || (int64_t)tokens * top_k > (1 << 30) ? QGEMV_INVALID_ARG
                                                                                                  : QGEMV_OK;
}

int rows_call(bool quantize, int type, const void* rows, int64_t ld, const void* blocks, int64_t N, int K, void* stream)
{
    if (wait_timeouts_pending()) return QGEMV_WAIT_TIMEOUT;
    if (!rows || !blocks || !known_type(type)) return QGEMV_INVALID_ARG;
    const int st = check_blocks(N, K);
    if (st) return st;
    if (ld < K) return QGEMV_INVALID_ARG;
    if (!aligned_to(blocks, 16) || !aligned_to(rows, type_bytes(type))) return QGEMV_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return quantize ? launch_quantize_mxfp4(type, rows, ld, const_cast<void*>(blocks), N, K, s)
                    : launch_dequantize_mxfp4(type, blocks, const_cast<void*>(rows), ld, N, K, s);
}

int route_call(int type, RouteArgs a, void* workspace, size_t ws_bytes, void* stream)
{
    if (wait_timeouts_pending()) return QGEMV_WAIT_TIMEOUT;
    if (!a.ids || !a.offsets || !a.order) return QGEMV_INVALID_ARG;
    if (a.experts < 1 || a.experts > MX_MAX_EXPERTS) return QGEMV_INVALID_ARG;
    const int st = check_slots(a.tokens, a.top_k);
    if (st) return st;
    const size_t need = route_workspace_bytes(a.tokens, a.experts);
    if (need && !workspace) return QGEMV_INVALID_ARG;
    if (ws_bytes < need) return QGEMV_WORKSPACE_TOO_SMALL;
    if (!aligned_to(a.ids, 4) || !aligned_to(a.weights, 4) || !aligned_to(a.offsets, 4) || !aligned_to(a.order, 4) ||
        !aligned_to(a.logits, type_bytes(type)) || (need && !aligned_to(workspace, 16)))
        return QGEMV_MISALIGNED;
    a.counts = static_cast<int32_t*>(workspace);
    return launch_route(type, a, static_cast<cudaStream_t>(stream));
}

// Partial results, then each slot's place among them.
size_t parts_bytes(int64_t slots, int N) { return ((size_t)slots * N * sizeof(float) + 15) & ~(size_t)15; }
size_t places_bytes(int64_t slots) { return ((size_t)slots * sizeof(int32_t) + 15) & ~(size_t)15; }

size_t product_workspace(int mode, int type, int tokens, int top_k, int experts, int K, int N)
{
    if (!known_type(type) || check_slots(tokens, top_k) || check_pack(experts, N, K)) return 0;
    const int64_t slots = (int64_t)tokens * top_k;
    return (mode == MX_DOWN ? parts_bytes(slots, N) + places_bytes(slots) : 0) +
           (mx_many_rows(slots, experts, K) ? mx_planes_bytes(type, mode == MX_DOWN ? slots : tokens, K) : 0);
}

int product_call(int mode, int type, const void* w, const void* w2, const void* x, int64_t ldx, const int32_t* offsets,
                 const int32_t* order, const float* weights, void* y, int64_t ldy, void* workspace, size_t ws_bytes,
                 int tokens, int top_k, int experts, int K, int N, void* stream)
{
    if (wait_timeouts_pending()) return QGEMV_WAIT_TIMEOUT;
    if (!w || (mode == MX_GATE_UP && !w2) || !offsets || (mode == MX_DOWN && !weights) || !known_type(type))
        return QGEMV_INVALID_ARG;
    int st = check_pack(experts, N, K);
    if (st) return st;
    st = check_slots(tokens, top_k);
    if (st) return st;
    if (!order && top_k != 1) return QGEMV_INVALID_ARG;
    if (tokens == 0) return QGEMV_OK;
    if (!x || !y || ldx < K || ldy < N) return QGEMV_INVALID_ARG;
    const size_t need = product_workspace(mode, type, tokens, top_k, experts, K, N);
    if (need && !workspace) return QGEMV_INVALID_ARG;
    if (ws_bytes < need) return QGEMV_WORKSPACE_TOO_SMALL;
    if (!aligned_to(w, 16) || !aligned_to(w2, 16) || !aligned_to(x, type_bytes(type)) || !aligned_to(y, type_bytes(type)) ||
        !aligned_to(offsets, 4) || !aligned_to(order, 4) || !aligned_to(weights, 4) || (need && !aligned_to(workspace, 16)))
        return QGEMV_MISALIGNED;
    MxArgs a{};
    a.w = static_cast<const uint8_t*>(w);
    a.w2 = static_cast<const uint8_t*>(w2);
    a.L = MxLayout{experts, N, K};
    a.x = x;
    a.ldx = ldx;
    a.offsets = offsets;
    a.order = order;
    a.slots = tokens * top_k;
    a.top_k = top_k;
    a.x_div = mode == MX_DOWN ? 1 : top_k;
    a.y = mode == MX_DOWN ? workspace : y;
    a.ldy = mode == MX_DOWN ? N : ldy;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (mode == MX_DOWN) {
        a.place_of = reinterpret_cast<int32_t*>(ws + parts_bytes(a.slots, N));
        ws += parts_bytes(a.slots, N) + places_bytes(a.slots);
    }
    a.planes = ws;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = launch_mx_gemm(mode, type, a, s);
    if (st || mode != MX_DOWN) return st;
    return launch_mx_combine(type, static_cast<const float*>(workspace), a.place_of, order, weights, y, ldy, tokens, top_k,
                             N, s);
}

}  // namespace

extern "C" {

size_t mxfp4_bytes(int64_t N, int K) { return check_blocks(N, K) ? 0 : (size_t)N * (K / 32) * MX_BYTES; }

size_t mxfp4_pack_bytes(int experts, int N, int K)
{
    return check_pack(experts, N, K) ? 0 : (size_t)MxLayout{experts, N, K}.bytes();
}

int quantize_mxfp4(int type, const void* x, int64_t ldx, void* blocks, int64_t N, int K, void* stream)
{
    return rows_call(true, type, x, ldx, blocks, N, K, stream);
}

int dequantize_mxfp4(int type, const void* blocks, void* y, int64_t ldy, int64_t N, int K, void* stream)
{
    return rows_call(false, type, y, ldy, blocks, N, K, stream);
}

int qpack_mxfp4(const void* w_canon, void* w_pack, int experts, int N, int K, void* stream)
{
    if (wait_timeouts_pending()) return QGEMV_WAIT_TIMEOUT;
    if (!w_canon || !w_pack) return QGEMV_INVALID_ARG;
    const int st = check_pack(experts, N, K);
    if (st) return st;
    if (!aligned_to(w_canon, 16) || !aligned_to(w_pack, 16)) return QGEMV_MISALIGNED;
    return launch_qpack_mxfp4(w_canon, w_pack, MxLayout{experts, N, K}, static_cast<cudaStream_t>(stream));
}

size_t moe_route_workspace_bytes(int tokens, int experts, int top_k)
{
    if (experts < 1 || experts > MX_MAX_EXPERTS || check_slots(tokens, top_k)) return 0;
    return route_workspace_bytes(tokens, experts);
}

int moe_route(int type, const void* logits, int64_t ld, int32_t* ids, float* weights, int32_t* offsets, int32_t* order,
              void* workspace, size_t ws_bytes, int tokens, int experts, int top_k, int score, int renormalize,
              float scale, void* stream)
{
    if ((!logits && tokens) || !weights || !known_type(type) || ld < experts || top_k > experts ||
        (score != QGEMV_SOFTMAX && score != QGEMV_SIGMOID) || !std::isfinite(scale))
        return QGEMV_INVALID_ARG;
    RouteArgs a{};
    a.logits = logits ? logits : weights;  // (no token: not read)
    a.ld = ld;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.order = order;
    a.tokens = tokens;
    a.experts = experts;
    a.top_k = top_k;
    a.sigmoid = score == QGEMV_SIGMOID;
    a.renormalize = renormalize != 0;
    a.scale = scale;
    return route_call(type, a, workspace, ws_bytes, stream);
}

int moe_group(const int32_t* ids, int32_t* offsets, int32_t* order, void* workspace, size_t ws_bytes, int tokens,
              int experts, int top_k, void* stream)
{
    RouteArgs a{};
    a.ids = const_cast<int32_t*>(ids);
    a.offsets = offsets;
    a.order = order;
    a.tokens = tokens;
    a.experts = experts;
    a.top_k = top_k;
    return route_call(QGEMV_F32, a, workspace, ws_bytes, stream);
}

size_t qgemm_mxfp4_workspace_bytes(int type, int tokens, int top_k, int experts, int K, int N)
{
    return product_workspace(MX_GEMM, type, tokens, top_k, experts, K, N);
}

size_t moe_gate_up_mxfp4_workspace_bytes(int type, int tokens, int top_k, int experts, int K, int N)
{
    return product_workspace(MX_GATE_UP, type, tokens, top_k, experts, K, N);
}

size_t moe_down_mxfp4_workspace_bytes(int type, int tokens, int top_k, int experts, int K, int N)
{
    return product_workspace(MX_DOWN, type, tokens, top_k, experts, K, N);
}

int qgemm_mxfp4(int type, const void* w_pack, const void* x, int64_t ldx, const int32_t* offsets, const int32_t* order,
                void* y, int64_t ldy, void* workspace, size_t ws_bytes, int tokens, int top_k, int experts, int K, int N,
                void* stream)
{
    return product_call(MX_GEMM, type, w_pack, nullptr, x, ldx, offsets, order, nullptr, y, ldy, workspace, ws_bytes,
                        tokens, top_k, experts, K, N, stream);
}

int moe_gate_up_mxfp4(int type, const void* w_gate, const void* w_up, const void* x, int64_t ldx, const int32_t* offsets,
                      const int32_t* order, void* h, int64_t ldh, void* workspace, size_t ws_bytes, int tokens, int top_k,
                      int experts, int K, int N, void* stream)
{
    return product_call(MX_GATE_UP, type, w_gate, w_up, x, ldx, offsets, order, nullptr, h, ldh, workspace, ws_bytes,
                        tokens, top_k, experts, K, N, stream);
}

int moe_down_mxfp4(int type, const void* w_down, const void* h, int64_t ldh, const int32_t* offsets,
                   const int32_t* order, const float* weights, void* out, int64_t ldo, void* workspace, size_t ws_bytes,
                   int tokens, int top_k, int experts, int K, int N, void* stream)
{
    return product_call(MX_DOWN, type, w_down, nullptr, h, ldh, offsets, order, weights, out, ldo, workspace, ws_bytes,
                        tokens, top_k, experts, K, N, stream);
}

}  // extern "C"
