// attn_paged, the plain kernel: one CTA per (q row, q head), its warps over
// the positions in turn, an online softmax per warp, the warps joined in
// shared memory.
#include "kvcache.cuh"

namespace qgemv {
namespace {

constexpr int WARPS = 8;

template <int FMT, typename T, int NB>
__global__ void __launch_bounds__(WARPS * 32) attn_plain_kernel(const AttnArgs a, unsigned int* st)
{
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float s_m[WARPS], s_l[WARPS], s_o[WARPS][NB * 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    const int head = blockIdx.y, kvh = head / a.group;
    const int b = (int)(row / a.rows), i = (int)(row - (int64_t)b * a.rows);
    const AttnSpan sp(a, a.lens[b]);
    const int end = sp.end(i), begin = sp.begin(i);
    const T* q = static_cast<const T*>(a.q) + row * a.q_row + head * a.q_head;
    float qv[NB], o[NB], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
        qv[k] = to_f32(q[k * 32 + lane]) * a.scale;
        o[k] = 0.0f;
    }
    constexpr int CB = kv_code_bytes(FMT), HALF = kv_half_bytes(FMT, NB);
    auto value = [&](const uint8_t* half, int r, int k) {
        const uint8_t* c = half + (k * KV_TILE + r) * CB;
        if (FMT == QGEMV_KV_F16) return __half2float(reinterpret_cast<const __half*>(c)[lane]);
        const float d = __half2float(
            *reinterpret_cast<const __half*>(half + NB * KV_TILE * CB + (k * KV_TILE + kv_scale_place(r)) * 2));
        return d * (float)(FMT == QGEMV_KV_Q8_0 ? (int)c[lane] - 128 : (int)((c[lane & 15] >> ((lane & 16) / 4)) & 15) - 8);
    };
    for (int p = sp.first() + warp; p < sp.last(); p += WARPS) {
        const int page = a.table[b * a.ld_table + p / a.L.page_tokens];
        const int64_t off = a.L.tile_offset(page, kvh, p % a.L.page_tokens / KV_TILE);
        if (off < 0 || !QG_OK(qg_in(off, a.L.tile_bytes, a.L.bytes()), st, 721)) {
            l = __int_as_float(0x7fffffff);
            continue;
        }
        if (p < begin || p >= end) continue;
        const uint8_t* tile = a.cache + off;
        const int r = p % KV_TILE;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < NB; ++k) s = fmaf(qv[k], value(tile, r, k), s);
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float m2 = fmaxf(m, s), base = m2 == -INFINITY ? 0.0f : m2;
        const float old = expf(m - base), w = expf(s - base);
        m = m2;
        l = l * old + w;
#pragma unroll
        for (int k = 0; k < NB; ++k) o[k] = o[k] * old + w * value(tile + HALF, r, k);
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) s_o[warp][k * 32 + lane] = o[k];
    __syncthreads();
    float M = -INFINITY, L = sp.bad ? __int_as_float(0x7fffffff) : 0.0f;
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, s_m[w]);
    const float base = M == -INFINITY ? 0.0f : M;
    for (int w = 0; w < WARPS; ++w) L += s_l[w] * expf(s_m[w] - base);
    for (int k = threadIdx.x; k < NB * 32; k += WARPS * 32) {
        float v = 0.0f;
        for (int w = 0; w < WARPS; ++w) v += s_o[w][k] * expf(s_m[w] - base);
        static_cast<T*>(a.out)[row * a.o_row + head * a.o_head + k] = from_f32<T>(L == 0.0f ? 0.0f : v / L);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row * a.heads + head] = L == 0.0f ? -INFINITY : M + logf(L);
}

template <int FMT, typename T, int NB>
int launch(const AttnArgs& a, cudaStream_t s)
{
    if (launch_pdl(attn_plain_kernel<FMT, T, NB>, dim3((unsigned)(a.batch * a.rows), (unsigned)a.heads),
                   dim3(WARPS * 32), 0, s, a, wait_timeout_counter()) != cudaSuccess)
        return QGEMV_CUDA_ERROR;
    return cudaGetLastError() == cudaSuccess ? QGEMV_OK : QGEMV_CUDA_ERROR;
}

template <int FMT, typename T>
int launch_dim(const AttnArgs& a, cudaStream_t s)
{
    switch (a.L.nb) {
    case 2: return launch<FMT, T, 2>(a, s);
    case 3: return launch<FMT, T, 3>(a, s);
    case 4: return launch<FMT, T, 4>(a, s);
    default: return launch<FMT, T, 8>(a, s);
    }
}

template <int FMT>
int launch_type(int type, const AttnArgs& a, cudaStream_t s)
{
    if (type == QGEMV_F32) return launch_dim<FMT, float>(a, s);
    if (type == QGEMV_F16) return launch_dim<FMT, __half>(a, s);
    return launch_dim<FMT, __nv_bfloat16>(a, s);
}

}  // namespace

size_t attn_workspace_bytes(int, int, int, int, int) { return ATTN_COUNTER_BYTES; }

int launch_attn_paged(int fmt, int type, const AttnArgs& a, cudaStream_t s)
{
    if (fmt == QGEMV_KV_F16) return launch_type<QGEMV_KV_F16>(type, a, s);
    if (fmt == QGEMV_KV_Q8_0) return launch_type<QGEMV_KV_Q8_0>(type, a, s);
    return launch_type<QGEMV_KV_Q4_0>(type, a, s);
}

}  // namespace qgemv
