// kv_write and kv_read: new tokens' keys and values into the block-quantized
// paged cache, and cache slots back into rows.
//
// Eight lanes take one block (32 values of one token, head and K or V), four
// values each: one 16-byte (fp32) or 8-byte load a lane, the block's maximum
// over three shuffles, and one store of the lane's codes.  Both are bound by
// memory: (values * element size + values * (34/32 | 18/32 | 2)) bytes.
#include "kvcache.cuh"

namespace qgemv {
namespace {

constexpr int KV_THREADS = 256;
constexpr int KV_GROUPS = KV_THREADS / 8;  // blocks a CTA holds at a time

// Four values of a block -> the lane's codes and the block's scale, by eight
// consecutive lanes (sub = lane & 7 holds values 4 sub .. 4 sub + 3).
struct KvCodes {
    uint32_t word;  // q8_0: four bytes; q4_0: the byte pairs' nibbles (sub < 4)
    float d;
};

template <int FMT>
__device__ __forceinline__ KvCodes kv_encode(const float (&x)[4], int lane)
{
    const int sub = lane & 7;
    // magnitudes compare as integers, a NaN above an infinity above the rest
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool fine = top < 0x7f800000u;
    float d;
    if (FMT == QGEMV_KV_Q8_0) {
        d = __fdiv_rn(__uint_as_float(top), 127.0f);
    } else {
        // the first value of that magnitude, with its sign
        int at = 32;
        float m = 0.0f;
#pragma unroll
        for (int i = 3; i >= 0; --i)
            if ((__float_as_uint(x[i]) & 0x7fffffffu) == top) {
                at = 4 * sub + i;
                m = x[i];
            }
        int first = at;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
        m = __shfl_sync(0xffffffffu, m, (lane & 24) + ((first >> 2) & 7));
        d = __fmul_rn(m, -0.125f);
    }
    const bool use = fine && d != 0.0f;
    KvCodes o;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float y = use ? __fdiv_rn(x[i], d) : 0.0f;
        if (FMT == QGEMV_KV_Q8_0) {
            const int q = max(-127, min(127, (int)roundf(y)));
            word |= (uint32_t)(q + 128) << (8 * i);
        } else {
            const int q = max(0, min(15, (int)floorf(__fadd_rn(y, 8.5f))));
            word |= (uint32_t)q << (8 * i);
        }
    }
    if (FMT == QGEMV_KV_Q4_0) word |= __shfl_xor_sync(0xffffffffu, word, 4) << 4;  // right for sub < 4
    o.word = word;
    o.d = fine ? fminf(fmaxf(d, -65504.0f), 65504.0f) : __int_as_float(0x7fffffff);
    return o;
}

// The (token, K or V, head, block) of a CTA's group of eight lanes: a CTA
// takes KV_GROUPS consecutive items of the order [token][K, V][head][block].
struct KvItem {
    int64_t token;
    int which, head, block;
    bool in;
};

__device__ __forceinline__ KvItem kv_item(const KvArgs& a, int64_t base, int group)
{
    const int per = 2 * a.L.heads * a.L.nb;  // items of one token
    const int64_t t0 = base / per;
    int r = (int)(base - t0 * per) + group;
    KvItem it;
    it.token = t0 + r / per;
    r %= per;
    it.which = r / (a.L.heads * a.L.nb);
    r -= it.which * (a.L.heads * a.L.nb);
    it.head = r / a.L.nb;
    it.block = r - it.head * a.L.nb;
    it.in = it.token < a.n_tokens;
    return it;
}

template <int FMT, typename T>
__global__ void __launch_bounds__(KV_THREADS) kv_write_kernel(const KvArgs a, unsigned int* st)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane & 7;
    const bool wide = a.k.wide<T>() && a.v.wide<T>();
    const int64_t total = (int64_t)a.n_tokens * 2 * a.L.heads * a.L.nb;
    for (int64_t base = (int64_t)blockIdx.x * KV_GROUPS; base < total; base += (int64_t)gridDim.x * KV_GROUPS) {
        const KvItem it = kv_item(a, base, threadIdx.x >> 3);
        const int64_t slot = it.in ? a.slots[it.token] : -1;
        const int64_t off = a.L.slot_offset(slot, it.head);
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (off >= 0) {
            const KvRows& rows = it.which ? a.v : a.k;
            const T* p = static_cast<const T*>(rows.base) + it.token * rows.token + it.head * rows.head +
                         it.block * QK + 4 * sub;
            load_values(p, wide, x);
        }
        uint8_t* half = a.cache + off + it.which * kv_half_bytes(FMT, a.L.nb);
        const int row = off >= 0 ? (int)(slot % KV_TILE) : 0;
        uint8_t* codes = half + (it.block * KV_TILE + row) * kv_code_bytes(FMT);
        if constexpr (FMT == QGEMV_KV_F16) {
            if (off < 0 || !QG_OK(qg_in(codes - a.cache, 64, a.L.bytes()), st, 701)) continue;
            const __half2 lo = __halves2half2(__float2half_rn(x[0]), __float2half_rn(x[1]));
            const __half2 hi = __halves2half2(__float2half_rn(x[2]), __float2half_rn(x[3]));
            uint2 w;
            w.x = *reinterpret_cast<const uint32_t*>(&lo);
            w.y = *reinterpret_cast<const uint32_t*>(&hi);
            reinterpret_cast<uint2*>(codes)[sub] = w;
        } else {
            const KvCodes c = kv_encode<FMT>(x, lane);  // every lane: shuffles inside
            if (off < 0 || !QG_OK(qg_in(codes - a.cache, kv_code_bytes(FMT), a.L.bytes()), st, 702)) continue;
            if (FMT == QGEMV_KV_Q8_0 || sub < 4) reinterpret_cast<uint32_t*>(codes)[sub] = c.word;
            uint8_t* scales = half + a.L.nb * KV_TILE * kv_code_bytes(FMT) +
                              (it.block * KV_TILE + kv_scale_place(row)) * 2;
            if (sub == 0 && QG_OK(qg_in(scales - a.cache, 2, a.L.bytes()), st, 703))
                *reinterpret_cast<__half*>(scales) = __float2half_rn(c.d);
        }
    }
}

template <int FMT, typename T>
__global__ void __launch_bounds__(KV_THREADS) kv_read_kernel(const KvArgs a, unsigned int* st)
{
    pdl_launch_dependents();
    pdl_wait();
    const int sub = threadIdx.x & 7;
    const bool wide = a.k.wide<T>() && a.v.wide<T>();
    const int64_t total = (int64_t)a.n_tokens * 2 * a.L.heads * a.L.nb;
    for (int64_t base = (int64_t)blockIdx.x * KV_GROUPS; base < total; base += (int64_t)gridDim.x * KV_GROUPS) {
        const KvItem it = kv_item(a, base, threadIdx.x >> 3);
        if (!it.in) continue;
        const int64_t slot = a.slots[it.token];
        const int64_t off = a.L.slot_offset(slot, it.head);
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (off >= 0 && QG_OK(qg_in(off, a.L.tile_bytes, a.L.bytes()), st, 711)) {
            const uint8_t* half = a.cache + off + it.which * kv_half_bytes(FMT, a.L.nb);
            const int row = (int)(slot % KV_TILE);
            const uint8_t* codes = half + (it.block * KV_TILE + row) * kv_code_bytes(FMT);
            if constexpr (FMT == QGEMV_KV_F16) {
                load_values(reinterpret_cast<const __half*>(codes) + 4 * sub, true, x);
            } else {
                const float d = __half2float(*reinterpret_cast<const __half*>(
                    half + a.L.nb * KV_TILE * kv_code_bytes(FMT) + (it.block * KV_TILE + kv_scale_place(row)) * 2));
                const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[FMT == QGEMV_KV_Q8_0 ? sub : sub & 3];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int q = FMT == QGEMV_KV_Q8_0 ? (int)((w >> (8 * i)) & 255u) - 128
                                                       : (int)((w >> (8 * i + (sub & 4))) & 15u) - 8;
                    x[i] = d * (float)q;  // 11 bits times 8: exact
                }
            }
        }
        const KvRows& rows = it.which ? a.v : a.k;
        T* p = static_cast<T*>(rows.base) + it.token * rows.token + it.head * rows.head + it.block * QK + 4 * sub;
        store_values(p, wide, x);
    }
}

template <bool WRITE, int FMT, typename T>
int launch_kv(const KvArgs& a, cudaStream_t s)
{
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return QGEMV_CUDA_ERROR;
    const int64_t total = (int64_t)a.n_tokens * 2 * a.L.heads * a.L.nb;
    int64_t grid = (total + KV_GROUPS - 1) / KV_GROUPS;
    if (grid > (int64_t)di.sms * 64) grid = (int64_t)di.sms * 64;
    auto kern = WRITE ? kv_write_kernel<FMT, T> : kv_read_kernel<FMT, T>;
    if (launch_pdl(kern, dim3((unsigned)grid), dim3(KV_THREADS), 0, s, a, wait_timeout_counter()) != cudaSuccess)
        return QGEMV_CUDA_ERROR;
    return cudaGetLastError() == cudaSuccess ? QGEMV_OK : QGEMV_CUDA_ERROR;
}

template <bool WRITE, int FMT>
int launch_kv_type(int type, const KvArgs& a, cudaStream_t s)
{
    if (type == QGEMV_F32) return launch_kv<WRITE, FMT, float>(a, s);
    if (type == QGEMV_F16) return launch_kv<WRITE, FMT, __half>(a, s);
    return launch_kv<WRITE, FMT, __nv_bfloat16>(a, s);
}

template <bool WRITE>
int launch_kv_fmt(int fmt, int type, const KvArgs& a, cudaStream_t s)
{
    if (fmt == QGEMV_KV_F16) return launch_kv_type<WRITE, QGEMV_KV_F16>(type, a, s);
    if (fmt == QGEMV_KV_Q8_0) return launch_kv_type<WRITE, QGEMV_KV_Q8_0>(type, a, s);
    return launch_kv_type<WRITE, QGEMV_KV_Q4_0>(type, a, s);
}

}  // namespace

int launch_kv_write(int fmt, int type, const KvArgs& a, cudaStream_t s) { return launch_kv_fmt<true>(fmt, type, a, s); }
int launch_kv_read(int fmt, int type, const KvArgs& a, cudaStream_t s) { return launch_kv_fmt<false>(fmt, type, a, s); }

}  // namespace qgemv
