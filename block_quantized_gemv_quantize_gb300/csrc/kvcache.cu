// kv_write and kv_read: new tokens' keys and values into the block-quantized
// paged cache, and cache slots back into rows.
//
// Both are bound by memory once their index arithmetic is small beside it:
// (values * element size + values * (34/32 | 18/32 | 2)) bytes a direction.
// Four lanes take one block (32 values of one token, head and K or V), eight
// values each, so that a block's maximum takes two shuffles.  A warp takes four
// consecutive tokens and KV_PAIRS pairs of neighbouring blocks: tokens that
// follow one another in the cache then fill whole 128-byte lines of codes and
// share the 32 bytes of scales, a row is read or written 128 bytes (16-bit
// types) or 256 at a time, each lane has all its loads in flight at once, and
// the slot's division by the page is done once for all its pairs.
#include "kvcache.cuh"

namespace qgemv {
namespace {

constexpr int KV_WARPS = 8, KV_THREADS = 32 * KV_WARPS;
constexpr int KV_TOKENS = 4 * KV_WARPS;  // of a CTA
constexpr int KV_PAIRS = 4;              // pairs of blocks of a warp

// The eight values of lane sub (0 .. 3) of a block: 8 sub .. 8 sub + 7, or in
// two runs, 4 sub .. + 3 and 16 + 4 sub .. + 3.  Two runs keep fp32 accesses of
// 16 bytes next to one another, and hold both nibbles of q4_0's bytes.
template <int FMT, typename T>
constexpr bool kv_two_runs = FMT == QGEMV_KV_Q4_0 || sizeof(T) == 4;

template <bool RUNS, typename T>
__device__ __forceinline__ void load_lane(const T* p, int sub, bool wide, float (&v)[8])
{
    if constexpr (RUNS) {
        float lo[4], hi[4];
        load_values(p + 4 * sub, wide, lo);
        load_values(p + 16 + 4 * sub, wide, hi);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = lo[k], v[4 + k] = hi[k];
    } else {
        load_values(p + 8 * sub, wide, v);
    }
}

template <bool RUNS, typename T>
__device__ __forceinline__ void store_lane(T* p, int sub, bool wide, const float (&v)[8])
{
    if constexpr (RUNS) {
        const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
        store_values(p + 4 * sub, wide, lo);
        store_values(p + 16 + 4 * sub, wide, hi);
    } else {
        store_values(p + 8 * sub, wide, v);
    }
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Adding 3 * 2^22 rounds a number below 2^22 to a whole one, which then stands
// in the low bits; the format's offset (128 or 8) goes in with it.
constexpr float KV_ROUND = 12582912.0f;

// A lane's eight values of a block -> its code words (q4_0: one) and the
// block's scale; by all lanes of the warp, values beyond the rows being zero.
//
// The code is defined by the fp32 quotient x / d.  x * (1 / d) differs from it
// by less than 2^-15 (two roundings of at most 2^-24 against one, |x / d| <=
// 127), so the two round to the same code unless the product lies within 2^-13
// of where the code changes, or 1 / d overflows: those few lanes divide.
template <int FMT, bool RUNS>
__device__ __forceinline__ void kv_encode(float (&x)[8], int sub, uint32_t (&word)[2], float& scale)
{
    constexpr bool Q8 = FMT == QGEMV_KV_Q8_0;
    // magnitudes compare as integers, a NaN above an infinity above the rest
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool fine = top < 0x7f800000u;
    float d;
    if (Q8) {
        d = __fdiv_rn(__uint_as_float(top), 127.0f);
    } else {
        // the first value of that magnitude, and its sign
        int first = 64;
#pragma unroll
        for (int k = 7; k >= 0; --k) {
            const int at = RUNS ? 4 * sub + (k & 3) + 4 * (k & 4) : 8 * sub + k;
            const uint32_t bits = __float_as_uint(x[k]);
            if ((bits & 0x7fffffffu) == top) first = 2 * at + (int)(bits >> 31);
        }
        first = min(first, __shfl_xor_sync(0xffffffffu, first, 1));
        first = min(first, __shfl_xor_sync(0xffffffffu, first, 2));
        d = __fmul_rn(__uint_as_float(top | (uint32_t)(first & 1) << 31), -0.125f);
    }
    scale = fine ? fminf(fmaxf(d, -65504.0f), 65504.0f) : __int_as_float(0x7fffffff);
    const bool use = fine && d != 0.0f;
    const float inv = use ? __frcp_rn(d) : 0.0f;
    if (!fine) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = 0.0f;
    }
    constexpr float magic = KV_ROUND + (Q8 ? 128.0f : 8.0f);
    uint32_t n[8];
    float off = use && fabsf(d) < 0x1p-126f ? 1.0f : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float y = __fmul_rn(x[k], inv);
        if (!Q8) y = fminf(y, 7.25f);  // from 7 on the code is 15
        const float r = __fadd_rn(y, magic);
        off = fmaxf(off, fabsf(__fsub_rn(y, __fsub_rn(r, magic))));
        n[k] = __float_as_uint(r);
    }
    if (off > 0.5f - 0x1p-13f) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float y = __fdiv_rn(x[k], d);
            n[k] = Q8 ? (uint32_t)(max(-127, min(127, (int)roundf(y))) + 128)
                      : (uint32_t)max(0, min(15, (int)floorf(__fadd_rn(y, 8.5f))));
        }
    }
    word[0] = low_bytes(n[0], n[1], n[2], n[3]);
    word[1] = low_bytes(n[4], n[5], n[6], n[7]);
    if (!Q8) word[0] |= word[1] << 4;
}

// One lane's part of a unit of work: a token and, for pair j, a block.
struct KvPlace {
    int64_t token;
    KvLayout::Slot at;
    int block0, n_blocks;  // blocks in the order [K, V][head][block]
    bool in;
    __device__ __forceinline__ KvPlace(const KvArgs& a, int64_t group, int lane)
    {
        token = group * KV_TOKENS + (threadIdx.x >> 5) * 4 + (lane >> 3);
        in = token < a.n_tokens;
        at = a.L.slot(in ? a.slots[token] : -1);
        n_blocks = 2 * a.L.heads * a.L.nb;
        block0 = blockIdx.x * 2 * KV_PAIRS + (lane >> 2 & 1);
    }
};

struct KvBlock {
    int which, head, block;
    __device__ __forceinline__ KvBlock(const KvLayout& L, int n)
    {
        const int per = L.heads * L.nb;
        which = n >= per;
        n -= which * per;
        head = (int)((uint32_t)n / (uint32_t)L.nb);
        block = n - head * L.nb;
    }
    __device__ __forceinline__ int64_t element(const KvRows& r, int64_t token) const
    {
        return token * r.token + head * r.head + block * QK;
    }
};

template <int FMT, typename T>
__global__ void __launch_bounds__(KV_THREADS) kv_write_kernel(const KvArgs a, unsigned int* st)
{
    constexpr bool RUNS = kv_two_runs<FMT, T>;
    constexpr int CODE = kv_code_bytes(FMT);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane & 3;
    const bool wide = a.k.wide<T>() && a.v.wide<T>();
    for (int64_t group = blockIdx.y; group * KV_TOKENS < a.n_tokens; group += gridDim.y) {
        const KvPlace at(a, group, lane);
        float x[KV_PAIRS][8];
#pragma unroll
        for (int j = 0; j < KV_PAIRS; ++j) {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[j][k] = 0.0f;
            const int n = at.block0 + 2 * j;
            if (at.at.page < 0 || n >= at.n_blocks) continue;
            const KvBlock b(a.L, n);
            const KvRows& rows = b.which ? a.v : a.k;
            load_lane<RUNS>(static_cast<const T*>(rows.base) + b.element(rows, at.token), sub, wide, x[j]);
        }
#pragma unroll
        for (int j = 0; j < KV_PAIRS; ++j) {
            const int n = at.block0 + 2 * j;
            uint32_t word[2];
            float d;
            if constexpr (FMT != QGEMV_KV_F16) kv_encode<FMT, RUNS>(x[j], sub, word, d);  // shuffles: every lane
            if (at.at.page < 0 || n >= at.n_blocks) continue;
            const KvBlock b(a.L, n);
            uint8_t* half = a.cache + a.L.tile_offset(at.at.page, b.head, at.at.tile) + b.which * kv_half_bytes(FMT, a.L.nb);
            uint8_t* codes = half + (b.block * KV_TILE + at.at.row) * CODE;
            if (!QG_OK(qg_in(codes - a.cache, CODE, a.L.bytes()), st, 741)) continue;
            if constexpr (FMT == QGEMV_KV_F16) {
                store_lane<RUNS>(reinterpret_cast<__half*>(codes), sub, true, x[j]);
            } else {
                uint32_t* w = reinterpret_cast<uint32_t*>(codes);
                if constexpr (FMT == QGEMV_KV_Q4_0) w[sub] = word[0];
                else if constexpr (RUNS) w[sub] = word[0], w[4 + sub] = word[1];
                else reinterpret_cast<uint2*>(codes)[sub] = make_uint2(word[0], word[1]);
                uint8_t* scale = half + a.L.nb * KV_TILE * CODE + (b.block * KV_TILE + kv_scale_place(at.at.row)) * 2;
                if (sub == 0 && QG_OK(qg_in(scale - a.cache, 2, a.L.bytes()), st, 742))
                    *reinterpret_cast<__half*>(scale) = __float2half_rn(d);
            }
        }
    }
}

// Four bytes as numbers less `offset`: 2^23 + byte is 0x4B000000 | byte.
__device__ __forceinline__ void kv_numbers(uint32_t w, float offset, float* v)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + k)) - (8388608.0f + offset);
}

template <int FMT, typename T>
__global__ void __launch_bounds__(KV_THREADS) kv_read_kernel(const KvArgs a, unsigned int* st)
{
    constexpr bool RUNS = kv_two_runs<FMT, T>;
    constexpr int CODE = kv_code_bytes(FMT);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane & 3;
    const bool wide = a.k.wide<T>() && a.v.wide<T>();
    for (int64_t group = blockIdx.y; group * KV_TOKENS < a.n_tokens; group += gridDim.y) {
        const KvPlace at(a, group, lane);
        if (!at.in) continue;
        uint32_t word[KV_PAIRS][FMT == QGEMV_KV_F16 ? 4 : 2];
        __half d[KV_PAIRS];
#pragma unroll
        for (int j = 0; j < KV_PAIRS; ++j) {
#pragma unroll
            for (uint32_t& w : word[j]) w = 0;
            d[j] = __half(0.0f);
            const int n = at.block0 + 2 * j;
            if (at.at.page < 0 || n >= at.n_blocks) continue;
            const KvBlock b(a.L, n);
            const uint8_t* half = a.cache + a.L.tile_offset(at.at.page, b.head, at.at.tile) + b.which * kv_half_bytes(FMT, a.L.nb);
            const uint8_t* codes = half + (b.block * KV_TILE + at.at.row) * CODE;
            if (!QG_OK(qg_in(codes - a.cache, CODE, a.L.bytes()), st, 743)) continue;
            if constexpr (FMT == QGEMV_KV_F16) {
                const uint2* w = reinterpret_cast<const uint2*>(codes);
                const uint2 lo = w[RUNS ? sub : 2 * sub], hi = w[RUNS ? 4 + sub : 2 * sub + 1];
                word[j][0] = lo.x, word[j][1] = lo.y, word[j][2] = hi.x, word[j][3] = hi.y;
            } else {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(codes);
                if constexpr (FMT == QGEMV_KV_Q4_0) {
                    word[j][0] = w[sub];
                } else if constexpr (RUNS) {
                    word[j][0] = w[sub], word[j][1] = w[4 + sub];
                } else {
                    const uint2 both = reinterpret_cast<const uint2*>(codes)[sub];
                    word[j][0] = both.x, word[j][1] = both.y;
                }
                const uint8_t* scale = half + a.L.nb * KV_TILE * CODE + (b.block * KV_TILE + kv_scale_place(at.at.row)) * 2;
                if (QG_OK(qg_in(scale - a.cache, 2, a.L.bytes()), st, 744)) d[j] = *reinterpret_cast<const __half*>(scale);
            }
        }
#pragma unroll
        for (int j = 0; j < KV_PAIRS; ++j) {
            const int n = at.block0 + 2 * j;
            if (n >= at.n_blocks) continue;
            float x[8];
            if constexpr (FMT == QGEMV_KV_F16) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&word[j][k]));
                    x[2 * k] = f.x, x[2 * k + 1] = f.y;
                }
            } else {
                if constexpr (FMT == QGEMV_KV_Q4_0) {
                    kv_numbers(word[j][0] & 0x0F0F0F0Fu, 8.0f, x);
                    kv_numbers(word[j][0] >> 4 & 0x0F0F0F0Fu, 8.0f, x + 4);
                } else {
                    kv_numbers(word[j][0], 128.0f, x);
                    kv_numbers(word[j][1], 128.0f, x + 4);
                }
                const float f = __half2float(d[j]);
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] *= f;  // 11 bits times 8: exact
                if (at.at.page < 0) {                   // (zeros, not minus zeros)
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = 0.0f;
                }
            }
            const KvBlock b(a.L, n);
            const KvRows& rows = b.which ? a.v : a.k;
            store_lane<RUNS>(static_cast<T*>(rows.base) + b.element(rows, at.token), sub, wide, x);
        }
    }
}

template <bool WRITE, int FMT, typename T>
int launch_kv(const KvArgs& a, cudaStream_t s)
{
    const int64_t groups = ((int64_t)a.n_tokens + KV_TOKENS - 1) / KV_TOKENS;
    const dim3 grid((2 * a.L.heads * a.L.nb + 2 * KV_PAIRS - 1) / (2 * KV_PAIRS), (unsigned)(groups < 65535 ? groups : 65535));
    auto kern = WRITE ? kv_write_kernel<FMT, T> : kv_read_kernel<FMT, T>;
    if (launch_pdl(kern, grid, dim3(KV_THREADS), 0, s, a, wait_timeout_counter()) != cudaSuccess)
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
