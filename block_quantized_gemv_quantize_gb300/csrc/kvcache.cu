// kv_write and kv_read: new tokens' keys and values into the block-quantized
// paged cache, and cache slots back into rows.
//
// Both are bound by memory once their index arithmetic is small beside it:
// (values * element size + values * (34/32 | 18/32 | 2)) bytes a direction.
// Four lanes take one block (32 values of one token, head and K or V), eight
// values each.  A warp takes four consecutive tokens and KV_PAIRS pairs of
// neighbouring blocks: tokens that follow one another in the cache then fill
// whole 128-byte lines of codes and share the 32 bytes of scales, a row is read or
// written 128 bytes (16-bit types) or 256 at a time, each lane has all its loads
// in flight at once, and the slot's division by the page is done once for all its
// pairs.  (Eight lanes a block, one block a lane at a time and 64-bit divisions a
// block were bound by instructions at a fourth of these rates.)
//
// 60000 tokens of 8 heads of 128 (GB/s read and written, of 6790 measured for a
// copy): kv_read 6.2 to 6.6 TB/s in every format and type but q4_0 to bf16 (5.8);
// kv_write 6.2 (fp32 to q8_0), 5.2 (fp32 to q4_0), 6.4 to 6.7 (to f16), and 3.8
// and 2.5 from bf16 to q8_0 and q4_0, where the instructions of the quantizing
// bound it: half of a warp's blocks hold a value on a code's border (kv_encode).
// (From fp32 to q4_0 and q8_0 four blocks' values do not fit the 64 registers that
// four CTAs an SM leave a thread: 24 and 12 bytes of them are spilled.)
#include "kvcache.cuh"

namespace qgemv {
namespace {

constexpr int KV_WARPS = 8, KV_THREADS = 32 * KV_WARPS;
constexpr int KV_TOKENS = 4 * KV_WARPS;  // of a CTA
constexpr int KV_CTAS = 16;              // least CTAs for an SM that long calls are cut into
constexpr int KV_PAIRS = 4;              // pairs of blocks of a warp, one for each lane of a quad

// The eight values of lane sub (0 .. 3) of a block: 8 sub .. 8 sub + 7, or in
// two runs, 4 sub .. + 3 and 16 + 4 sub .. + 3.  Two runs keep fp32 accesses of
// 16 bytes next to one another, and hold both nibbles of q4_0's bytes.
template <int FMT, typename T>
constexpr bool kv_two_runs = FMT == QGEMV_KV_Q4_0 || sizeof(T) == 4;

// Whether a CTA of kv_write goes through several chunks of a row.  It saves 5 to
// 10 % where the quantizing leaves registers for it; from 16-bit rows to q4_0 it
// costs 20 % (60000 tokens of 1024 values: 149 us against 124).
template <int FMT, typename T>
constexpr bool kv_write_loops = !(FMT == QGEMV_KV_Q4_0 && sizeof(T) == 2);

// A lane's eight values as they are in memory.
template <typename T>
struct alignas(16) KvRaw {
    T v[8];
};

template <bool RUNS, typename T>
__device__ __forceinline__ void load_lane(const T* p, int sub, bool wide, KvRaw<T>& x)
{
    if constexpr (RUNS && sizeof(T) == 4) {
        if (wide) {
            reinterpret_cast<uint4*>(x.v)[0] = reinterpret_cast<const uint4*>(p)[sub];
            reinterpret_cast<uint4*>(x.v)[1] = reinterpret_cast<const uint4*>(p)[4 + sub];
            return;
        }
    } else if constexpr (RUNS) {
        if (wide) {
            reinterpret_cast<uint2*>(x.v)[0] = reinterpret_cast<const uint2*>(p)[sub];
            reinterpret_cast<uint2*>(x.v)[1] = reinterpret_cast<const uint2*>(p)[4 + sub];
            return;
        }
    } else if (wide) {
        *reinterpret_cast<uint4*>(x.v) = reinterpret_cast<const uint4*>(p)[sub];
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) x.v[k] = p[RUNS ? 4 * sub + (k & 3) + 4 * (k & 4) : 8 * sub + k];
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

// The larger magnitude; NaN if either is.
__device__ __forceinline__ float max_abs(float a, float b)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
    return m;
}

// What the four lanes of a block's quad know of its values after the first
// pass: the largest magnitude (NaN if one is) and, for q4_0, twice the place of
// the first value that has it, plus its sign.
struct KvTop {
    float mag;
    int key;
    template <bool KEY>
    __device__ __forceinline__ void join(const KvTop& o)
    {
        if (KEY && (o.mag > mag || (o.mag == mag && o.key < key))) key = o.key;
        mag = max_abs(mag, o.mag);
    }
    template <bool KEY>
    __device__ __forceinline__ KvTop from(int lanes) const
    {
        return {__shfl_xor_sync(0xffffffffu, mag, lanes), KEY ? __shfl_xor_sync(0xffffffffu, key, lanes) : 0};
    }
};

// A lane's own eight values of a block.
template <int FMT, bool RUNS>
__device__ __forceinline__ KvTop kv_top(const float (&x)[8], int sub)
{
    KvTop t{fabsf(x[0]), 2 * (RUNS ? 4 : 8) * sub + (int)(__float_as_uint(x[0]) >> 31)};
#pragma unroll
    for (int k = 1; k < 8; ++k) {
        if (FMT == QGEMV_KV_Q4_0) {
            const int at = RUNS ? 4 * sub + (k & 3) + 4 * (k & 4) : 8 * sub + k;
            if (fabsf(x[k]) > t.mag) t.key = 2 * at + (int)(__float_as_uint(x[k]) >> 31);
        }
        t.mag = max_abs(t.mag, x[k]);
    }
    return t;
}

// The largest magnitude alone, of 16-bit values two at a time.
__device__ __forceinline__ float kv_top_pairs(const KvRaw<__half>& x)
{
    const __half2* p = reinterpret_cast<const __half2*>(x.v);
    const __half2 m = __hmax2_nan(__hmax2_nan(__habs2(p[0]), __habs2(p[1])), __hmax2_nan(__habs2(p[2]), __habs2(p[3])));
    return max_abs(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float kv_top_pairs(const KvRaw<__nv_bfloat16>& x)
{
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(x.v);
    const __nv_bfloat162 m =
        __hmax2_nan(__hmax2_nan(__habs2(p[0]), __habs2(p[1])), __hmax2_nan(__habs2(p[2]), __habs2(p[3])));
    return max_abs(__low2float(m), __high2float(m));
}

// Four blocks' tops over the quad: lane sub gets that of block sub.
template <bool KEY>
__device__ __forceinline__ KvTop kv_scatter(const KvTop (&t)[4], int sub)
{
    const bool up = sub & 2, odd = sub & 1;
    KvTop a = up ? t[2] : t[0], b = up ? t[3] : t[1];
    a.join<KEY>((up ? t[0] : t[2]).from<KEY>(2));
    b.join<KEY>((up ? t[1] : t[3]).from<KEY>(2));
    KvTop own = odd ? b : a;
    own.join<KEY>((odd ? a : b).from<KEY>(1));
    return own;
}

// A block's d: NaN where a value is no number or infinite, 0 where all codes are
// to be those of zero.
template <int FMT>
__device__ __forceinline__ float kv_d(const KvTop& t)
{
    if (!(t.mag < INFINITY)) return __int_as_float(0x7fffffff);
    return FMT == QGEMV_KV_Q8_0 ? __fdiv_rn(t.mag, 127.0f) : __fmul_rn(t.key & 1 ? -t.mag : t.mag, -0.125f);
}

// Adding 3 * 2^22 rounds a number below 2^22 to a whole one, which then stands
// in the low bits; the format's offset (128 or 8) goes in with it.
constexpr float KV_ROUND = 12582912.0f;

// A lane's eight values of a block -> its code words (q4_0: one), given d and
// kv_inverse(d); by all lanes of the warp, `d` standing in lane `from` of it.
//
// The code is defined by the fp32 quotient x / d.  y = x * (1 / d) differs from
// it by less than 2^-15 (two roundings of at most 2^-24 against one, |x / d| <=
// 127), so the two round to the same code unless y lies within 2^-14 of where
// the code changes.  bf16 rows often have such values (their quotients are
// ratios of 8-bit numbers), so a division there costs as much as all the rest;
// two corrections y += (x - y d) (1 / d) give the same fp32 number: after the
// first y is within one unit of x / d, and the second is then exactly the
// rounded quotient where 1 / d is the correctly rounded inverse of a d whose
// mantissa is not all ones (P. W. Markstein, IBM J. Res. Dev. 34, 1990).
// Blocks without such an inverse divide.
__device__ __forceinline__ float kv_inverse(float d)
{
    if (d == 0.0f) return 0.0f;
    const bool odd = (__float_as_uint(d) & 0x7fffffu) == 0x7fffffu;  // (a NaN d among them)
    return fabsf(d) >= 0x1p-100f && !odd ? __frcp_rn(d) : INFINITY;
}

template <int FMT>
__device__ __forceinline__ void kv_encode(const float (&x)[8], float d, float inverse, int from, uint32_t (&word)[2])
{
    constexpr bool Q8 = FMT == QGEMV_KV_Q8_0;
    constexpr float magic = KV_ROUND + (Q8 ? 128.0f : 8.0f);
    const float inv = __shfl_sync(0xffffffffu, inverse, from);
    uint32_t n[8];
    float off = fabsf(inv) == INFINITY ? 1.0f : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        float y0, y1, r0, r1, w0 = magic, w1 = magic;
        mul_f32x2(y0, y1, x[k], x[k + 1], inv, inv);
        if (!Q8) y0 = fminf(y0, 7.25f), y1 = fminf(y1, 7.25f);  // from 7 on the code is 15
        add_f32x2(r0, r1, y0, y1, magic, magic);
        fma_f32x2(w0, w1, r0, r1, -1.0f, -1.0f);
        add_f32x2(w0, w1, w0, w1, y0, y1);  // y less the whole number
        off = fmaxf(off, fmaxf(fabsf(w0), fabsf(w1)));
        n[k] = __float_as_uint(r0), n[k + 1] = __float_as_uint(r1);
    }
    auto code = [](float q) {
        return Q8 ? (uint32_t)(max(-127, min(127, (int)roundf(q))) + 128)
                  : (uint32_t)max(0, min(15, (int)floorf(__fadd_rn(q, 8.5f))));
    };
    const bool far = off > 0.5f - 0x1p-14f;
    float dd = 0.0f;
    if (__any_sync(0xffffffffu, far)) {
        dd = __shfl_sync(0xffffffffu, d, from);
        if (far) {
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                float q0, q1;
                mul_f32x2(q0, q1, x[k], x[k + 1], inv, inv);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float r0 = x[k], r1 = x[k + 1];
                    fma_f32x2(r0, r1, q0, q1, -dd, -dd);
                    fma_f32x2(q0, q1, r0, r1, inv, inv);
                }
                n[k] = code(q0), n[k + 1] = code(q1);
            }
        }
    }
    word[0] = low_bytes(n[0], n[1], n[2], n[3]);
    word[1] = low_bytes(n[4], n[5], n[6], n[7]);
    if (inv == INFINITY) {  // one at a time: rare, and so without registers of its own
        word[0] = word[1] = 0;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
            float v = x[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) v = k == i ? x[i] : v;
            const uint32_t c = code(fabsf(dd) > 0.0f ? __fdiv_rn(v, dd) : 0.0f) << (8 * (k & 3));  // (no d: zeros)
            if (k < 4) word[0] |= c;
            else word[1] |= c;
        }
    }
    if (!Q8) word[0] |= word[1] << 4;
}

// A lane's token: where its rows are, and its place in the cache.
template <int FMT, typename T>
struct KvToken {
    T *k, *v;          // its rows
    uint8_t* codes;    // block 0 of head 0's K; null outside the cache
    uint32_t scales;   // from there to that block's scale
    bool in;
    __device__ __forceinline__ KvToken(const KvArgs& a, int64_t group, int lane)
    {
        const int64_t token = group * KV_TOKENS + (threadIdx.x >> 5) * 4 + (lane >> 3);
        in = token < a.n_tokens;
        const KvLayout::Slot at = a.L.slot(in ? a.slots[token] : -1);
        codes = at.page < 0 ? nullptr : a.cache + a.L.tile_offset(at.page, 0, at.tile) + at.row * kv_code_bytes(FMT);
        scales = a.L.nb * KV_TILE * kv_code_bytes(FMT) + 2 * kv_scale_place(at.row) - at.row * kv_code_bytes(FMT);
        k = static_cast<T*>(a.k.base) + token * a.k.token;
        v = static_cast<T*>(a.v.base) + token * a.v.token;
    }
};

// Block n of a token, in the order [K, V][head][block].
struct KvBlock {
    bool second;        // V
    uint32_t head, block;
    __device__ __forceinline__ KvBlock(const KvArgs& a, uint32_t n)
    {
        const uint32_t per = (uint32_t)(a.L.heads * a.L.nb);
        second = n >= per;
        if (second) n -= per;
        head = a.L.nb == 1 ? n : __umulhi(n, a.nb_inverse);
        block = n - head * (uint32_t)a.L.nb;
    }
    // from a token's first code to this block's (a page is below 4 GB)
    template <int FMT>
    __device__ __forceinline__ uint32_t codes(const KvArgs& a) const
    {
        return head * a.head_bytes + (second ? (uint32_t)kv_half_bytes(FMT, a.L.nb) : 0u) +
               block * (KV_TILE * kv_code_bytes(FMT));
    }
    // from there to the scale, beyond KvToken::scales
    template <int FMT>
    __device__ __forceinline__ uint32_t scale() const { return block * KV_TILE * 2 - block * (KV_TILE * kv_code_bytes(FMT)); }
    template <int FMT, typename T>
    __device__ __forceinline__ T* row(const KvArgs& a, const KvToken<FMT, T>& t) const
    {
        return (second ? t.v : t.k) + (int64_t)head * (second ? a.v.head : a.k.head) + block * QK;
    }
};

template <int FMT, typename T>
__global__ void __launch_bounds__(KV_THREADS, 4) kv_write_kernel(const KvArgs a, unsigned int* st)
{
    constexpr bool RUNS = kv_two_runs<FMT, T>;
    constexpr int CODE = kv_code_bytes(FMT);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane & 3;
    const bool wide = a.k.wide<T>() && a.v.wide<T>();
    const int n_blocks = 2 * a.L.heads * a.L.nb;
    for (int64_t group = blockIdx.y; group * KV_TOKENS < a.n_tokens; group += gridDim.y) {
        const KvToken<FMT, T> t(a, group, lane);
        for (int chunk = blockIdx.x; chunk * 2 * KV_PAIRS < n_blocks; chunk += gridDim.x) {
            const int block0 = chunk * 2 * KV_PAIRS + (lane >> 2 & 1);
            KvRaw<T> raw[KV_PAIRS];
#pragma unroll
            for (int j = 0; j < KV_PAIRS; ++j) {
                const int n = block0 + 2 * j;
                if (t.codes && n < n_blocks) {
                    load_lane<RUNS>(KvBlock(a, n).row(a, t), sub, wide, raw[j]);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) raw[j].v[k] = from_f32<T>(0.0f);
                }
            }
            // the scales: lane sub of a quad works out pair sub's
            float d = 0.0f, inverse = 0.0f;
            if constexpr (FMT != QGEMV_KV_F16) {
                KvTop top[KV_PAIRS];
#pragma unroll
                for (int j = 0; j < KV_PAIRS; ++j) {
                    if constexpr (FMT == QGEMV_KV_Q8_0 && sizeof(T) == 2) {
                        top[j] = {kv_top_pairs(raw[j]), 0};
                    } else {
                        float x[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = to_f32(raw[j].v[k]);
                        top[j] = kv_top<FMT, RUNS>(x, sub);
                    }
                }
                d = kv_d<FMT>(kv_scatter<FMT == QGEMV_KV_Q4_0>(top, sub));
                inverse = kv_inverse(d);
                const int n = block0 + 2 * sub;
                if (t.codes && n < n_blocks) {
                    const KvBlock b(a, n);
                    uint8_t* scale = t.codes + b.codes<FMT>(a) + (t.scales + b.scale<FMT>());
                    if (QG_OK(qg_in(scale - a.cache, 2, a.L.bytes()), st, 742))  // (a NaN stays)
                        *reinterpret_cast<__half*>(scale) = __float2half_rn(fabsf(d) > 65504.0f ? copysignf(65504.0f, d) : d);
                }
            }
#pragma unroll
            for (int j = 0; j < KV_PAIRS; ++j) {
                const int n = block0 + 2 * j;
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = to_f32(raw[j].v[k]);
                uint32_t word[2];
                if constexpr (FMT != QGEMV_KV_F16) kv_encode<FMT>(x, d, inverse, (lane & 28) + j, word);  // shuffles: every lane
                if (!t.codes || n >= n_blocks) continue;
                uint8_t* codes = t.codes + KvBlock(a, n).codes<FMT>(a);
                if (!QG_OK(qg_in(codes - a.cache, CODE, a.L.bytes()), st, 741)) continue;
                if constexpr (FMT == QGEMV_KV_F16) {
                    store_lane<RUNS>(reinterpret_cast<__half*>(codes), sub, true, x);
                } else {
                    uint32_t* w = reinterpret_cast<uint32_t*>(codes);
                    if constexpr (FMT == QGEMV_KV_Q4_0) w[sub] = word[0];
                    else if constexpr (RUNS) w[sub] = word[0], w[4 + sub] = word[1];
                    else reinterpret_cast<uint2*>(codes)[sub] = make_uint2(word[0], word[1]);
                }
            }
            if constexpr (!kv_write_loops<FMT, T>) break;
        }
    }
}

// Four bytes as numbers less `offset`: 2^23 + byte is 0x4B000000 | byte.
__device__ __forceinline__ void kv_numbers(uint32_t w, float offset, float* v)
{
#pragma unroll
    for (int k = 0; k < 4; k += 2)
        add_f32x2(v[k], v[k + 1], __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + k)),
                  __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441 + k)), -(8388608.0f + offset), -(8388608.0f + offset));
}

template <int FMT, typename T>
__global__ void __launch_bounds__(KV_THREADS, 5) kv_read_kernel(const KvArgs a, unsigned int* st)
{
    constexpr bool RUNS = kv_two_runs<FMT, T>;
    constexpr int CODE = kv_code_bytes(FMT);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane & 3;
    const bool wide = a.k.wide<T>() && a.v.wide<T>();
    const int n_blocks = 2 * a.L.heads * a.L.nb;
    for (int64_t group = blockIdx.y; group * KV_TOKENS < a.n_tokens; group += gridDim.y) {
        const KvToken<FMT, T> t(a, group, lane);
        if (!t.in) continue;
        for (int chunk = blockIdx.x; chunk * 2 * KV_PAIRS < n_blocks; chunk += gridDim.x) {
            const int block0 = chunk * 2 * KV_PAIRS + (lane >> 2 & 1);
            uint32_t word[KV_PAIRS][FMT == QGEMV_KV_F16 ? 4 : 2];
            __half d[KV_PAIRS];
#pragma unroll
            for (int j = 0; j < KV_PAIRS; ++j) {
#pragma unroll
                for (uint32_t& w : word[j])  // zeros, for a slot outside the cache
                    w = FMT == QGEMV_KV_F16 ? 0u : (FMT == QGEMV_KV_Q8_0 ? 0x80808080u : 0x88888888u);
                d[j] = __half(0.0f);
                const int n = block0 + 2 * j;
                if (!t.codes || n >= n_blocks) continue;
                const KvBlock b(a, n);
                const uint8_t* codes = t.codes + b.codes<FMT>(a);
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
                    const uint8_t* scale = codes + (t.scales + b.scale<FMT>());
                    if (QG_OK(qg_in(scale - a.cache, 2, a.L.bytes()), st, 744)) d[j] = *reinterpret_cast<const __half*>(scale);
                }
            }
#pragma unroll
            for (int j = 0; j < KV_PAIRS; ++j) {
                const int n = block0 + 2 * j;
                if (n >= n_blocks) continue;
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
                    const float f = __half2float(d[j]);  // 11 bits times 8: exact
#pragma unroll
                    for (int k = 0; k < 8; k += 2) mul_f32x2(x[k], x[k + 1], x[k], x[k + 1], f, f);
                }
                store_lane<RUNS>(KvBlock(a, n).row(a, t), sub, wide, x);
            }
        }
    }
}

template <bool WRITE, int FMT, typename T>
int launch_kv(const KvArgs& a, cudaStream_t s)
{
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return QGEMV_CUDA_ERROR;
    const int64_t groups = ((int64_t)a.n_tokens + KV_TOKENS - 1) / KV_TOKENS;
    // A CTA goes through several chunks of its tokens' rows where that leaves
    // KV_CTAS for every SM, so that long calls find each slot's place once for many
    // blocks (131071 tokens of q8_0: 149 us with a CTA a chunk, 129 so).
    const int64_t chunks = (2 * a.L.heads * a.L.nb + 2 * KV_PAIRS - 1) / (2 * KV_PAIRS);
    int64_t each = groups * chunks / ((int64_t)di.sms * KV_CTAS);
    if ((WRITE && !kv_write_loops<FMT, T>) || each < 1) each = 1;
    const dim3 grid((unsigned)((chunks + each - 1) / each), (unsigned)(groups < 65535 ? groups : 65535));
    KvArgs args = a;
    args.head_bytes = (uint32_t)(a.L.tiles() * a.L.tile_bytes);
    args.nb_inverse = 0xffffffffu / (uint32_t)a.L.nb + 1;
    auto kern = WRITE ? kv_write_kernel<FMT, T> : kv_read_kernel<FMT, T>;
    if (launch_pdl(kern, grid, dim3(KV_THREADS), 0, s, args, wait_timeout_counter()) != cudaSuccess)
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
