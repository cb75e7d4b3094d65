// Products of MXFP4 experts with few rows each (mma.sync kernel).
//
// y[s][n] = sum_k w[n][k] x[s][k].  A code is a half exactly, so 16 rows of
// codes are the A operand of m16n8k16 as the pack has them (four conversions a
// word, no integer work), 8 rows of x the B operand, and a block's two
// products a sum of 32 terms in fp32 that its scale then multiplies: one fused
// multiply-add an output and block, exact but for the sum's own rounding.
// x as halves: fp16 rows are what they are; bf16 rows go by a power of two
// that brings the row's largest finite element to [2^14, 2^15), which keeps
// every element to 2^-39 of it (all eight bits of those within 2^-31); fp32
// rows are two such terms (22 bits and a sign) of elements within 2^-15.
//
// Bound by the weights' bytes: 17/32 of a byte a value, read once if an
// expert's rows fit one row tile of 8.  A warp streams units of 16 rows x 64 values of two
// tiles (gate's and up's, or neighbours of one weight: 2 x 544 B, contiguous over K)
// through a ring of its own in shared memory by asynchronous copies, `parts` warps
// of a CTA share a pair's K and add up through shared memory behind a barrier of their
// own, and a CTA runs through a contiguous range of (expert, row tile, pair), so that x is
// staged once for many tiles.  The ring runs ahead across tiles and experts.
// 64 experts of 1408 x 5120, gate and up, a bf16 row each: 490 MB in 90 us, 5.4 TB/s;
// six fp32 tokens of 6 of 64 experts, 199 MB in 53 us (two terms of x, uneven shares);
// one token, 46 MB in 19.4 us, of which 5 before the first product.
#pragma once

#include "mxfp4.cuh"

#include <type_traits>

namespace qgemv {

constexpr int MXS_WARPS = 16, MXS_THREADS = MXS_WARPS * 32;  // of a CTA, one an SM
constexpr int MXS_STAGES = 4;  // of a warp's ring, a unit of two tiles each
constexpr int MXS_ROWS = 8;    // of x at most in a row tile
constexpr int MXS_RED = 20;    // floats of a column of 16 in the exchange (no bank conflicts)

// Halves that a value of a row of x takes.
template <typename T>
constexpr int MX_TERMS = sizeof(T) == 4 ? 2 : 1;

struct MxsPlan {
    int rows;     // of x in a row tile
    int parts;    // warps that share a tile's K
    int x_bytes;  // of a staged row and term
    int grid;
    size_t smem;
};

// Where the row tiles' table lies in shared memory: after the rings, the exchange and the rows of x.
template <int TERMS>
__device__ __forceinline__ int* mxs_before(uint8_t* sm, const MxsPlan& p)
{
    return reinterpret_cast<int*>(sm + MXS_WARPS * MXS_STAGES * 2 * MX_UNIT_BYTES + MXS_WARPS * 2 * MXS_ROWS * MXS_RED * sizeof(float) +
                                  (size_t)p.rows * TERMS * p.x_bytes);
}

__device__ __forceinline__ void cp_async16(void* smem, const void* gmem)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem));
}
__device__ __forceinline__ void cp_async16(uint32_t smem, const void* gmem)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem));
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The eight codes of a word as halves, two for each byte.
__device__ __forceinline__ void e2m1_halves(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// The experts' row tiles: before[e] of them come before expert e's, whose
// slots are order[start[e]] .. order[start[e + 1] - 1].  Offsets that do not fit the
// slots are cut, and one below an earlier one counts as that, so that no slot is
// in two ranges and the row tiles are no more than the slots allow.
__device__ __forceinline__ int mx_clamped(const int32_t* offsets, int e, int slots)
{
    return max(0, min(slots, offsets[e]));
}

template <int THREADS>
__device__ int mx_row_tiles(const MxArgs& a, int rows, int* before, int* start, int* sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int base = 0, falls = 0;
    for (int lo = 0; lo < a.L.experts; lo += THREADS) {
        const int e = lo + threadIdx.x;
        int n = 0, s0 = 0, s1 = 0;
        if (e < a.L.experts) {
            s0 = mx_clamped(a.offsets, e, a.slots), s1 = mx_clamped(a.offsets, e + 1, a.slots);
            start[e] = s0;
            n = s1 > s0 ? (s1 - s0 + rows - 1) / rows : 0;
        }
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(~0u, s, o);
            if (lane >= o) s += up;
        }
        if (lane == 31) sums[warp] = s;
        falls |= __syncthreads_or(s1 < s0);
        int mine = base;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) mine += sums[w];
            base += sums[w];
        }
        if (e < a.L.experts) before[e] = mine + s - n;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        before[a.L.experts] = base;
        start[a.L.experts] = mx_clamped(a.offsets, a.L.experts, a.slots);
        if (falls)  // (not from a router: once more, one after another)
            for (int e = 0, all = 0; e < a.L.experts; ++e) {
                start[e + 1] = max(start[e], start[e + 1]);
                before[e] = all;
                before[e + 1] = all += (start[e + 1] - start[e] + rows - 1) / rows;
            }
    }
    __syncthreads();
    return before[a.L.experts];
}

// The slots that no expert has: rows of zeros, and no place among the partial
// results.
template <int MODE, typename O>
__device__ void mx_rest(const MxArgs& a, O* y, const int* start, unsigned int* status)
{
    const int lo = start[0], hi = start[a.L.experts];
    const int rest = lo + a.slots - hi;
    for (int i = blockIdx.x; i < rest; i += gridDim.x) {
        const int at = i < lo ? i : hi + i - lo;
        const int s = a.order ? a.order[at] : at;
        if (s < 0 || s >= a.slots) continue;
        if constexpr (MODE == MX_DOWN) {
            if (threadIdx.x == 0 && QG_OK(qg_in(s, 1, a.slots), status, 316)) a.place_of[s] = -1;
        } else {
            for (int n = threadIdx.x; n < a.L.N; n += blockDim.x)
                if (QG_OK(qg_in((int64_t)s * a.ldy + n, 1, (int64_t)a.slots * a.ldy), status, 310))
                    y[(int64_t)s * a.ldy + n] = from_f32<O>(0.0f);
        }
    }
}

// g / (1 + e^-g), below zero as g e^g / (1 + e^g): there e^-g would be infinite from -88 on, and
// the result, -5e-37 then, zero.  For outputs of 16 bits the fast exponential and
// quotient, (4 + 1.2 |g|) 2^-23 off.
template <typename T>
__device__ __forceinline__ float mx_silu(float g)
{
    if constexpr (sizeof(T) == 4) {
        const float t = expf(-fabsf(g));
        return (g < 0.0f ? g * t : g) / (1.0f + t);
    } else {
        const float t = __expf(-fabsf(g));
        return __fdividef(g < 0.0f ? g * t : g, 1.0f + t);
    }
}

// ---- rows of a weight with scales far apart ------------------------------------------
//
// What the products make of a row marked by 255 is anything, in that row alone; its results
// are then written over by these, a warp a row and slot: NaN, or fp32 sums of the blocks, apart
// by 64 powers of two.  Hardly ever needed (neighbouring blocks are about as large as one another), and
// slow: one row of the weights in 1000 makes a token's gate and up (64 experts of 1408 x 5120) 35 us for 20, 4096 tokens' 3.7 ms
// for 0.43.  Behind the products' loops, from hidden arguments, it takes none of their registers.

// The arguments with sizes that the compiler does not know for those of the products: what it
// could compute once for both would take registers of their loops.
__device__ __forceinline__ MxArgs mx_hidden(MxArgs a)
{
    asm volatile("" : "+r"(a.L.experts), "+r"(a.L.N), "+r"(a.L.K));
    return a;
}

// The largest scale byte of row r of a tile among blocks that are not all zeros, 255 if one is NaN.
// By a warp, four lanes a block.
__device__ __forceinline__ int mx_marked_top(const uint8_t* tile, int units, int r)
{
    const int lane = threadIdx.x & 31;
    int top = 0;
    for (int b = lane >> 2; b < 2 * units; b += 8) {
        const uint8_t* unit = tile + (b >> 1) * MX_UNIT_BYTES;
        const int at = (b & 1) * 2 + (r >> 3), e = unit[MX_UNIT_CODES + (r & 7) * 4 + at];
        const uint32_t word = *reinterpret_cast<const uint32_t*>(unit + (4 * (r & 7) + (lane & 3)) * 16 + at * 4);
        if ((word & 0x77777777u) || e == 255) top = max(top, e);
    }
    return __reduce_max_sync(~0u, top);
}

// Row r of a tile times a row of x, 2^p being what scale byte `top` stands for.  By a warp, four
// lanes a block.
template <typename X>
__device__ __forceinline__ float mx_marked_product(const uint8_t* tile, int units, int r, int top, int p, const X& x)
{
    const int lane = threadIdx.x & 31, t = lane & 3;
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = lane >> 2; b < 2 * units; b += 8) {
        const uint8_t* unit = tile + (b >> 1) * MX_UNIT_BYTES;
        const int at = (b & 1) * 2 + (r >> 3), l = max(0, top - (int)unit[MX_UNIT_CODES + (r & 7) * 4 + at]);
        uint32_t h[4];
        e2m1_halves(*reinterpret_cast<const uint32_t*>(unit + (4 * (r & 7) + t) * 16 + at * 4), h);
        float v[8], sum = 0.0f;
        x.values(b, t, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 w = __half22float2(*reinterpret_cast<const __half2*>(h + i));
            sum = fmaf(w.y, v[2 * i + 1], fmaf(w.x, v[2 * i], sum));
        }
        sum *= __uint_as_float((uint32_t)(127 - (l & 63)) << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j) part[j] += l >> 6 == j ? sum : 0.0f;
    }
    float y = 0.0f;
#pragma unroll
    for (int j = 3; j >= 0; --j) {
#pragma unroll
        for (int o = 16; o; o >>= 1) part[j] += __shfl_xor_sync(~0u, part[j], o);
        y += mul_pow2(part[j], max(-378, p + x.exponent - 64 * j));
    }
    return y;
}

// The outputs of row r of an expert's tile for the cnt slots from place s0 on, if it is marked.
// By a warp.
template <typename T, int MODE, typename O, typename X>
__device__ __forceinline__ void mx_marked_row(const MxArgs& a, O* y, int e, int tile, int r, int64_t s0, int cnt, X& x,
                                              unsigned int* status)
{
    constexpr bool PAIR = MODE == MX_GATE_UP;
    const int units = a.L.units(), n = tile * MX_TILE_N + r;
    if (tile >= a.L.tiles() || n >= a.L.N) return;
    const int64_t at = e * a.L.expert_bytes() + tile * a.L.tile_bytes();
    const uint8_t *w = a.w + at, *w2 = PAIR ? a.w2 + at : w;
    const uint8_t mark = w[units * MX_UNIT_BYTES + r], mark2 = w2[units * MX_UNIT_BYTES + r];
    if (mark != 255 && mark2 != 255) return;
    // (the other of a pair need not be marked: its bytes are 127 - l)
    const int top = mark == 255 ? mx_marked_top(w, units, r) : 127, top2 = PAIR && mark2 == 255 ? mx_marked_top(w2, units, r) : 127;
    const bool nan = top == 255 || top2 == 255;
    const int p = (mark == 255 ? top : mark) - 127, p2 = (mark2 == 255 ? top2 : mark2) - 127;
    for (int c = 0; c < cnt; ++c) {
        const int s = x.take(c);
        if (s < 0) continue;
        float v = __uint_as_float(0x7FC00000u);
        if (!nan) {
            v = mx_marked_product(w, units, r, top, p, x);
            if constexpr (PAIR) v = mx_silu<T>(v) * mx_marked_product(w2, units, r, top2, p2, x);
        }
        const int64_t to = (MODE == MX_DOWN ? s0 + c : (int64_t)s) * a.ldy + n;
        if ((threadIdx.x & 31) == 0 && QG_OK(qg_in(to, 1, (int64_t)a.slots * a.ldy), status, 315)) y[to] = from_f32<O>(v);
    }
}

// Eight neighbouring values of a row (`wide`: 16-byte aligned), zeros from n on.
template <typename T>
__device__ __forceinline__ void mx_load8(const T* p, bool wide, int n, float (&v)[8])
{
    if (wide && n >= 8) {
        alignas(16) T t[8];
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(t)[i] = reinterpret_cast<const uint4*>(p)[i];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = to_f32(t[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < n ? to_f32(p[k]) : 0.0f;
    }
}

__device__ __forceinline__ uint32_t mx_halves(__half a, __half b)
{
    return (uint32_t)__half_as_ushort(a) | (uint32_t)__half_as_ushort(b) << 16;
}

// The power of two that a row goes by, from its largest finite magnitude's bits:
// 2^-e brings it to [2^14, 2^15), a subnormal one too (e: -163 .. 113).
__device__ __forceinline__ int mx_row_exponent(uint32_t top)
{
    return top == 0 ? 0 : top < 0x00800000u ? -132 - __clz((int)top) : (int)(top >> 23) - 141;
}

// 2^-e as two factors: fp32 numbers end at 2^127.
struct MxRowFactor {
    float a, b;
    __device__ explicit MxRowFactor(int e)
    {
        const int p = min(127, -e);
        a = __uint_as_float((uint32_t)(p + 127) << 23);
        b = __uint_as_float((uint32_t)(-e - p + 127) << 23);
    }
};

// Eight values times 2^-e as halves, and of fp32 values what that leaves.
template <typename T>
__device__ __forceinline__ void mx_row_halves(const float (&v)[8], const MxRowFactor& f, __half (&h)[8], __half (&l)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float y = v[j] * f.a * f.b;
        h[j] = __float2half_rn(y);
        if constexpr (MX_TERMS<T> == 2) l[j] = isfinite(y) ? __float2half_rn(y - __half2float(h[j])) : __float2half_rn(0.0f);
    }
}

// The cnt rows of a row tile into shared memory, as the product takes them: a
// block has 16 bytes for each t, values 4 t .. 4 t + 3 and 16 + 4 t .. 16 + 4 t
// + 3.  A warp takes 256 values of a row at a time, a lane eight neighbouring
// ones: half a piece of two t each.
template <typename T>
__device__ void mxs_stage(const MxArgs& a, const MxsPlan& p, uint8_t* xs, const int* slot_of, int* x_exp,
                          uint32_t* x_top, int cnt, unsigned int* status)
{
    constexpr int TERMS = MX_TERMS<T>;
    constexpr bool SCALED = !std::is_same<T, __half>::value;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int K = a.L.K, padded = a.L.units() * MX_UNIT_K, pieces = (padded + 255) / 256;
    const T* x = static_cast<const T*>(a.x);
    const bool wide = ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)(a.ldx * (int64_t)sizeof(T))) & 15u) == 0;
    if constexpr (SCALED) {
        for (int i = warp; i < cnt * pieces; i += MXS_WARPS) {
            const int row = i / pieces, k = (i - row * pieces) * 256 + lane * 8, s = max(0, slot_of[row]);
            float v[8];
            mx_load8(x + (int64_t)(s / a.x_div) * a.ldx + k, wide, max(0, K - k), v);
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t m = __float_as_uint(v[j]) & 0x7FFFFFFFu;
                top = max(top, m < 0x7F800000u ? m : 0u);
            }
            top = __reduce_max_sync(~0u, top);
            if (lane == 0) atomicMax(&x_top[row], top);
        }
        __syncthreads();
        if ((int)threadIdx.x < cnt) x_exp[threadIdx.x] = mx_row_exponent(x_top[threadIdx.x]);
        __syncthreads();
    }
    for (int i = warp; i < cnt * pieces; i += MXS_WARPS) {
        const int row = i / pieces, k = (i - row * pieces) * 256 + lane * 8, s = max(0, slot_of[row]);
        if (k >= padded) continue;
        float v[8];
        mx_load8(x + (int64_t)(s / a.x_div) * a.ldx + k, wide, max(0, K - k), v);
        uint8_t* to = xs + (size_t)row * TERMS * p.x_bytes;
        __half h[8], l[8];
        mx_row_halves<T>(v, MxRowFactor(SCALED ? x_exp[row] : 0), h, l);
        if (QG_OK(qg_in(k * 2, 16, p.x_bytes - 64) && row < p.rows, status, 313)) {
            const int q = (k >> 3) & 3;
            uint8_t* o = to + (k & ~31) * 2 + (q & 1) * 32 + (q >> 1) * 8;
            *reinterpret_cast<uint2*>(o) = make_uint2(mx_halves(h[0], h[1]), mx_halves(h[2], h[3]));
            *reinterpret_cast<uint2*>(o + 16) = make_uint2(mx_halves(h[4], h[5]), mx_halves(h[6], h[7]));
            if constexpr (TERMS == 2) {
                o += p.x_bytes;
                *reinterpret_cast<uint2*>(o) = make_uint2(mx_halves(l[0], l[1]), mx_halves(l[2], l[3]));
                *reinterpret_cast<uint2*>(o + 16) = make_uint2(mx_halves(l[4], l[5]), mx_halves(l[6], l[7]));
            }
        }
    }
    __syncthreads();
}

// Where a warp is in its CTA's range of (pairs of) tiles: tile `tile` of row tile rt, whose
// tiles below `end` are the CTA's, `left` tiles after those.  The warps of a tile
// take every step-th one from `first` on.
struct MxCursor {
    int64_t left;
    int rt, e, tile, end, tiles, first, step;
    __device__ void start(int64_t i0, int64_t i1, int all_tiles, int mine, int together, const int* before, int experts)
    {
        tiles = all_tiles;
        first = mine;
        step = together;
        rt = (int)(i0 / tiles);
        const int lo_tile = (int)(i0 - (int64_t)rt * tiles);
        end = (int)min((int64_t)tiles, lo_tile + (i1 - i0));
        left = i1 - i0 - (end - lo_tile);
        tile = lo_tile + first;
        int lo = 0, hi = experts - 1;  // the last expert with before[e] <= rt: it has that row tile
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (before[mid] <= rt) lo = mid;
            else hi = mid - 1;
        }
        e = lo;
    }
    // The next row tile of the range, if there is one.
    __device__ bool next_rows(const int* before)
    {
        if (left == 0) return false;
        ++rt;
        while (rt >= before[e + 1]) ++e;
        end = (int)min((int64_t)tiles, left);
        left -= end;
        tile = first;
        return true;
    }
};

// Rows of x as they are in memory, for mx_marked_row: take() goes to one, and returns its slot.
template <typename T>
struct MxsPlaceRows {
    const MxArgs& a;
    int place;
    const T* row = nullptr;
    int exponent = 0;
    __device__ int take(int c)
    {
        const int s = a.order ? a.order[place + c] : place + c;
        if (s < 0 || s >= a.slots) return -1;
        row = static_cast<const T*>(a.x) + (int64_t)(s / a.x_div) * a.ldx;
        if constexpr (!std::is_same<T, __half>::value) {
            uint32_t top = 0;
            for (int k = threadIdx.x & 31; k < a.L.K; k += 32) {
                const uint32_t m = __float_as_uint(to_f32(row[k])) & 0x7FFFFFFFu;
                top = max(top, m < 0x7F800000u ? m : 0u);
            }
            exponent = mx_row_exponent(__reduce_max_sync(~0u, top));
        }
        return s;
    }
    __device__ void values(int b, int t, float (&v)[8]) const
    {
        const MxRowFactor f(exponent);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 32 * b < a.L.K ? to_f32(row[32 * b + 4 * t + (i & 3) + (i >> 2) * 16]) * f.a * f.b : 0.0f;
    }
};

// The marked rows of a warp's tiles, once more.
template <typename T, int MODE>
__device__ __forceinline__ void mxs_marked_rows(const MxArgs& a, const MxsPlan& p, const int* before, unsigned int* status)
{
    using O = typename std::conditional<MODE == MX_DOWN, float, T>::type;
    constexpr int W = MODE == MX_GATE_UP ? 1 : 2;
    const int* start = before + a.L.experts + 1;
    const int warp = threadIdx.x >> 5, tiles = (a.L.tiles() + W - 1) / W;
    const int64_t items = (int64_t)before[a.L.experts] * tiles;
    MxCursor at;
    at.start(items * blockIdx.x / gridDim.x, items * (blockIdx.x + 1) / gridDim.x, tiles, warp / p.parts, MXS_WARPS / p.parts, before,
             a.L.experts);
    do {
        const int place = start[at.e] + (at.rt - before[at.e]) * p.rows, cnt = min(p.rows, start[at.e + 1] - place);
        MxsPlaceRows<T> rows{a, place};
        for (; at.tile < at.end; at.tile += at.step)
            for (int i = warp % p.parts; i < W * MX_TILE_N; i += p.parts)
                mx_marked_row<T, MODE>(a, static_cast<O*>(a.y), at.e, at.tile * W + i / MX_TILE_N, i % MX_TILE_N, place, cnt, rows, status);
    } while (at.next_rows(before));
}

// (A call leaves the registers of the loop before it alone, mostly: six fp32 tokens' down product takes
// 35.4 us with it, 37.1 without; their gate and up 55.9 and 53.4.)
template <typename T, int MODE>
__device__ __noinline__ void mxs_marked_call(MxArgs a, MxsPlan p, const int* before, unsigned int* status)
{
    mxs_marked_rows<T, MODE>(a, p, before, status);
}

template <typename T, int MODE>
__global__ void __launch_bounds__(MXS_THREADS, 1) mxs_kernel(MxArgs a, MxsPlan p, unsigned int* status)
{
    using O = typename std::conditional<MODE == MX_DOWN, float, T>::type;
    constexpr int TERMS = MX_TERMS<T>, WARPS = MXS_WARPS, STAGES = MXS_STAGES, COLS = MXS_ROWS;
    // two tiles at a time: gate's and up's, or neighbours of one weight
    constexpr int W = 2, STAGE = W * MX_UNIT_BYTES;
    constexpr bool PAIR = MODE == MX_GATE_UP;
    extern __shared__ __align__(16) uint8_t sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    uint8_t* ring = sm + warp * (STAGES * STAGE);
    float* red = reinterpret_cast<float*>(sm + WARPS * STAGES * STAGE);
    constexpr int RED_ONE = WARPS * W * COLS * MXS_RED;
    uint8_t* xs = reinterpret_cast<uint8_t*>(red + RED_ONE);
    int* before = mxs_before<TERMS>(sm, p);
    int* start = before + a.L.experts + 1;
    int* sums = start + a.L.experts + 1;
    int* slot_of = sums + 32;
    int* x_exp = slot_of + COLS;
    uint32_t* x_top = reinterpret_cast<uint32_t*>(x_exp + COLS);

    pdl_launch_dependents();
    pdl_wait();
    const int n_rt = mx_row_tiles<WARPS * 32>(a, p.rows, before, start, sums);
    O* y = static_cast<O*>(a.y);
    mx_rest<MODE>(a, y, start, status);

    const int parts = p.parts, together = WARPS / parts;  // tiles that the CTA works on at a time
    const int tiles = PAIR ? a.L.tiles() : (a.L.tiles() + 1) / 2, units = a.L.units();  // (pairs of tiles)
    const int64_t items = (int64_t)n_rt * tiles;
    const int64_t i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
    if (i0 >= i1) return;
    const int mine = warp / parts, part = warp % parts;
    const int u0 = units * part / parts, u1 = units * (part + 1) / parts;
    const int64_t tile_bytes = a.L.tile_bytes(), expert_bytes = a.L.expert_bytes();

    // Where a pair's two tiles start (one behind the last tile is the last again, and goes nowhere).
    auto tile_pair = [&](int e, int pair, const uint8_t*& w, const uint8_t*& w2) {
        if constexpr (PAIR) {
            w = a.w + e * expert_bytes + pair * tile_bytes;
            w2 = a.w2 + e * expert_bytes + pair * tile_bytes;
        } else {
            w = a.w + e * expert_bytes + 2 * pair * tile_bytes;
            w2 = 2 * pair + 1 < a.L.tiles() ? w + tile_bytes : w;
        }
    };
    MxCursor load;
    load.start(i0, i1, tiles, mine, together, before, a.L.experts);
    MxCursor at = load;

    int load_n = 0, load_stage = 0;  // units left of the item, stage of the next one
    bool load_more = u0 < u1;
    load.tile -= together;  // (one before the first)
    // this lane's 16 bytes of a unit's codes, of both tiles, and (lanes 0 .. 3) of their scales
    const uint8_t *lw = nullptr, *lw2 = nullptr, *ls = nullptr;
    const uint32_t ring_at = smem_u32(ring) + lane * 16;
    const uint32_t ring_scale = smem_u32(ring) + (lane >> 1) * MX_UNIT_BYTES + MX_UNIT_CODES + (lane & 1) * 16;
    // One more unit of the warp's stream into the ring (or an empty group at its end).
    auto issue = [&]() {
        while (load_n == 0 && load_more) {  // the next tile
            load.tile += together;
            if (load.tile >= load.end) {
                load_more = load.next_rows(before);
                load.tile -= together;
                continue;
            }
            const uint8_t *w = a.w, *w2 = a.w2;
            tile_pair(load.e, load.tile, w, w2);
            w += (int64_t)u0 * MX_UNIT_BYTES;
            w2 += (int64_t)u0 * MX_UNIT_BYTES;
            lw = w + lane * 16;
            lw2 = w2 + lane * 16;
            ls = (lane >= 2 ? w2 : w) + MX_UNIT_CODES + (lane & 1) * 16;
            load_n = u1 - u0;
        }
        if (load_n > 0) {
            const uint32_t to = load_stage * STAGE;
            if (QG_OK(qg_in(lw - lane * 16 - a.w, MX_UNIT_BYTES, a.L.bytes()), status, 311)) {
                cp_async16(ring_at + to, lw);
                cp_async16(ring_at + to + MX_UNIT_BYTES, lw2);
                if (lane < 4) cp_async16(ring_scale + to, ls);
            }
            lw += MX_UNIT_BYTES;
            lw2 += MX_UNIT_BYTES;
            ls += MX_UNIT_BYTES;
            --load_n;
            if (++load_stage == STAGES) load_stage = 0;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue();

    // the warps of a tile (a barrier of their own, so that tiles run on their own)
    auto together_barrier = [&]() {
        if (parts > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + mine), "r"(parts * 32) : "memory");
        else __syncwarp();
    };
    int stage = 0;
    bool marked = false;  // a row met
    do {
        __syncthreads();  // the rows before are done with
        const int place = start[at.e] + (at.rt - before[at.e]) * p.rows, cnt = min(p.rows, start[at.e + 1] - place);
        if (threadIdx.x < COLS) {
            int s = -1;
            if ((int)threadIdx.x < cnt) {
                s = a.order ? a.order[place + threadIdx.x] : place + (int)threadIdx.x;
                if (s < 0 || s >= a.slots) s = -1;
            }
            slot_of[threadIdx.x] = s;
            if (MODE == MX_DOWN && s >= 0 && QG_OK(qg_in(s, 1, a.slots), status, 317))
                a.place_of[s] = place + threadIdx.x;  // (whoever has this row tile writes the same)
            x_exp[threadIdx.x] = 0;
            x_top[threadIdx.x] = 0;
        }
        __syncthreads();
        mxs_stage<T>(a, p, xs, slot_of, x_exp, x_top, cnt, status);
        // (columns behind the last row repeat it and go nowhere)
        const uint8_t* xrow = xs + (size_t)min(g, cnt - 1) * TERMS * p.x_bytes + t * 16;
#pragma unroll 1
        for (; at.tile < at.end; at.tile += together) {
            // this lane's row of the tiles in the epilogue, and its scales
            const int n = at.tile * (PAIR ? MX_TILE_N : 2 * MX_TILE_N) + (lane & 15);
            int tops[2];
            {
                const uint8_t *w, *w2;
                tile_pair(at.e, at.tile, w, w2);
                tops[0] = w[(int64_t)units * MX_UNIT_BYTES + (lane & 15)];
                tops[1] = w2[(int64_t)units * MX_UNIT_BYTES + (lane & 15)];
            }
            float acc[W][4] = {};
#pragma unroll 1
            for (int u = u0; u < u1; ++u) {
                cp_async_wait<STAGES - 2>();
                __syncwarp();
                const uint8_t* from = ring + stage * STAGE;
                uint4 code[W];
                uint32_t scale[W];
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    code[w] = *reinterpret_cast<const uint4*>(from + w * MX_UNIT_BYTES + lane * 16);
                    scale[w] = *reinterpret_cast<const uint32_t*>(from + w * MX_UNIT_BYTES + MX_UNIT_CODES + g * 4);
                }
                if (++stage == STAGES) stage = 0;
                issue();  // (into the stage read one step ago: every lane has its words of it)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t ag[W][4], ah[W][4];
                    float sg[W], sh[W];
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        e2m1_halves(b ? code[w].z : code[w].x, ag[w]);
                        e2m1_halves(b ? code[w].w : code[w].y, ah[w]);
                        sg[w] = __uint_as_float((b ? scale[w] << 7 : scale[w] << 23) & 0x7F800000u);
                        sh[w] = __uint_as_float((b ? scale[w] >> 1 : scale[w] << 15) & 0x7F800000u);
                    }
                    uint4 x[TERMS];
#pragma unroll
                    for (int k = 0; k < TERMS; ++k)
                        x[k] = *reinterpret_cast<const uint4*>(xrow + (size_t)k * p.x_bytes + (2 * u + b) * 64);
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int k = 0; k < TERMS; ++k) {
                            mma_f16(c, ag[w][0], ah[w][0], ag[w][1], ah[w][1], x[k].x, x[k].y);
                            mma_f16(c, ag[w][2], ah[w][2], ag[w][3], ah[w][3], x[k].z, x[k].w);
                        }
                        fma_f32x2(acc[w][0], acc[w][1], c[0], c[1], sg[w], sg[w]);
                        fma_f32x2(acc[w][2], acc[w][3], c[2], c[3], sh[w], sh[w]);
                    }
                }
            }
            // the warps of a tile add up and write it on their own
            float* r = red + (warp - part) * (W * COLS * MXS_RED);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                float* c = r + ((part * W + w) * COLS + 2 * t) * MXS_RED + g;
                c[0] = acc[w][0];
                c[MXS_RED] = acc[w][1];
                c[8] = acc[w][2];
                c[MXS_RED + 8] = acc[w][3];
            }
            together_barrier();
            for (int c = 2 * part + (lane >> 4); c < cnt; c += 2 * parts) {
                if (slot_of[c] < 0) continue;
                const int64_t s = MODE == MX_DOWN ? place + c : slot_of[c];  // the output's row
                float v[W];
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float* from = r + (w * COLS + c) * MXS_RED + (lane & 15);
                    float sum = 0.0f;
#pragma unroll 4
                    for (int k = 0; k < parts; ++k) sum += from[k * (W * COLS * MXS_RED)];
                    v[w] = mul_pow2(sum, tops[w] - 127 + x_exp[c]);
                }
                if constexpr (PAIR) {
                    if (n < a.L.N && QG_OK(qg_in(s * a.ldy + n, 1, (int64_t)a.slots * a.ldy), status, 312))
                        y[s * a.ldy + n] = from_f32<O>(mx_silu<T>(v[0]) * v[1]);
                } else {
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        if (n + w * MX_TILE_N < a.L.N && QG_OK(qg_in(s * a.ldy + n + w * MX_TILE_N, 1, (int64_t)a.slots * a.ldy), status, 314))
                            y[s * a.ldy + n + w * MX_TILE_N] = from_f32<O>(v[w]);
                }
            }
            together_barrier();
            marked |= tops[0] == 255 || tops[1] == 255;
        }
    } while (at.next_rows(before));
    cp_async_wait<0>();
    if (__any_sync(~0u, marked)) {  // (the warps of a tile have met the same)
        uint32_t zero = 0;
        asm volatile("" : "+r"(zero));
        const int* table = mxs_before<TERMS>(sm + zero, p);
        if constexpr (PAIR) mxs_marked_rows<T, MODE>(mx_hidden(a), p, table, status);
        else mxs_marked_call<T, MODE>(a, p, table, status);
    }
}

}  // namespace qgemv
